// Host side of the router and the 8-bit floating point entry points: argument
// checks (before any HIP call), workspace layout and launch sequences.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>

#include "host.h"

using namespace chord;

namespace {

constexpr int kRouteMaxK = 32;
constexpr int kRouteMaxGroups = 64;
// One wave a token, and a launch has fewer than 2^32 threads.
constexpr int kRouteMaxTokens = 1 << 25;
// Codes of one expert are addressed with 32-bit offsets.
constexpr int64_t kMaxOperand = ((int64_t)1 << 31) - 1;

// How a dense product runs: the weight-streaming kernel (tiles of 16 tokens x 16
// outputs, K over the waves of a workgroup), or the tiled kernel with tile_rows
// tokens x 256 outputs and K in parts that a second launch adds.
struct F8GemmPlan {
  bool stream;
  int tile_rows;
  int parts;
};

// The cheapest by estimate, in us on an MI355X: a round of 256 workgroups takes
// 4 and so much per chunk, adding parts 4.5 and its bytes.  Fitted to sweeps
// over M = 1 .. 4096 with N = 128 .. 7168, K = 500 .. 7168; where both sides
// were near (within 10 %) it may pick the slower.  Measured, stream / tiled:
// M=17 N=7168 K=2048 10.0 / 11.9; M=32 N=4096 K=512 3.8 / 8.8, K=7168 16.6 / 15.9;
// M=100 N=576 K=7168 9.5 / 14.4, N=1024 K=1024 4.5 / 10.8, N=2112 K=7168 30.3 /
// 17.4; M=128 N=1024 K=4096 9.6 / 14.3, N=4096 K=512 7.2 / 10.3, K=7168 58 / 23;
// M=512 N=4096 rows x parts 64x2 32.9, 128x4 34.3, 256x8 41.6; M=2048 128x1 60.4,
// 256x2 78.9, 64x1 89.5.  Up to 128 rows a round of the streaming kernel is given
// what its chunks take and a launch of whole tiles 2.5 more; with more rows, where
// a weight tile is read again more than eight times, a round 3.5 besides (M=200
// N=4096 K=7168 89 / 25, N=2112 K=1024 9.5 / 11.7, N=1024 K=1024 5.8 / 11.0; M=400
// N=2112 K=1024 14.8 / 12.6: short K would gain from the former there, too).
F8GemmPlan f8_gemm_plan(int64_t M, int N, int K) {
  constexpr int64_t kCus = 256;  // (of the model, so that the workspace depends on sizes alone)
  const int nc = (int)f8_chunks(K);
  const int64_t tiles = f8_tiles(N), slices = (tiles + 15) / 16;
  F8GemmPlan best{true, 0, 1};
  if (M <= 16) return best;
  const int64_t streams = (M + 15) / 16 * tiles;
  double cost = 3.0 + std::max(1.0, (double)streams / kCus) * (3.5 + 0.09 * nc);
  const bool few = M <= 128;
  if (few) cost = std::min(cost, 3.0 + (double)((streams + kCus - 1) / kCus) * (0.1 + 0.113 * nc));
  const struct {
    int rows;
    double chunk;
  } shapes[] = {{64, 0.75}, {96, 0.85}, {128, 1.0}, {192, 1.42}, {256, 1.82}};
  for (const auto& s : shapes) {
    const int64_t items = (M + s.rows - 1) / s.rows * slices;
    for (int parts : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (parts > nc || (parts > 1 && items * parts > 2 * kCus)) break;
      const double rounds = (double)((items * parts + kCus - 1) / kCus);
      double c = rounds * (4.0 + (nc + parts - 1) / parts * s.chunk);
      if (parts > 1) c += 4.5 + parts * (double)M * tiles * 16 * 8 / 4e6;
      else if (few) c += 2.5;
      if (c < cost) {
        cost = c;
        best = F8GemmPlan{false, s.rows, parts};
      }
    }
  }
  return best;
}
size_t f8_gemm_ws(const F8GemmPlan& p, int64_t M, int N) {
  return p.parts > 1 ? (size_t)p.parts * M * f8_tiles(N) * 16 * sizeof(float) : 0;
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

chord_status check_shape(int role, int E, int N, int K) {
  if (role != CHORD_ROLE_GATE_UP && role != CHORD_ROLE_DOWN && role != CHORD_ROLE_PLAIN)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "role %d", role);
  if (E < 1 || N < 1 || K < 1) return fail(CHORD_ERR_INVALID_ARGUMENT, "E=%d N=%d K=%d", E, N, K);
  if (role == CHORD_ROLE_PLAIN) {
    if (E != 1) return fail(CHORD_ERR_UNSUPPORTED, "a plain weight has one matrix, not %d", E);
  } else {
    if (E > kMaxExperts) return fail(CHORD_ERR_UNSUPPORTED, "more than %d local experts", kMaxExperts);
    if (N % kF8Block != 0 || K % kF8Block != 0)
      return fail(CHORD_ERR_UNSUPPORTED, "N=%d and K=%d must be multiples of 128", N, K);
    if (role == CHORD_ROLE_GATE_UP && N % (2 * kF8Block) != 0)
      return fail(CHORD_ERR_UNSUPPORTED, "gate_up N=%d: I must be a multiple of 128", N);
  }
  if (K > 1 << 22) return fail(CHORD_ERR_UNSUPPORTED, "K=%d above 2^22", K);
  if ((int64_t)f8_tiles(N) * f8_chunks(K) * kF8BlockBytes > kMaxOperand)
    return fail(CHORD_ERR_UNSUPPORTED, "a weight of [%d, %d] exceeds 2 GiB", N, K);
  return CHORD_OK;
}

chord_status check_f8_weight(const chord_f8_weight* w, const char* name, int role) {
  if (!w) return fail(CHORD_ERR_INVALID_ARGUMENT, "%s is NULL", name);
  if (w->magic != CHORD_F8_WEIGHT_MAGIC || w->version != CHORD_F8_WEIGHT_VERSION)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "%s is not a packed 8-bit weight handle", name);
  if (!w->data) return fail(CHORD_ERR_INVALID_ARGUMENT, "%s has no data", name);
  if (w->role != role)
    return fail(CHORD_ERR_LAYOUT_MISMATCH, "%s has role %d, expected %d", name, w->role, role);
  if (w->block != kF8Block) return fail(CHORD_ERR_UNSUPPORTED, "%s block size %d", name, w->block);
  CHORD_CHECK(check_shape(w->role, w->num_experts, w->n, w->k));
  if (w->bytes < f8_packed_bytes(w->num_experts, w->n, w->k))
    return fail(CHORD_ERR_INVALID_ARGUMENT, "%s byte count too small", name);
  return CHORD_OK;
}

// The weight's part of a GEMM's arguments.
F8GemmArgs weight_args(const chord_f8_weight* w, int kind, int cus) {
  F8GemmArgs g{};
  g.kind = kind;
  g.wq = static_cast<const uint8_t*>(w->data);
  g.ws = reinterpret_cast<const float*>(g.wq + f8_code_bytes(w->num_experts, w->n, w->k));
  g.n_tiles = (int)f8_tiles(w->n);
  g.n_chunks = (int)f8_chunks(w->k);
  g.nb = (w->n + kF8Block - 1) / kF8Block;
  g.N = w->n;
  g.num_cus = cus;
  g.num_experts = w->num_experts;
  return g;
}

// ---- layer workspace --------------------------------------------------------
constexpr int kF8MaxBlockM = kF8SmallRows;  // rows per alignment block at most

struct F8Ws {
  size_t align, sorted, experts, ntpp, status, tiles, xq, xs, h, hq, hs, y, yu, total;
  int64_t max_padded;
  int max_tiles;
};

F8Ws f8_ws(int T, int k, int E_l, int H, int I) {
  F8Ws w{};
  w.max_padded = chord_moe_align_max_padded(T, k, E_l, kF8MaxBlockM);
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    const size_t o = off;
    off += ((size_t)bytes + 255) & ~(size_t)255;
    return o;
  };
  w.align = take((int64_t)chord_moe_align_workspace_bytes(T, k, E_l, kF8MaxBlockM));
  w.sorted = take(w.max_padded * 4);
  w.experts = take((w.max_padded + 15) / 16 * 4);
  w.ntpp = take(4);
  w.status = take(sizeof(DevStatus));
  w.max_tiles = (int)(w.max_padded / kF8MoeTileRows) + E_l + 1;
  w.tiles = take(w.max_tiles * sizeof(TileDesc));
  w.xq = take((int64_t)T * H);
  w.xs = take((int64_t)T * f8_chunks(H) * 4);
  w.hq = take(w.max_padded * I);
  w.hs = take(w.max_padded * f8_chunks(I) * 4);
  // (h in fp32 is quantised, or used up, before y is written.)
  const size_t both = off;
  w.h = take(w.max_padded * I * 4);
  const size_t h_end = off;
  off = both;
  w.y = take((int64_t)T * k * H * 2);
  w.yu = take((int64_t)T * k * H / 32);
  w.total = std::max(off, h_end);
  return w;
}

// How a layer call runs, from its expected rows per expert.
struct F8MoePlan {
  int block_m;          // rows per alignment block
  bool small;           // tiled GEMMs over the alignment blocks (else over built tiles)
  bool stream_gate_up;  // small: gate_up by the weight-streaming kernel
  bool exact;           // large: gate_up in fp32 sums (else they always are)
  int blocks;           // expected alignment blocks with rows
  const char* text;
};
// Measured over layers of H = 1024 .. 7168, I = 256 .. 2048 with 4 .. 384 experts,
// in us for a call:
// - gate_up by the streaming kernel, whose many small workgroups start at once,
//   as long as they are few (w < 3 a CU), else by tiles, which read a block's
//   tokens once (streaming / tiled): 4 experts of 7168 x 256 with 20 rows each
//   (w = 112) 34 / 54, with 120 (w = 272) 47 / 70; of 4096 x 1024 with 25 (w = 538)
//   41 / 50, with 100 (w = 1728) 86 / 87; 16 of 2048 x 768 with 12 (w = 921) 40 / 38.
// - Tiles over alignment blocks, two workgroups a CU and gate_up in fp32 sums, below
//   24 rows an expert, else tiles over up to 224 rows of an expert (blocks /
//   large): 16 rows 385 / 416 and 426 / 463, 24 rows 458 / 422 and 507 / 479 (48
//   experts of 7168 x 2048, 384 of 7168 x 256).  Also above where the blocks' tiles
//   leave a CU one workgroup, within 15 % either way and exact: 8 of 1024 x 512 with
//   50 rows 32 / 37, 16 of 640 x 768 with 50 33 / 38, 4 of 4096 x 1024 with 50 57 /
//   57 and with 100 67 / 60, 2 of 7168 x 1024 with 100 82 / 76; with more workgroups
//   it does not pay: 16 of 2048 x 768 with 100 84 / 57.
// - Blocks of 32 rows above 8 an expert (16 / 32 rows): 10.7 rows 392 / 372 and 441 /
//   402, 16 rows 530 / 385 and 588 / 426, 4 rows 353 / 355 and 363 / 367.
// - Large tiles: gate_up in fp32 sums below 64 rows an expert, where the weights' bytes
//   are still the bound, else summed by the 8-bit instruction (fp32 / 8-bit): 43 rows
//   443 / 443 and 552 / 556, 54 rows 455 / 454, 71 rows 498 / 483, 85 rows 532 / 504 and
//   716 / 703, 128 rows 658 / 568, 170 rows 797 / 634 (48 experts of 7168 x 2048, 384 of
//   7168 x 256); 100 rows 61 / 57 (16 of 2048 x 768).  CHORD_F8_FP32_SUMS=1
//   (environment, read once) takes fp32 sums at every size.
bool fp32_sums() {
  static const bool on = [] {
    const char* s = getenv("CHORD_F8_FP32_SUMS");
    return s != nullptr && atoi(s) != 0;
  }();
  return on;
}
F8MoePlan f8_moe_plan(int T, int k, int E_g, int E_l, int I, int cus) {
  const int eg = E_g > E_l ? E_g : E_l;
  const double tok_e = (double)T * k / eg;
  const double active = std::max(1.0, E_l * (1.0 - pow(1.0 - 1.0 / eg, (double)T * k)));
  const double rows = tok_e * E_l / active;  // of an expert with rows
  auto blocks = [&](int m) { return active * std::max(1.0, rows / m + 0.5); };
  F8MoePlan p{};
  p.stream_gate_up = blocks(16) * (2 * I / 32) < 3.0 * cus;
  p.small = p.stream_gate_up || tok_e < 24.0 || blocks(32) * (2 * I / 256) < cus;
  p.block_m = p.small && !p.stream_gate_up && tok_e > 8.0 ? 32 : 16;
  p.blocks = (int)std::min(blocks(p.block_m), 1e9);
  p.exact = tok_e < 64.0 || fp32_sums();
  p.text = !p.small ? "f8 moe: tiles of up to 224 rows"
           : p.stream_gate_up ? "f8 moe: blocks of 16 rows, streaming gate_up"
           : p.block_m == 16 ? "f8 moe: blocks of 16 rows" : "f8 moe: blocks of 32 rows";
  return p;
}

chord_status check_moe_sizes(int T, int k, int E_l, int H, int I) {
  if (T < 0 || k < 1 || E_l < 1 || H < 1 || I < 1)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "T=%d k=%d E_l=%d H=%d I=%d", T, k, E_l, H, I);
  if (H % kF8Block != 0 || I % kF8Block != 0)
    return fail(CHORD_ERR_UNSUPPORTED, "H=%d and I=%d must be multiples of 128", H, I);
  if (E_l > kMaxExperts) return fail(CHORD_ERR_UNSUPPORTED, "more than %d local experts", kMaxExperts);
  const int64_t slots = (int64_t)T * k;
  if (slots >= (int64_t)1 << 30) return fail(CHORD_ERR_UNSUPPORTED, "T*k=%lld", (long long)slots);
  // (Codes of x and h are loaded with 32-bit offsets; y is stored with 64-bit ones.)
  if ((int64_t)T * H > kMaxOperand) return fail(CHORD_ERR_UNSUPPORTED, "codes of x exceed 2 GiB");
  const int64_t rows = chord_moe_align_max_padded(T, k, E_l, kF8MaxBlockM);
  if (rows * I > kMaxOperand) return fail(CHORD_ERR_UNSUPPORTED, "codes of h exceed 2 GiB");
  return CHORD_OK;
}

}  // namespace

extern "C" {

chord_status chord_moe_route(const void* logits, int dtype, int64_t ld, int T, int E,
                             const float* bias, int k, int scoring, int n_group, int topk_group,
                             int renormalize, float scaling, int32_t* topk_ids,
                             float* topk_weights, void* stream) {
  clear_last_error();
  if (dtype != CHORD_DTYPE_F32 && dtype != CHORD_DTYPE_BF16 && dtype != CHORD_DTYPE_F16)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "dtype %d", dtype);
  if (scoring != CHORD_SCORE_SOFTMAX && scoring != CHORD_SCORE_SIGMOID)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "scoring %d", scoring);
  if (T < 0) return fail(CHORD_ERR_INVALID_ARGUMENT, "T=%d", T);
  if (E < 1 || E > kMaxExperts)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "E=%d (1..%d)", E, kMaxExperts);
  if (ld < E) return fail(CHORD_ERR_INVALID_ARGUMENT, "row stride %lld below E=%d", (long long)ld, E);
  if (n_group < 1 || n_group > kRouteMaxGroups || E % n_group != 0)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "n_group=%d must divide E=%d (1..%d)", n_group, E,
                kRouteMaxGroups);
  if (topk_group < 1 || topk_group > n_group)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "topk_group=%d (1..n_group=%d)", topk_group, n_group);
  if (k < 1 || k > kRouteMaxK || k > topk_group * (E / n_group))
    return fail(CHORD_ERR_INVALID_ARGUMENT, "k=%d (1..min(%d, %d experts to choose from))", k,
                kRouteMaxK, topk_group * (E / n_group));
  if (!std::isfinite(scaling))
    return fail(CHORD_ERR_INVALID_ARGUMENT, "scaling is not finite");
  if (T > kRouteMaxTokens) return fail(CHORD_ERR_UNSUPPORTED, "T=%d above %d", T, kRouteMaxTokens);
  if (T == 0) return CHORD_OK;
  if (!logits || !topk_ids || !topk_weights)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "null pointer argument");
  CHORD_CHECK(check_device(nullptr));
  RouteArgs a{};
  a.logits = logits;
  a.dtype = dtype;
  a.ld = ld;
  a.T = T;
  a.E = E;
  a.k = k;
  a.bias = bias;
  a.sigmoid = scoring == CHORD_SCORE_SIGMOID;
  a.n_group = n_group;
  a.topk_group = topk_group;
  const uint32_t per = (uint32_t)(E / n_group);
  a.group_magic = ((1u << 20) + per - 1) / per;
  a.renorm = renormalize != 0;
  a.scaling = scaling;
  a.ids = topk_ids;
  a.weights = topk_weights;
  HIP_TRY(launch_route(a, static_cast<hipStream_t>(stream)), "route launch");
  return CHORD_OK;
}

size_t chord_f8_packed_bytes(int role, int E, int N, int K) {
  clear_last_error();
  return check_shape(role, E, N, K) == CHORD_OK ? f8_packed_bytes(E, N, K) : 0;
}

chord_status chord_f8_pack(int role, const chord_f8* codes, const float* scales, int E, int N,
                           int K, int block, void* dst, size_t dst_bytes,
                           chord_f8_weight* handle, void* stream) {
  clear_last_error();
  if (!codes || !scales || !dst || !handle)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (block != kF8Block)
    return fail(CHORD_ERR_UNSUPPORTED, "block size %d (only 128 is supported)", block);
  CHORD_CHECK(check_shape(role, E, N, K));
  if (!aligned(dst, 16)) return fail(CHORD_ERR_INVALID_ARGUMENT, "dst must be 16-byte aligned");
  const size_t need = f8_packed_bytes(E, N, K);
  if (dst_bytes < need)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "dst has %zu bytes, %zu needed", dst_bytes, need);
  CHORD_CHECK(check_device(nullptr));
  HIP_TRY(launch_f8_pack(codes, scales, E, N, K, role == CHORD_ROLE_GATE_UP ? 1 : 0,
                         static_cast<uint8_t*>(dst), static_cast<hipStream_t>(stream)),
          "8-bit pack launch");
  *handle = chord_f8_weight{};
  handle->magic = CHORD_F8_WEIGHT_MAGIC;
  handle->version = CHORD_F8_WEIGHT_VERSION;
  handle->role = role;
  handle->num_experts = E;
  handle->n = N;
  handle->k = K;
  handle->block = kF8Block;
  handle->data = dst;
  handle->bytes = need;
  return CHORD_OK;
}

chord_status chord_f8_quantize(const chord_bf16* x, int64_t T, int K, int64_t ld, chord_f8* codes,
                               float* scales, void* stream) {
  clear_last_error();
  if (T < 0 || K < 1) return fail(CHORD_ERR_INVALID_ARGUMENT, "T=%lld K=%d", (long long)T, K);
  if (ld < K)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "row stride %lld below K=%d", (long long)ld, K);
  if (T == 0) return CHORD_OK;
  if (T > (int64_t)1 << 40 || K > 1 << 30)
    return fail(CHORD_ERR_UNSUPPORTED, "T=%lld K=%d", (long long)T, K);
  if (!x || !codes || !scales) return fail(CHORD_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (!aligned(codes, 16)) return fail(CHORD_ERR_INVALID_ARGUMENT, "codes must be 16-byte aligned");
  CHORD_CHECK(check_device(nullptr));
  F8QuantArgs q{};
  q.x = x;
  q.T = T;
  q.ld = ld;
  q.K = K;
  q.q = codes;
  q.s = scales;
  HIP_TRY(launch_f8_quantize(q, static_cast<hipStream_t>(stream)), "quantize launch");
  return CHORD_OK;
}

chord_status chord_f8_gemm(const chord_f8* codes, const float* scales, int64_t M,
                           const chord_f8_weight* w, chord_bf16* out, int64_t ld, void* workspace,
                           size_t ws_bytes, void* stream) {
  clear_last_error();
  CHORD_CHECK(check_f8_weight(w, "w", CHORD_ROLE_PLAIN));
  if (M < 0) return fail(CHORD_ERR_INVALID_ARGUMENT, "M=%lld", (long long)M);
  if (ld < w->n)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "row stride %lld below N=%d", (long long)ld, w->n);
  if (M == 0) return CHORD_OK;
  if (M >= (int64_t)1 << 31) return fail(CHORD_ERR_UNSUPPORTED, "M=%lld", (long long)M);
  if (!codes || !scales || !out) return fail(CHORD_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (!aligned(codes, 16)) return fail(CHORD_ERR_INVALID_ARGUMENT, "codes must be 16-byte aligned");
  const F8GemmPlan plan = f8_gemm_plan(M, w->n, w->k);
  const size_t need = f8_gemm_ws(plan, M, w->n);
  if (need > 0 && (!workspace || ws_bytes < need))
    return fail(CHORD_ERR_WORKSPACE, "workspace %zu bytes, %zu needed", ws_bytes, need);
  if (need > 0 && !aligned(workspace, 16))
    return fail(CHORD_ERR_WORKSPACE, "the workspace must be 16-byte aligned");
  int cus = 0;
  CHORD_CHECK(check_device(&cus));
  F8GemmArgs g = weight_args(w, kF8Plain, cus);
  g.tile_rows = plan.tile_rows;
  g.parts = plan.parts;
  g.partials = static_cast<float*>(workspace);
  g.aq = codes;
  g.as = scales;
  g.a_rows = M;
  g.out = out;
  g.ld = ld;
  hipStream_t st = static_cast<hipStream_t>(stream);
  HIP_TRY(plan.stream ? launch_f8_gemm(g, st) : launch_f8_tile(g, false, st), "8-bit GEMM launch");
  if (plan.stream) {
    set_last_plan("f8 gemm: streaming");
  } else {
    char text[64];
    snprintf(text, sizeof(text), "f8 gemm: tiles of %d rows, K in %d", plan.tile_rows, plan.parts);
    set_last_plan(text);
  }
  return CHORD_OK;
}

size_t chord_f8_gemm_workspace_bytes(int64_t M, int N, int K) {
  clear_last_error();
  if (M < 0 || check_shape(CHORD_ROLE_PLAIN, 1, N, K) != CHORD_OK) return 0;
  return f8_gemm_ws(f8_gemm_plan(M, N, K), M, N);
}

size_t chord_f8_moe_workspace_bytes(int T, int k, int E_l, int H, int I) {
  clear_last_error();
  if (check_moe_sizes(T, k, E_l, H, I) != CHORD_OK) return 0;
  return f8_ws(T, k, E_l, H, I).total;
}

chord_status chord_f8_moe(const chord_bf16* x, int T, int H, int I, const chord_f8_weight* w13,
                          const chord_f8_weight* w2, const int32_t* topk_ids,
                          const float* topk_weights, int k, int expert_begin,
                          int num_global_experts, chord_bf16* out, void* workspace,
                          size_t ws_bytes, void* stream) {
  clear_last_error();
  CHORD_CHECK(check_f8_weight(w13, "w13", CHORD_ROLE_GATE_UP));
  CHORD_CHECK(check_f8_weight(w2, "w2", CHORD_ROLE_DOWN));
  const int E_l = w13->num_experts;
  CHORD_CHECK(check_moe_sizes(T, k, E_l, H, I));
  if (w13->n != 2 * I || w13->k != H)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "w13 is [%d,%d], expected [2I=%d, H=%d]", w13->n, w13->k,
                2 * I, H);
  if (w2->n != H || w2->k != I)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "w2 is [%d,%d], expected [H=%d, I=%d]", w2->n, w2->k, H, I);
  if (w2->num_experts != E_l)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "w13 has %d experts, w2 %d", E_l, w2->num_experts);
  if (T == 0) return CHORD_OK;
  if (!x || !topk_ids || !topk_weights || !out)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (!aligned(x, 16) || !aligned(out, 16))
    return fail(CHORD_ERR_INVALID_ARGUMENT, "x and out must be 16-byte aligned");
  const F8Ws ws = f8_ws(T, k, E_l, H, I);
  if (!workspace || ws_bytes < ws.total)
    return fail(CHORD_ERR_WORKSPACE, "workspace %zu bytes, %zu needed", ws_bytes, ws.total);
  if (!aligned(workspace, 256))
    return fail(CHORD_ERR_WORKSPACE, "the workspace must be 256-byte aligned");
  int cus = 0;
  CHORD_CHECK(check_device(&cus));
  hipStream_t st = static_cast<hipStream_t>(stream);
  uint8_t* p = static_cast<uint8_t*>(workspace);
  if (f8_small_fits(T, k, H, I)) {
    const F8GemmArgs w13a = weight_args(w13, kF8GateUp, cus), w2a = weight_args(w2, kF8Down, cus);
    F8SmallArgs s{};
    s.x = x;
    s.T = T;
    s.k = k;
    s.H = H;
    s.I = I;
    s.topk_ids = topk_ids;
    s.topk_weights = topk_weights;
    s.expert_begin = expert_begin;
    s.num_experts = E_l;
    s.w13 = w13a.wq;
    s.s13 = w13a.ws;
    s.w2 = w2a.wq;
    s.s2 = w2a.ws;
    s.h = reinterpret_cast<float*>(p + ws.h);
    s.out = out;
    s.num_cus = cus;
    HIP_TRY(launch_f8_small(s, st), "small layer launch");
    set_last_plan("f8 moe: a handful of tokens, two launches");
    return CHORD_OK;
  }
  int32_t* sorted = reinterpret_cast<int32_t*>(p + ws.sorted);
  int32_t* experts = reinterpret_cast<int32_t*>(p + ws.experts);
  int32_t* ntpp = reinterpret_cast<int32_t*>(p + ws.ntpp);

  F8QuantArgs q{};
  q.x = x;
  q.T = T;
  q.ld = H;
  q.K = H;
  q.q = p + ws.xq;
  q.s = reinterpret_cast<float*>(p + ws.xs);
  HIP_TRY(launch_f8_quantize(q, st), "quantize launch");
  const F8MoePlan plan = f8_moe_plan(T, k, num_global_experts, E_l, I, cus);
  CHORD_CHECK(chord_moe_align(topk_ids, T, k, expert_begin, E_l, plan.block_m, sorted, experts, ntpp,
                              ws.max_padded, p + ws.align,
                              chord_moe_align_workspace_bytes(T, k, E_l, plan.block_m), 0, st));
  const TileDesc* tiles = reinterpret_cast<const TileDesc*>(p + ws.tiles);
  const DevStatus* status = reinterpret_cast<const DevStatus*>(p + ws.status);
  if (!plan.small) {
    TileBuildArgs tb{};
    tb.layout = kIndexed;
    tb.num_experts = E_l;
    tb.tile_tokens = plan.block_m;
    tb.big_tokens = kF8MoeTileRows;
    tb.max_tiles_b = ws.max_tiles;
    tb.max_ksplit = 2;
    tb.expert_ids = experts;
    tb.ntpp = ntpp;
    tb.block_m = plan.block_m;
    tb.max_padded = ws.max_padded;
    tb.tiles_b = reinterpret_cast<TileDesc*>(p + ws.tiles);
    tb.status = reinterpret_cast<DevStatus*>(p + ws.status);
    HIP_TRY(launch_build_tiles(tb, st), "tile builder launch");
  }
  auto rows_of = [&](F8GemmArgs& g) {
    g.sorted_ids = sorted;
    g.expert_ids = experts;
    g.ntpp = ntpp;
    g.block_m = plan.block_m;
    g.max_padded = ws.max_padded;
    g.topk = k;
    g.n_flat = (int64_t)T * k;
    g.est_blocks = plan.blocks;
    g.tiles = tiles;
    g.status = status;
  };
  uint8_t* hq = p + ws.hq;
  float* hs = reinterpret_cast<float*>(p + ws.hs);
  F8GemmArgs g = weight_args(w13, kF8GateUp, cus);
  rows_of(g);
  g.aq = q.q;
  g.as = q.s;
  g.a_rows = T;
  g.ld = I;
  if (plan.stream_gate_up) {
    g.out = p + ws.h;
    HIP_TRY(launch_f8_gemm(g, st), "gate_up launch");
    F8QuantArgs qh{};
    qh.x = p + ws.h;
    qh.is_f32 = 1;
    qh.T = ws.max_padded;
    qh.rows = ntpp;
    qh.ld = I;
    qh.K = I;
    qh.q = hq;
    qh.s = hs;
    HIP_TRY(launch_f8_quantize(qh, st), "quantize launch");
  } else {
    g.out = hq;
    g.hs = hs;
    g.exact = plan.exact;
    HIP_TRY(launch_f8_tile(g, plan.small, st), "gate_up launch");
  }

  F8GemmArgs d = weight_args(w2, kF8Down, cus);
  rows_of(d);
  d.aq = hq;
  d.as = hs;
  d.a_rows = ws.max_padded;
  d.out = p + ws.y;
  d.yu = p + ws.yu;
  d.ld = H;
  HIP_TRY(plan.small && d.n_chunks <= 2 ? launch_f8_short_down(d, st) : launch_f8_tile(d, plan.small, st),
          "down launch");

  F8CombineArgs c{};
  c.y = reinterpret_cast<const uint16_t*>(p + ws.y);
  c.yu = p + ws.yu;
  c.topk_ids = topk_ids;
  c.topk_weights = topk_weights;
  c.T = T;
  c.k = k;
  c.H = H;
  c.expert_begin = expert_begin;
  c.num_experts = E_l;
  c.out = reinterpret_cast<uint16_t*>(out);
  HIP_TRY(launch_f8_combine(c, st), "combine launch");
  set_last_plan(plan.text);
  return CHORD_OK;
}

}  // extern "C"
