// Host side of the operators around a layer: norms between blocks, the dense 16-bit
// product and the router's balance.  Argument checks (before any HIP call),
// workspace layout and launches.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "host.h"

using namespace chord;

namespace {

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool known(int dtype) {
  return dtype == CHORD_DTYPE_F32 || dtype == CHORD_DTYPE_BF16 || dtype == CHORD_DTYPE_F16;
}

// ---- norms -------------------------------------------------------------------
constexpr int kNormMaxH = 32768;  // 1024 threads x 4 x 8 values

chord_status norm_part(const chord_norm_weight* w, const char* name, int dtype, NormPart* p) {
  *p = NormPart{};
  if (!w) return CHORD_OK;
  if (!w->weight) return fail(CHORD_ERR_INVALID_ARGUMENT, "%s has no weight", name);
  if (w->kind != CHORD_NORM_RMS && w->kind != CHORD_NORM_LAYER)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "%s kind %d", name, w->kind);
  if (w->dtype != dtype && w->dtype != CHORD_DTYPE_F32)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "%s dtype %d (dtype %d or fp32)", name, w->dtype, dtype);
  // (Squares below the smallest normal number vanish beside it.)
  if (!std::isnormal(w->eps) || w->eps < 0.f)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "%s eps %g must be a positive normal number", name, w->eps);
  if (!std::isfinite(w->offset)) return fail(CHORD_ERR_INVALID_ARGUMENT, "%s offset is not finite", name);
  *p = NormPart{w->weight, w->bias, w->dtype, w->kind, w->eps, w->offset};
  return CHORD_OK;
}

// ---- balance -----------------------------------------------------------------
constexpr int kBalanceMaxTokens = 1 << 25;
constexpr int kBalanceMaxK = 1024;
constexpr int kBalanceMaxSeq = 65535;  // (grid dimension)

struct BalancePlan {
  int parts, chunks;
  int64_t rows;
  size_t counts, total;
};

BalancePlan balance_plan(int T, int E, int k, int n_seq) {
  BalancePlan p{};
  const int64_t L = T / n_seq;
  const int64_t slots = L * k;
  p.parts = slots <= 16384 ? 0 : (int)std::min<int64_t>(16, (slots + 16383) / 16384);
  // Rows of a workgroup: one a wave, up to four where that fills the CUs, and more where
  // there would be over 1024 workgroups.  Short sequences in one, which then needs no second
  // launch: a wave goes through its rows one after the other, the longer each the more
  // experts it has, so up to 64 rows and 384 groups of 64 logits.  us a call (the launches
  // alone), one / two launches: 64 rows of 256 experts 14.5 (14.3) / 18.1 (9.6), of 384 17.0
  // (16.9) / 18.2 (10.5), of 1024 36.3 (36.3) / 18.4 (15.5); 16 of 1024 16.0 (15.7) / 18.3.
  p.rows = std::max<int64_t>({8, std::min<int64_t>(32, (T + 255) / 256), (T + 1023) / 1024});
  if (L <= 64 && L * ((E + 63) / 64) <= 384) p.rows = std::max<int64_t>(p.rows, 64);
  p.chunks = (int)std::max<int64_t>(1, (L + p.rows - 1) / p.rows);
  size_t off = 0;
  if (p.parts > 0) off += ((size_t)n_seq * p.parts * (E + 1) * 4 + 15) & ~(size_t)15;
  p.counts = off;
  if (p.chunks > 1) off += (size_t)n_seq * p.chunks * E * 4;
  p.total = off;
  return p;
}

chord_status check_balance_sizes(int T, int E, int k, int n_seq) {
  if (T < 0) return fail(CHORD_ERR_INVALID_ARGUMENT, "T=%d", T);
  if (E < 1 || E > kMaxExperts) return fail(CHORD_ERR_INVALID_ARGUMENT, "E=%d (1..%d)", E, kMaxExperts);
  if (k < 1 || k > kBalanceMaxK) return fail(CHORD_ERR_INVALID_ARGUMENT, "k=%d (1..%d)", k, kBalanceMaxK);
  if (n_seq < 1 || T % n_seq != 0)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "n_seq=%d must divide T=%d", n_seq, T);
  if (n_seq > kBalanceMaxSeq) return fail(CHORD_ERR_UNSUPPORTED, "n_seq=%d above %d", n_seq, kBalanceMaxSeq);
  if (T > kBalanceMaxTokens) return fail(CHORD_ERR_UNSUPPORTED, "T=%d above %d", T, kBalanceMaxTokens);
  if ((int64_t)T * k >= (int64_t)1 << 31) return fail(CHORD_ERR_UNSUPPORTED, "T*k=%lld", (long long)T * k);
  return CHORD_OK;
}

// ---- product -----------------------------------------------------------------
constexpr int64_t kLinearMaxRows = (int64_t)1 << 29;  // of x, and of W
constexpr int kLinearMaxK = 1 << 20;

chord_status check_linear_sizes(int64_t ldx, int64_t ldw, int64_t M, int N, int K, int gated) {
  if (M < 0 || N < 1 || K < 1)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "M=%lld N=%d K=%d", (long long)M, N, K);
  if (ldx < K || ldw < K)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "row strides %lld (x) and %lld (w) below K=%d", (long long)ldx,
                (long long)ldw, K);
  if (M >= kLinearMaxRows || (int64_t)N * (gated ? 2 : 1) >= kLinearMaxRows || K > kLinearMaxK)
    return fail(CHORD_ERR_UNSUPPORTED, "M=%lld N=%d K=%d", (long long)M, N, K);
  return CHORD_OK;
}

// Whether rows can be read in place: 16-byte pieces, and offsets inside a tile of up
// to 256 rows that stay below 2^31.
bool rows_in_place(const void* p, int64_t ld, int K) {
  return aligned(p, 16) && ld % 8 == 0 && K % 8 == 0 && ld <= (int64_t)1 << 21;
}

// How a product runs: the weight-streaming form with tiles of 16 to 64 tokens, or
// LDS tiles with K in parts that a second launch adds.
struct LinearPlan {
  bool stream;
  int tokens;        // stream
  int shape, parts;  // tiles
  bool copy_x, copy_w;
  int K;  // of the rows that are read
  size_t x, w, partials, total;  // workspace: copies, sums
};

// us: of a chunk of 64 along K, on a workgroup alone.
const struct {
  int rows, outs;
  double us;
} kLinearShapes[] = {{256, 256, 1.15}, {128, 256, 0.60}, {128, 128, 0.40}, {64, 128, 0.28}};

// The cheapest by estimate, in us on an MI355X with 256 workgroups a round (one a CU in
// every form).  Streaming: a launch 3.4; a step of its 8 waves is bound by the lines that
// a CU takes, (16 + tokens) x 128 bytes a wave, less alone than beside 255 others; or the
// weights' bytes at 6.5 TB/s.  Tiles: a launch and a round's start, chunks, up to 30 %
// slower on a full chip, and for parts another launch and their bytes.  Over 50 sizes
// with every form measured (M = 1, 16, 32, 64, 100, 128, 256, 512, 1024, 2048; N x K =
// 384 x 7168, 2112 x 7168, 4096 x 7168, 7168 x 2048, 1024 x 1024) what it picks takes 0.2 %
// more than the best on average.  Streaming with 16, 32, 64 tokens / best tiles, us: M=16
// N=4096 K=7168 13.0 13.3 14.1 / 16.9; M=32 N=2112 19.0 11.7 13.7 / 14.2; M=64 N=384 7.5 8.8
// 12.3 / 11.5, N=2112 32.7 25.4 19.5 / 15.3, N=4096 42.3 24.1 17.3 / 18.9; M=100 N=2112 43.9
// 33.0 29.2 / 17.7.  Tiles: M=512 N=4096 64x128 40.8, 128x128 in 2 41.2, 128x256 in 4 41.9,
// 256x256 in 4 43.0; M=2048 N=2112 128x256 77.2, 256x256 84.4; M=8192 N=384 256x256 130, in
// 4 parts 63, 128x256 80, 128x128 56, 64x128 66.  All of it with inputs that the caches
// hold: x of 8192 rows from HBM takes 77 with 128x128, where 256x256 in 4 parts takes 74 and
// 128x256 in 2 parts 71.
LinearPlan linear_plan(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t M, int N, int K, int gated) {
  constexpr int64_t kCus = 256;  // (of the model, so that the workspace depends on sizes alone)
  LinearPlan p{};
  p.copy_x = !rows_in_place(x, ldx, K);
  p.copy_w = !rows_in_place(w, ldw, K);
  p.K = (K + 7) / 8 * 8;
  p.parts = 1;
  const int64_t rows = (int64_t)N * (gated ? 2 : 1);
  const int chunks = (p.K + 63) / 64;
  double best = 1e300;
  auto full = [&](int64_t items) { return std::min(1.0, (double)items / kCus); };
  for (int tokens : {16, 32, 64}) {
    const int64_t items = (M + tokens - 1) / tokens * ((N + (gated ? 7 : 15)) / (gated ? 8 : 16));
    const double rounds = (double)((items + kCus - 1) / kCus), steps = (double)((chunks + 7) / 8);
    const double lines = rounds * steps * (16 + tokens) * 0.0073 * (1.0 + 0.6 * std::sqrt(full(items)));
    const double cost = 3.4 + 1.5 * (rounds - 1) +
                        std::max(rounds > 1 ? 1.25 * lines : lines, (double)rows * p.K * 2 / 6.5e6);
    if (cost < best) {
      best = cost;
      p.stream = true;
      p.tokens = tokens;
    }
  }
  for (int s = 0; s < 4; ++s) {
    const int64_t items = (M + kLinearShapes[s].rows - 1) / kLinearShapes[s].rows *
                          ((rows + kLinearShapes[s].outs - 1) / kLinearShapes[s].outs);
    for (int parts : {1, 2, 4, 8, 16}) {
      if (parts > 1 && (parts > chunks || items * parts > 2 * kCus)) break;
      double rounds = (double)((items * parts + kCus - 1) / kCus);
      const int64_t rest = items * parts % kCus;
      if (s == 0 && rest > 0 && 2 * rest <= kCus) rounds -= 0.4;  // (the last round in halves)
      double cost = 2.5 + rounds * (1.2 + (chunks + parts - 1) / parts * kLinearShapes[s].us *
                                              (1.0 + 0.3 * full(items * parts)));
      if (parts > 1) cost += 4.0 + parts * (double)M * rows * 8 / 3.8e6;
      if (cost < best) {
        best = cost;
        p.stream = false;
        p.shape = s;
        p.parts = parts;
      }
    }
  }
  auto take = [&](bool on, int64_t bytes) {
    const size_t o = p.total;
    if (on) p.total += ((size_t)bytes + 255) & ~(size_t)255;
    return o;
  };
  p.x = take(p.copy_x, M * p.K * 2);
  p.w = take(p.copy_w, rows * p.K * 2);
  p.partials = take(p.parts > 1, (int64_t)p.parts * M * ((N + 15) / 16 * 16) * (gated ? 2 : 1) * 4);
  return p;
}

}  // namespace

extern "C" {

chord_status chord_norm(const void* x, int64_t ldx, int dtype, int64_t T, int H,
                        const chord_norm_weight* post, const void* gate, int gate_dtype,
                        int64_t gate_row, int64_t gate_col, int gate_sigmoid, float scale,
                        const void* residual, int64_t ldr, void* sum, int64_t lds,
                        int stream_dtype, const chord_norm_weight* pre, void* out, int64_t ldo,
                        chord_f8* codes, float* scales, void* stream) {
  clear_last_error();
  NormArgs a{};
  if (!known(dtype)) return fail(CHORD_ERR_INVALID_ARGUMENT, "dtype %d", dtype);
  CHORD_CHECK(norm_part(post, "post", dtype, &a.post));
  CHORD_CHECK(norm_part(pre, "pre", dtype, &a.pre));
  if (stream_dtype != dtype && stream_dtype != CHORD_DTYPE_F32)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "stream_dtype %d (dtype %d or fp32)", stream_dtype, dtype);
  if (T < 0 || H < 1) return fail(CHORD_ERR_INVALID_ARGUMENT, "T=%lld H=%d", (long long)T, H);
  if (H > kNormMaxH) return fail(CHORD_ERR_UNSUPPORTED, "H=%d above %d", H, kNormMaxH);
  if (T >= (int64_t)1 << 31) return fail(CHORD_ERR_UNSUPPORTED, "T=%lld", (long long)T);
  if (!std::isfinite(scale)) return fail(CHORD_ERR_INVALID_ARGUMENT, "scale is not finite");
  if (T == 0) return CHORD_OK;
  if (!sum && !out && !codes) return fail(CHORD_ERR_INVALID_ARGUMENT, "nothing to write");
  if ((out || codes) && !pre)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "out and codes are the norm's, and pre is NULL");
  if (pre && !out && !codes) return fail(CHORD_ERR_INVALID_ARGUMENT, "pre without out or codes");
  if (!codes != !scales) return fail(CHORD_ERR_INVALID_ARGUMENT, "codes and scales come together");
  if (ldx < H || (residual && ldr < H) || (sum && lds < H) || (out && ldo < H))
    return fail(CHORD_ERR_INVALID_ARGUMENT, "a row stride is below H=%d", H);
  if (gate) {
    if (gate_dtype != dtype && gate_dtype != CHORD_DTYPE_F32)
      return fail(CHORD_ERR_INVALID_ARGUMENT, "gate_dtype %d (dtype %d or fp32)", gate_dtype, dtype);
    if ((gate_col != 0 && gate_col != 1) || gate_row < 0)
      return fail(CHORD_ERR_INVALID_ARGUMENT, "gate strides %lld, %lld", (long long)gate_row, (long long)gate_col);
  }
  if (!x) return fail(CHORD_ERR_INVALID_ARGUMENT, "null pointer argument");
  if (codes && !aligned(codes, 16)) return fail(CHORD_ERR_INVALID_ARGUMENT, "codes must be 16-byte aligned");
  int cus = 0;
  CHORD_CHECK(check_device(&cus));
  a.num_cus = cus;
  a.x = x;
  a.ldx = ldx;
  a.dtype = dtype;
  a.T = T;
  a.H = H;
  a.gate = gate;
  a.gate_dtype = gate_dtype;
  a.gate_row = gate_row;
  a.gate_col = gate_col;
  a.gate_sigmoid = gate_sigmoid != 0;
  a.scale = scale;
  a.residual = residual;
  a.ldr = ldr;
  a.sum = sum;
  a.lds = lds;
  a.stream_dtype = stream_dtype;
  a.out = out;
  a.ldo = ldo;
  a.codes = codes;
  a.code_scales = scales;
  HIP_TRY(launch_norm(a, static_cast<hipStream_t>(stream)), "norm launch");
  return CHORD_OK;
}

size_t chord_moe_balance_workspace_bytes(int T, int E, int k, int n_seq) {
  clear_last_error();
  if (check_balance_sizes(T, E, k, n_seq) != CHORD_OK) return 0;
  return balance_plan(T, E, k, n_seq).total;
}

chord_status chord_moe_balance(const void* logits, int dtype, int64_t ld, int T, int E,
                               const float* bias, const int32_t* topk_ids, int k, int scoring,
                               int n_seq, int32_t* counts, int32_t* tokens, float* probs,
                               float* loss, const float* grad_loss, float* grad_logits,
                               void* workspace, size_t ws_bytes, void* stream) {
  clear_last_error();
  if (!known(dtype)) return fail(CHORD_ERR_INVALID_ARGUMENT, "dtype %d", dtype);
  if (scoring != CHORD_SCORE_SOFTMAX && scoring != CHORD_SCORE_SIGMOID)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "scoring %d", scoring);
  CHORD_CHECK(check_balance_sizes(T, E, k, n_seq));
  if (ld < E) return fail(CHORD_ERR_INVALID_ARGUMENT, "row stride %lld below E=%d", (long long)ld, E);
  if (!counts || !tokens || !probs || !loss || (T > 0 && (!logits || !topk_ids)))
    return fail(CHORD_ERR_INVALID_ARGUMENT, "null pointer argument");
  const BalancePlan plan = balance_plan(T, E, k, n_seq);
  if (plan.total > 0 && (!workspace || ws_bytes < plan.total))
    return fail(CHORD_ERR_WORKSPACE, "workspace %zu bytes, %zu needed", ws_bytes, plan.total);
  if (plan.total > 0 && !aligned(workspace, 16))
    return fail(CHORD_ERR_WORKSPACE, "the workspace must be 16-byte aligned");
  CHORD_CHECK(check_device(nullptr));
  BalanceArgs a{};
  a.logits = logits;
  a.dtype = dtype;
  a.ld = ld;
  a.L = T / n_seq;
  a.E = E;
  a.k = k;
  a.n_seq = n_seq;
  a.bias = bias;
  a.sigmoid = scoring == CHORD_SCORE_SIGMOID;
  a.ids = topk_ids;
  a.counts = counts;
  a.tokens = tokens;
  a.probs = probs;
  a.loss = loss;
  a.grad_loss = grad_loss;
  a.grad = grad_logits;
  a.parts = plan.parts;
  a.chunks = plan.chunks;
  a.rows = plan.rows;
  a.part_counts = reinterpret_cast<int32_t*>(workspace);
  a.part_probs = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.counts);
  HIP_TRY(launch_balance(a, static_cast<hipStream_t>(stream)), "balance launch");
  return CHORD_OK;
}

size_t chord_linear_workspace_bytes(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t M,
                                    int N, int K, int gated) {
  clear_last_error();
  if (check_linear_sizes(ldx, ldw, M, N, K, gated) != CHORD_OK || M == 0) return 0;
  return linear_plan(x, ldx, w, ldw, M, N, K, gated).total;
}

chord_status chord_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, int dtype,
                          int64_t M, int N, int K, const void* bias, int bias_dtype, int act,
                          int gated, float scale, const void* residual, int64_t ldr, void* out,
                          int64_t ldo, int out_dtype, void* workspace, size_t ws_bytes,
                          void* stream) {
  clear_last_error();
  if (!known(dtype)) return fail(CHORD_ERR_INVALID_ARGUMENT, "dtype %d", dtype);
  if (dtype == CHORD_DTYPE_F32) return fail(CHORD_ERR_UNSUPPORTED, "x and w must be bf16 or fp16");
  if (out_dtype != dtype && out_dtype != CHORD_DTYPE_F32)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "out_dtype %d (dtype %d or fp32)", out_dtype, dtype);
  if (bias && bias_dtype != dtype && bias_dtype != CHORD_DTYPE_F32)
    return fail(CHORD_ERR_INVALID_ARGUMENT, "bias_dtype %d (dtype %d or fp32)", bias_dtype, dtype);
  if (act < CHORD_ACT_NONE || act > CHORD_ACT_GELU_TANH) return fail(CHORD_ERR_INVALID_ARGUMENT, "act %d", act);
  if (!std::isfinite(scale)) return fail(CHORD_ERR_INVALID_ARGUMENT, "scale is not finite");
  CHORD_CHECK(check_linear_sizes(ldx, ldw, M, N, K, gated));
  if (ldo < N || (residual && ldr < N))
    return fail(CHORD_ERR_INVALID_ARGUMENT, "a row stride is below N=%d", N);
  if (M == 0) return CHORD_OK;
  if (!x || !w || !out) return fail(CHORD_ERR_INVALID_ARGUMENT, "null pointer argument");
  const LinearPlan plan = linear_plan(x, ldx, w, ldw, M, N, K, gated);
  if (plan.total > 0 && (!workspace || ws_bytes < plan.total))
    return fail(CHORD_ERR_WORKSPACE, "workspace %zu bytes, %zu needed", ws_bytes, plan.total);
  if (plan.total > 0 && !aligned(workspace, 256))
    return fail(CHORD_ERR_WORKSPACE, "the workspace must be 256-byte aligned");
  int cus = 0;
  CHORD_CHECK(check_device(&cus));
  hipStream_t st = static_cast<hipStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  LinearArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.w = static_cast<const uint16_t*>(w);
  a.ldw = ldw;
  a.M = M;
  a.N = N;
  a.K = K;
  a.f16 = dtype == CHORD_DTYPE_F16;
  a.gated = gated != 0;
  a.act = act;
  a.bias = bias;
  a.bias_f32 = bias_dtype == CHORD_DTYPE_F32;
  a.scale = scale;
  a.residual = residual;
  a.ldr = ldr;
  a.out = out;
  a.ldo = ldo;
  a.out_f32 = out_dtype == CHORD_DTYPE_F32;
  a.num_cus = cus;
  a.parts = plan.parts;
  a.partials = reinterpret_cast<float*>(ws + plan.partials);
  const int out_size = a.out_f32 ? 4 : 2;
  if (aligned(bias, a.bias_f32 ? 16 : 8)) a.wide |= kLinWideBias;
  if (aligned(residual, 4 * out_size) && ldr % 4 == 0) a.wide |= kLinWideResidual;
  if (aligned(out, 4 * out_size) && ldo % 4 == 0) a.wide |= kLinWideOut;
  auto pieces = [&](const void* p, int64_t ld) { return aligned(p, 16) && ld * out_size % 16 == 0; };
  a.direct = N % 8 == 0 && act != CHORD_ACT_GELU && pieces(out, ldo) && (!residual || pieces(residual, ldr));
  if (plan.copy_x) {
    uint16_t* to = reinterpret_cast<uint16_t*>(ws + plan.x);
    HIP_TRY(launch_copy_rows(a.x, ldx, M, K, plan.K, to, st), "copy launch");
    a.x = to;
    a.ldx = plan.K;
  }
  if (plan.copy_w) {
    uint16_t* to = reinterpret_cast<uint16_t*>(ws + plan.w);
    HIP_TRY(launch_copy_rows(a.w, ldw, (int64_t)N * (a.gated ? 2 : 1), K, plan.K, to, st), "copy launch");
    a.w = to;
    a.ldw = plan.K;
  }
  a.K = plan.K;
  HIP_TRY(plan.stream ? launch_linear_stream(a, plan.tokens, st) : launch_linear_tile(a, plan.shape, st), "product launch");
  if (plan.parts > 1) HIP_TRY(launch_linear_join(a, st), "product sum launch");
  char text[64];
  if (plan.stream) {
    snprintf(text, sizeof(text), "linear: streaming, %d tokens", plan.tokens);
  } else {
    snprintf(text, sizeof(text), "linear: tiles of %d x %d, K in %d", kLinearShapes[plan.shape].rows,
             kLinearShapes[plan.shape].outs, plan.parts);
  }
  set_last_plan(text);
  return CHORD_OK;
}

}  // extern "C"
