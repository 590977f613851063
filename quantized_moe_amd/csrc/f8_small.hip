// The W8A8 layer for a handful of tokens (T * k <= 32) in two launches.
// With one token the weights of its experts take about ten microseconds, and each
// further launch in front of or between the two products four to five, so here
// every workgroup groups the slots by expert itself (one wave, one ballot per
// expert), quantises the rows of x (or h) into LDS, which few rows make cheap,
// and the second launch adds up the slots of its outputs.  (One token, eight
// experts of 512 x 7168 and 7168 x 256 weights: 34 us in six launches; 25.5
// with each wave quantising what it multiplies, 16 columns at a time whether
// there are tokens for them or not; 18.5 so.)
//
// x and h are quantised as in the other forms, from the same 128 columns, and the
// slots added in the same ascending order.  y never leaves the workgroup and stays
// fp32 (fp16 with a shared exponent in the forms that write it to memory), and
// gate_up is always summed in fp32.
#include "f8_common.h"

namespace chord {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kTok = 16;  // rows per tile

__device__ __forceinline__ i32x8_t operand(u32x4_t a, u32x4_t b) {
  return i32x8_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// Quantises rows [rows, K] (`use`: which of them) into LDS, 16 lanes a group.
template <typename T, typename U>
__device__ __forceinline__ void quantize_rows(const T* src, int rows, int K, uint8_t* codes, float* scales,
                                              U&& use) {
  const int nc = K / kF8Block, part = threadIdx.x & 15;
  for (int g = threadIdx.x >> 4; g < rows * nc; g += kThreads / 16) {
    if (!use(g / nc)) continue;
    float v[8];
    const T* p = src + (int64_t)g * kF8Block + part * 8;
    if constexpr (sizeof(T) == 4) {
      const f32x4_t lo = reinterpret_cast<const f32x4_t*>(p)[0], hi = reinterpret_cast<const f32x4_t*>(p)[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
    } else {
      const u32x4_t u = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_to_f32(u[i] & 0xFFFFu);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    const F8Group q = f8_group(row_max16(m));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = q.inv != 0.f ? f8_value(q, v[i]) : 0.f;
    *reinterpret_cast<uint2*>(codes + g * kF8Block + part * 8) =
        make_uint2(f8_pack4(v[0], v[1], v[2], v[3]), f8_pack4(v[4], v[5], v[6], v[7]));
    if (part == 0) scales[g] = q.scale;
  }
}

// The local slots grouped by expert, in tiles of at most 16.
struct Routes {
  int list[kFusedMaxSlots];
  int expert[kFusedMaxSlots], start[kFusedMaxSlots], rows[kFusedMaxSlots];  // per tile
  int local[kFusedMaxSlots];  // per slot
  int tiles;
};
__device__ __forceinline__ void build_routes(Routes& r, const F8SmallArgs& a) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x, n = a.T * a.k;
    const int id = lane < n ? a.topk_ids[lane] : INT32_MIN;
    // (unsigned difference: no id, however far off, wraps into the range)
    const int e = (int)((uint32_t)id - (uint32_t)a.expert_begin);
    const bool loc = lane < n && id >= a.expert_begin && (uint32_t)e < (uint32_t)a.num_experts;
    r.local[lane] = loc ? 1 : 0;
    uint64_t left = __builtin_amdgcn_ballot_w64(loc);
    int rows = 0, tiles = 0;
    while (left != 0) {
      const int ex = __builtin_amdgcn_readlane(e, __builtin_ctzll(left));
      const uint64_t same = __builtin_amdgcn_ballot_w64(loc && e == ex);
      left &= ~same;
      const int c = __builtin_popcountll(same), nt = (c + kTok - 1) / kTok;
      if ((same >> lane) & 1) r.list[rows + __builtin_popcountll(same & ((1ull << lane) - 1))] = lane;
      if (lane < nt) {
        r.expert[tiles + lane] = ex;
        r.start[tiles + lane] = rows + kTok * lane;
        r.rows[tiles + lane] = min(kTok, c - kTok * lane);
      }
      rows += c;
      tiles += nt;
    }
    if (lane == 0) r.tiles = tiles;
  }
}

__device__ __forceinline__ void load_w(u32x4_t (&w)[2], const uint8_t* p) {
  w[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
  w[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p + 1024));
}

__device__ __forceinline__ i32x8_t read_codes(const uint8_t* p) {
  return operand(reinterpret_cast<const u32x4_t*>(p)[0], reinterpret_cast<const u32x4_t*>(p)[1]);
}

// h[slot] = silu(W1 x~) * (W3 x~).  A workgroup owns one interleaved weight tile
// (8 features) of one expert; its waves split K.
__global__ __launch_bounds__(kThreads) void small_gate_up(F8SmallArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];  // codes [T, H], scales [T, nc]
  __shared__ Routes rt;
  __shared__ f32x4_t red[kWaves][64];
  uint8_t* codes = smem;
  float* scales = reinterpret_cast<float*>(smem + a.T * a.H);
  build_routes(rt, a);
  quantize_rows(a.x, a.T, a.H, codes, scales, [](int) { return true; });
  __syncthreads();
  const int lane = threadIdx.x & 63, q = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nt = a.I / 8, nc = a.H / kF8Block, nb = 2 * a.I / kF8Block;
  const int c_lo = nc * wave / kWaves, c_hi = nc * (wave + 1) / kWaves;
  const int wstep = f8_slice_width(0, nt) * kF8BlockBytes;  // (2 I is a multiple of 256)
  // Chunks on their way.  Deeper than needed costs registers, so waves (T = 1: 8
  // experts of 7168 x 256, 4096 x 512 and 2048 x 768 with 4, 7, 8 and 10 chunks 18.8,
  // 18.4, 18.6, 29.7; 19.4, 19.2, 19.4, 30.3; 18.9, 19.1, 19.2, 24.9 us for the layer).
  constexpr int PF = 8;
  for (int item = blockIdx.x; item < rt.tiles * nt; item += gridDim.x) {
    const int ti = item / nt, t = item - ti * nt, e = rt.expert[ti];
    const bool live = col < rt.rows[ti];
    const int f = rt.list[rt.start[ti] + (live ? col : 0)];
    const uint8_t* wp = a.w13 + ((int64_t)e * nt * nc + f8_block(t, 0, nt, nc)) * kF8BlockBytes + lane * 16;
    const float* s0 = a.s13 + ((int64_t)e * nb + t / 16) * nc;
    const float* s1 = s0 + (int64_t)(nb / 2) * nc;
    const uint8_t* xp = codes + f / a.k * a.H + q * 32;
    const float* sp = scales + f / a.k * nc;
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    u32x4_t w[PF][2];
    if (c_lo < c_hi) {
#pragma unroll
      for (int p = 0; p < PF; ++p)
        if (c_lo + p < c_hi) load_w(w[p], wp + (int64_t)(c_lo + p) * wstep);
      for (int c0 = c_lo; c0 < c_hi; c0 += PF) {
#pragma unroll
        for (int p = 0; p < PF; ++p) {
          const int c = c0 + p;
          if (c >= c_hi) break;
          const f32x4_t r = f8_exact_product(operand(w[p][0], w[p][1]), read_codes(xp + c * kF8Block));
          if (c + PF < c_hi) load_w(w[p], wp + (int64_t)(c + PF) * wstep);
          const float f0 = sp[c] * s0[c], f1 = sp[c] * s1[c];
          acc[0] = __builtin_fmaf(r[0], f0, acc[0]);
          acc[1] = __builtin_fmaf(r[1], f1, acc[1]);
          acc[2] = __builtin_fmaf(r[2], f0, acc[2]);
          acc[3] = __builtin_fmaf(r[3], f1, acc[3]);
        }
      }
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
      f32x4_t v = red[0][lane];
#pragma unroll
      for (int u = 1; u < kWaves; ++u) v += red[u][lane];
      if (live)
        *reinterpret_cast<float2*>(a.h + (int64_t)f * a.I + t * 8 + 2 * q) =
            make_float2(silu_mul(v[0], v[1]), silu_mul(v[2], v[3]));
    }
    __syncthreads();
  }
}

// out[t] = bf16(sum over local slots of w * W2 h~).  A workgroup owns 16 outputs of
// every token; its waves take the tiles of the slots in turn, then add up.
__global__ __launch_bounds__(kThreads) void small_down(F8SmallArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];  // codes [T * k, I], scales [T * k, nc]
  __shared__ Routes rt;
  __shared__ float y[kFusedMaxSlots][17];
  uint8_t* codes = smem;
  float* scales = reinterpret_cast<float*>(smem + a.T * a.k * a.I);
  build_routes(rt, a);
  __syncthreads();
  quantize_rows(a.h, a.T * a.k, a.I, codes, scales, [&](int f) { return rt.local[f] != 0; });
  __syncthreads();
  const int lane = threadIdx.x & 63, q = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nt = a.H / 16, nc = a.I / kF8Block, nb = a.H / kF8Block;
  constexpr int PF = 4;
  for (int t = blockIdx.x; t < nt; t += gridDim.x) {
    const int wstep = f8_slice_width(t, nt) * kF8BlockBytes;
    for (int ti = wave; ti < rt.tiles; ti += kWaves) {
      const int e = __builtin_amdgcn_readfirstlane(rt.expert[ti]);
      const bool live = col < rt.rows[ti];
      const int f = rt.list[rt.start[ti] + (live ? col : 0)];
      const uint8_t* wp = a.w2 + ((int64_t)e * nt * nc + f8_block(t, 0, nt, nc)) * kF8BlockBytes + lane * 16;
      const float* s0 = a.s2 + ((int64_t)e * nb + t / 8) * nc;
      const uint8_t* hp = codes + f * a.I + q * 32;
      const float* sp = scales + f * nc;
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
      u32x4_t w[PF][2];
#pragma unroll
      for (int p = 0; p < PF; ++p)
        if (p < nc) load_w(w[p], wp + (int64_t)p * wstep);
      for (int c0 = 0; c0 < nc; c0 += PF) {
#pragma unroll
        for (int p = 0; p < PF; ++p) {
          const int c = c0 + p;
          if (c >= nc) break;
          const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
          const f32x4_t r = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              operand(w[p][0], w[p][1]), read_codes(hp + c * kF8Block), zero, 0, 0, 0, 0, 0, 0);
          if (c + PF < nc) load_w(w[p], wp + (int64_t)(c + PF) * wstep);
          const float fs = sp[c] * s0[c];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(r[i], fs, acc[i]);
        }
      }
      if (live) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[f][4 * q + i] = acc[i];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * 16; i += kThreads) {
      const int tok = i >> 4, n = i & 15;
      float s = 0.f;
      for (int j = 0; j < a.k; ++j) {
        const int f = tok * a.k + j;
        if (rt.local[f]) s = __builtin_fmaf(a.topk_weights[f], y[f][n], s);
      }
      a.out[(int64_t)tok * a.H + t * 16 + n] = to_bf16(s);
    }
    __syncthreads();
  }
}

}  // namespace

// Rows in LDS take this many bytes at most (with the tables, two workgroups a CU).
constexpr int64_t kRowBytes = 68 << 10;
int64_t row_bytes(int64_t rows, int K) { return rows * (K + K / kF8Block * 4); }

// Every workgroup quantises all rows, so with more slots the other forms win, the
// sooner the smaller the weights (here / there, in us): 24 slots, 64 experts of 7168
// x 256 37 / 50, 32 slots 45 / 52, 56 slots 64 / 68; 32 slots, 48 experts of 7168 x
// 2048 206 / 212, 16 of 1024 x 512 22 / 26, 64 of 2048 x 768 49 / 42; 64 slots 26 /
// 27 and 69 / 60, 16 of 1024 x 2048 43 / 43.
constexpr int kSmallSlots = 32;

bool f8_small_fits(int T, int k, int H, int I) {
  return T <= kFusedMaxTokens && (int64_t)T * k <= kSmallSlots && row_bytes(T, H) <= kRowBytes &&
         row_bytes((int64_t)T * k, I) <= kRowBytes;
}

hipError_t launch_f8_small(const F8SmallArgs& a, hipStream_t stream) {
  const int64_t tiles = (int64_t)a.T * a.k * (a.I / 8), most = (int64_t)a.num_cus * 2;
  auto run = [&](auto kernel, int64_t blocks, int64_t lds) {
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)kRowBytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), (size_t)lds,
                       stream, a);
    return hipGetLastError();
  };
  const hipError_t e = run(small_gate_up, tiles, row_bytes(a.T, a.H));
  if (e != hipSuccess) return e;
  return run(small_down, a.H / 16, row_bytes((int64_t)a.T * a.k, a.I));
}

}  // namespace chord
