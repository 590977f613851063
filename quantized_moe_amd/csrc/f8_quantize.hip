// Activations to e4m3 codes with one fp32 scale for each 128 columns of a row,
// and the packing of 8-bit weights.
//
// Quantising is bound by memory: 2 (or 4) bytes read and 1 written a value.  A
// row of 16 lanes holds one group, 8 values a lane, so the group's maximum is
// four register moves away and no value is read twice: 8192 x 7168 in 34 us, 5.2
// TB/s, the rate of a large copy.
#include "f8_common.h"

namespace chord {
namespace {

constexpr int kThreads = 256;
constexpr int kGroupsPerPass = kThreads / 16;

// Values j .. j+7 of a row as fp32, zeros from K on.  Wide: 16-byte aligned
// rows with K % 8 == 0, so the 8 values are all there or none is.  (fp32 rows are a
// layer's h, which are wide.)
template <bool F32, bool WIDE>
__device__ __forceinline__ void load8(const void* x, int64_t row, int j, int K, float (&v)[8]) {
  static_assert(WIDE || !F32);
  if (F32) {
    const float* p = static_cast<const float*>(x) + row;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (j < K) {
      a = *reinterpret_cast<const float4*>(p + j);
      b = *reinterpret_cast<const float4*>(p + j + 4);
    }
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    return;
  }
  const uint16_t* p = static_cast<const uint16_t*>(x) + row;
  if (WIDE) {
    uint4 a = make_uint4(0u, 0u, 0u, 0u);
    if (j < K) a = *reinterpret_cast<const uint4*>(p + j);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = j + i < K ? bf16_to_f32(p[j + i]) : 0.f;
  }
}

template <bool F32, bool WIDE>
__global__ __launch_bounds__(kThreads) void quantize_kernel(F8QuantArgs a) {
  const int chunks = (a.K + kF8Block - 1) / kF8Block;
  int64_t T = a.T;
  if (a.rows != nullptr) T = min(T, max((int64_t)0, (int64_t)*a.rows));
  const int64_t groups = T * chunks;
  const int part = threadIdx.x & 15;
  for (int64_t g = (int64_t)blockIdx.x * kGroupsPerPass + (threadIdx.x >> 4); g < groups;
       g += (int64_t)gridDim.x * kGroupsPerPass) {
    const int64_t t = g / chunks;
    const int c = (int)(g - t * chunks);
    float v[8];
    load8<F32, WIDE>(a.x, t * a.ld, c * kF8Block + part * 8, a.K, v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    const F8Group q = f8_group(row_max16(m));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = q.inv != 0.f ? f8_value(q, v[i]) : 0.f;
    uint2 o;
    o.x = f8_pack4(v[0], v[1], v[2], v[3]);
    o.y = f8_pack4(v[4], v[5], v[6], v[7]);
    *reinterpret_cast<uint2*>(a.q + g * kF8Block + part * 8) = o;
    if (part == 0) a.s[g] = q.scale;
  }
}

// One thread per 16 bytes of the packed codes.
__global__ __launch_bounds__(kThreads) void pack_codes(const uint8_t* __restrict__ src, int E, int N,
                                                       int K, int gate_up, uint8_t* __restrict__ dst) {
  const int64_t tiles = f8_tiles(N), chunks = f8_chunks(K);
  const int64_t n = E * tiles * chunks * (kF8BlockBytes / 16);
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kThreads) {
    const int lane = (int)(i & 63), half = (int)(i >> 6) & 1;
    const int64_t blk = i >> 7, e = blk / (tiles * chunks);
    const int in = (int)(blk - e * tiles * chunks);  // block inside the expert
    const int slice = in / (int)(kF8SliceTiles * chunks);
    const int width = f8_slice_width(slice * kF8SliceTiles, (int)tiles);
    const int rest = in - slice * (int)(kF8SliceTiles * chunks);
    const int c = rest / width, t = slice * kF8SliceTiles + rest % width;
    const int r = lane & 15;
    int row = t * kTileRows + r;
    if (gate_up) row = (r & 1) * (N / 2) + 8 * t + 2 * (r >> 2) + ((r >> 1) & 1);
    const int k = c * kF8Block + (lane >> 4) * 32 + half * 16;
    const uint8_t* p = src + (e * N + row) * (int64_t)K + k;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (row < N) {
      if (k + 16 <= K && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        v = *reinterpret_cast<const uint4*>(p);
      } else {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (k + j < K) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    reinterpret_cast<uint4*>(dst)[i] = v;
  }
}

__global__ __launch_bounds__(kThreads) void copy_scales(const float* __restrict__ s, int64_t n,
                                                        float* __restrict__ dst) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kThreads)
    dst[i] = s[i];
}

// out[t] = bf16(sum over local slots, ascending, of w * y), rounded once.  A wave
// owns 64 x kPieces 16-byte pieces of one token's row, so ids and weights are
// uniform: scalar loads, and no load at all for a slot without a row; two slots
// of a batch are on their way together (8192 tokens with one local slot each:
// batches of 2, 4, 8 take 44.5, 50, 62 us, the registers of larger ones cost
// waves; one thread per 16 bytes with its own ids 84).  Bound by memory.
constexpr int kCombineWaves = 4;
constexpr int kPieces = 2;
constexpr int kPiece = 8;  // outputs per piece

__global__ __launch_bounds__(64 * kCombineWaves) void combine_slots(F8CombineArgs a) {
  constexpr int B = 2;  // slots per batch
  const int nvec = a.H / kPiece, spans = (nvec + 64 * kPieces - 1) / (64 * kPieces);
  const int64_t wid = (int64_t)blockIdx.x * kCombineWaves + (threadIdx.x >> 6);
  const int t = __builtin_amdgcn_readfirstlane((int)(wid / spans));
  if (t >= a.T) return;
  const int v0 = __builtin_amdgcn_readfirstlane((int)(wid - (int64_t)t * spans)) * 64 * kPieces +
                 (int)(threadIdx.x & 63);
  const int64_t s0 = (int64_t)t * a.k;
  const int blocks = a.H / kF8YBlock;
  float acc[kPieces][kPiece];
#pragma unroll
  for (int p = 0; p < kPieces; ++p)
#pragma unroll
    for (int i = 0; i < kPiece; ++i) acc[p][i] = 0.f;
  for (int j0 = 0; j0 < a.k; j0 += B) {
    bool local[B];
#pragma unroll
    for (int u = 0; u < B; ++u) {
      const int e = a.topk_ids[s0 + min(j0 + u, a.k - 1)];
      // (unsigned difference: no id, however far off, wraps into the range)
      local[u] = j0 + u < a.k && e >= a.expert_begin &&
                 (uint32_t)e - (uint32_t)a.expert_begin < (uint32_t)a.num_experts;
    }
    u32x4_t y[B][kPieces];
    uint32_t exponent[B][kPieces];
    float w[B];
#pragma unroll
    for (int u = 0; u < B; ++u) {
      if (!local[u]) continue;
      const int64_t f = s0 + j0 + u;
      w[u] = a.topk_weights[f];
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const int v = min(v0 + 64 * p, nvec - 1);
        y[u][p] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(a.y + f * a.H) + v);
        exponent[u][p] = a.yu[f * blocks + v / (kF8YBlock / kPiece)];
      }
    }
#pragma unroll
    for (int u = 0; u < B; ++u) {
      if (!local[u]) continue;
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const float unit = __uint_as_float(exponent[u][p] << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const half2_t h = __builtin_bit_cast(half2_t, (uint32_t)y[u][p][i]);
          acc[p][2 * i] = __builtin_fmaf(w[u], unit * (float)h[0], acc[p][2 * i]);
          acc[p][2 * i + 1] = __builtin_fmaf(w[u], unit * (float)h[1], acc[p][2 * i + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int v = v0 + 64 * p;
    if (v >= nvec) continue;
    *reinterpret_cast<uint4*>(a.out + (int64_t)t * a.H + (int64_t)v * kPiece) =
        make_uint4(pk_bf16(acc[p][0], acc[p][1]), pk_bf16(acc[p][2], acc[p][3]),
                   pk_bf16(acc[p][4], acc[p][5]), pk_bf16(acc[p][6], acc[p][7]));
  }
}

unsigned grid_for(int64_t n, int64_t per, int64_t most) {
  const int64_t b = (n + per - 1) / per;
  return (unsigned)(b < 1 ? 1 : b > most ? most : b);
}

}  // namespace

hipError_t launch_f8_quantize(const F8QuantArgs& a, hipStream_t stream) {
  const int64_t groups = a.T * f8_chunks(a.K);
  const dim3 grid(grid_for(groups, kGroupsPerPass, 1 << 20)), block(kThreads);
  const int size = a.is_f32 ? 4 : 2;
  const bool wide = a.K % 8 == 0 && a.ld * size % 16 == 0 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0;
  if (a.is_f32 && !wide) return hipErrorInvalidValue;
  if (a.is_f32) hipLaunchKernelGGL((quantize_kernel<true, true>), grid, block, 0, stream, a);
  else if (wide) hipLaunchKernelGGL((quantize_kernel<false, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((quantize_kernel<false, false>), grid, block, 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_f8_combine(const F8CombineArgs& a, hipStream_t stream) {
  const int per = 64 * kPieces * kPiece;
  const int64_t waves = (int64_t)a.T * ((a.H + per - 1) / per);
  const dim3 grid((unsigned)((waves + kCombineWaves - 1) / kCombineWaves)), block(64 * kCombineWaves);
  hipLaunchKernelGGL(combine_slots, grid, block, 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_f8_pack(const uint8_t* q, const float* s, int E, int N, int K, int gate_up,
                          uint8_t* dst, hipStream_t stream) {
  const int64_t n = (int64_t)f8_code_bytes(E, N, K) / 16;
  hipLaunchKernelGGL(pack_codes, dim3(grid_for(n, kThreads, 1 << 16)), dim3(kThreads), 0, stream, q, E,
                     N, K, gate_up, dst);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t ns = (int64_t)E * ((N + kF8Block - 1) / kF8Block) * f8_chunks(K);
  hipLaunchKernelGGL(copy_scales, dim3(grid_for(ns, kThreads, 4096)), dim3(kThreads), 0, stream, s, ns,
                     reinterpret_cast<float*>(dst + f8_code_bytes(E, N, K)));
  return hipGetLastError();
}

}  // namespace chord
