// Dense product in 16 bits, form for few rows, and what both forms need beside them:
//
//   z = x W^T + bias,  h = act(z) or act(z of the gate) * z of the up rows,
//   out = [residual +] scale h
//
// Weights are the A operand of the matrix instruction (16 rows of W), tokens the B
// operand, so a lane's four results are four neighbouring outputs of one token.  A
// workgroup takes 16 rows of W (gated: 8 gate rows and their 8 up rows) and up to 64
// tokens; its waves take every eighth chunk of 64 along K and add up through LDS.
//
// A wave brings its chunks by buffer_load ... lds into a ring of its own, eight lanes to
// a row's 128 bytes, and reads them back as operands: no wave waits for another.  (Rows
// loaded as operands are a request for every lane: one token through 4096 x 7168 took
// 32 us so.)
//
// Bound by memory: one token through 4096 x 7168 (59 MB) in 12.2 us with its launch, 4.8
// TB/s (11.5 at a copy's 5.1); 64 tokens through 384 x 7168 in 8.7, 14 chunks a wave
// from a cold start.  With more tokens the lines that a CU takes bound it: (16 + tokens)
// x 128 bytes for each chunk of each wave.
#include <type_traits>

#include "linear_common.h"

namespace chord {
namespace {

constexpr int kStreamWaves = 8;
constexpr int kChunk = 64, kRowBytes = 2 * kChunk;

// XI: groups of 8 tokens; DEPTH: chunks of a wave on their way.  (Ordinary loads of
// weights: as non-temporal ones they, and the tokens beside them, took 14.1 us for 12.4
// with 16 tokens through 4096 x 7168.)
template <bool F16, int XI, int DEPTH>
__device__ __forceinline__ void stream_rows(const LinearArgs& a, uint8_t* lds) {
  constexpr int MT = XI / 2;  // token operands
  constexpr int kLoads = 2 + XI, kSlot = kLoads * 1024;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, col = lane & 15;
  uint8_t* const ring = lds + wave * (DEPTH * kSlot);
  const int per = a.gated ? 8 : 16;  // outputs of a workgroup
  const int tiles = (a.N + per - 1) / per;
  const int chunks = (a.K + kChunk - 1) / kChunk, tail = a.K - (chunks - 1) * kChunk;
  const int mine = (chunks - wave + kStreamWaves - 1) / kStreamWaves;
  // Lane's row and 16-byte piece in a load, and in an operand (as the tiled form).
  const int r = lane >> 3, p = (lane & 7) ^ (r & 6);
  const bool in_tail = p * 8 < tail;
  const int piece[2] = {(q ^ (col & 6)) * 16, ((4 + q) ^ (col & 6)) * 16};
  typedef __attribute__((address_space(3))) void* Lds;

  const int64_t items = (a.M + 8 * XI - 1) / (8 * XI) * tiles;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t m0 = (int64_t)__builtin_amdgcn_readfirstlane((int)(it / tiles)) * (8 * XI);
    const int n0 = __builtin_amdgcn_readfirstlane((int)(it % tiles)) * per;
    const int rows = (int)min((int64_t)(8 * XI), a.M - m0);
    const int lo = min(8, a.N - n0), hi = a.gated ? lo : max(0, min(8, a.N - n0 - 8));
    const __amdgpu_buffer_rsrc_t xres = row_buffer(a.x + m0 * a.ldx, rows, a.ldx, a.K);
    const __amdgpu_buffer_rsrc_t wres = row_buffer(a.w + (int64_t)n0 * a.ldw, lo, a.ldw, a.K);
    const __amdgpu_buffer_rsrc_t ures = row_buffer(a.w + ((int64_t)(a.gated ? a.N : 8) + n0) * a.ldw, hi, a.ldw, a.K);
    const uint32_t w_lo = r < lo ? (uint32_t)(r * a.ldw * 2 + p * 16) : kLinNothing;
    const uint32_t w_hi = r < hi ? (uint32_t)(r * a.ldw * 2 + p * 16) : kLinNothing;
    uint32_t xo[XI];
#pragma unroll
    for (int i = 0; i < XI; ++i) xo[i] = 8 * i + r < rows ? (uint32_t)((8 * i + r) * a.ldx * 2 + p * 16) : kLinNothing;
    auto load = [&](int slot, int i) {  // the wave's chunk i
      const int c = wave + i * kStreamWaves;
      const bool out = c == chunks - 1 && !in_tail;
      uint8_t* const to = ring + slot * kSlot;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wres, (Lds)to, 16, out ? kLinNothing : w_lo, c * kRowBytes, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ures, (Lds)(to + 1024), 16, out ? kLinNothing : w_hi, c * kRowBytes, 0,
                                               0);
#pragma unroll
      for (int x = 0; x < XI; ++x)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(xres, (Lds)(to + 2048 + x * 1024), 16, out ? kLinNothing : xo[x],
                                                 c * kRowBytes, 0, 0);
    };
    auto wait = [&](auto outstanding) {
      constexpr int vm = decltype(outstanding)::value;
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt((vm & 15) | (7 << 4) | (15 << 8) | ((vm >> 4) << 14));
      __builtin_amdgcn_sched_barrier(0);
    };
    f32x4_t acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](int slot) {
      const uint8_t* const at = ring + slot * kSlot + col * kRowBytes;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(at + piece[j]);
#pragma unroll
        for (int t = 0; t < MT; ++t)
          acc[t] = mfma16<F16>(w, *reinterpret_cast<const u32x4_t*>(at + 2048 + t * 2048 + piece[j]), acc[t]);
      }
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (d < mine) load(d, d);
    int slot = 0;
    for (int i = 0; i < mine; ++i) {
      if (i + DEPTH <= mine) wait(std::integral_constant<int, (DEPTH - 1) * kLoads>{});
      else wait(std::integral_constant<int, 0>{});
      compute(slot);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));  // the slot is read
      __builtin_amdgcn_sched_barrier(0);
      if (i + DEPTH < mine) load(slot, i + DEPTH);
      slot = slot + 1 == DEPTH ? 0 : slot + 1;
    }
    __syncthreads();
    f32x4_t* const red = reinterpret_cast<f32x4_t*>(lds);  // [waves][MT][64]
#pragma unroll
    for (int t = 0; t < MT; ++t) red[(wave * MT + t) * 64 + lane] = acc[t];
    __syncthreads();
    if (wave < MT) {
      const int64_t m = m0 + wave * 16 + col;
      if (wave * 16 + col < rows && q * 4 < per) {
        f32x4_t z = {0.f, 0.f, 0.f, 0.f}, up = z;
#pragma unroll
        for (int u = 0; u < kStreamWaves; ++u) z += red[(u * MT + wave) * 64 + lane];
        if (a.gated) {
#pragma unroll
          for (int u = 0; u < kStreamWaves; ++u) up += red[(u * MT + wave) * 64 + lane + 32];
        }
        store_out4(a, m, n0 + 4 * q, z, up);
      }
    }
    __syncthreads();
  }
}

template <bool F16, int XI, int DEPTH>
__global__ __launch_bounds__(64 * kStreamWaves) void linear_stream(LinearArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  stream_rows<F16, XI, DEPTH>(a, lds);
}

// Adds the parts of K, ascending, and finishes the outputs.
__global__ __launch_bounds__(256) void linear_join(LinearArgs a) {
  const int half = (a.N + 15) / 16 * 16, pitch = a.gated ? 2 * half : half, quads = half / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.M * quads; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / quads;
    const int n = (int)(i - m * quads) * 4;
    f32x4_t z = {0.f, 0.f, 0.f, 0.f}, up = z;
    const float* p = a.partials + m * pitch + n;
#pragma unroll 4
    for (int u = 0; u < a.parts; ++u) {
      z += *reinterpret_cast<const f32x4_t*>(p + (int64_t)u * a.M * pitch);
      if (a.gated) up += *reinterpret_cast<const f32x4_t*>(p + (int64_t)u * a.M * pitch + half);
    }
    store_out4(a, m, n, z, up);
  }
}

// (A vector of words that need no more than a word's alignment.)
typedef uint32_t u32x4a4_t __attribute__((ext_vector_type(4), aligned(4)));

// Rows of K values to 16-byte aligned rows of `to` values, the rest of them zeros.
__global__ __launch_bounds__(256) void copy_rows(const uint16_t* __restrict__ src, int64_t ld, int64_t rows, int K,
                                                 int to, uint16_t* __restrict__ dst) {
  const int vecs = to / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * vecs; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / vecs;
    const int k = (int)(i - r * vecs) * 8;
    const uint16_t* p = src + r * ld + k;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    // Words of two values; where they lie across the words of memory one value more is
    // read on both sides, as long as that is inside the matrix.
    const bool across = (reinterpret_cast<uintptr_t>(p) & 2) != 0;
    const bool before = k > 0 || r > 0, behind = k + 9 <= K || r + 1 < rows;
    if (!across && k + 8 <= K) {
      const u32x4a4_t v = *reinterpret_cast<const u32x4a4_t*>(p);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = v[j];
    } else if (across && before && behind && k + 8 <= K) {
      const u32x4a4_t v = *reinterpret_cast<const u32x4a4_t*>(p - 1);
      const uint32_t last = *reinterpret_cast<const uint32_t*>(p + 7);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = v[j] >> 16 | (j < 3 ? v[j + 1] : last) << 16;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (k + j < K) w[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
    }
    reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace

hipError_t launch_linear_stream(const LinearArgs& a, int tokens, hipStream_t stream) {
  auto run = [&](auto kernel, int xi, int depth) {
    const int per = a.gated ? 8 : 16;
    const int64_t items = (a.M + 8 * xi - 1) / (8 * xi) * ((a.N + per - 1) / per), most = (int64_t)1 << 20;
    const int lds = kStreamWaves * depth * (2 + xi) * 1024;
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(items < most ? items : most)), dim3(64 * kStreamWaves), lds, stream, a);
    return hipGetLastError();
  };
#define CHORD_LINEAR_STREAM(XI, DEPTH) \
  return a.f16 ? run(linear_stream<true, XI, DEPTH>, XI, DEPTH) : run(linear_stream<false, XI, DEPTH>, XI, DEPTH)
  switch (tokens) {
    case 16: CHORD_LINEAR_STREAM(2, 4);
    case 32: CHORD_LINEAR_STREAM(4, 3);
    default: CHORD_LINEAR_STREAM(8, 2);
  }
#undef CHORD_LINEAR_STREAM
}

hipError_t launch_linear_join(const LinearArgs& a, hipStream_t stream) {
  const int64_t n = (a.M * ((a.N + 15) / 16 * 4) + 255) / 256, most = (int64_t)a.num_cus * 16;
  hipLaunchKernelGGL(linear_join, dim3((unsigned)(n < most ? n : most)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_copy_rows(const uint16_t* src, int64_t ld, int64_t rows, int K, int to, uint16_t* dst,
                            hipStream_t stream) {
  const int64_t n = (rows * (to / 8) + 255) / 256, most = (int64_t)1 << 16;
  hipLaunchKernelGGL(copy_rows, dim3((unsigned)(n < most ? n : most)), dim3(256), 0, stream, src, ld, rows, K, to,
                     dst);
  return hipGetLastError();
}

}  // namespace chord
