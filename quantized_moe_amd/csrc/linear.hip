// Dense product in 16 bits, form for few rows, and what both forms need beside them:
//
//   z = x W^T + bias,  h = act(z) or act(z of the gate) * z of the up rows,
//   out = [residual +] scale h
//
// Weights are the A operand of the matrix instruction (16 rows of W), tokens the B
// operand, so a lane's four results are four neighbouring outputs of one token.  A
// workgroup streams 16 rows of W (gated: 8 gate rows and their 8 up rows) from memory
// straight into registers; its waves split K and add up through LDS.
#include <type_traits>

#include "linear_common.h"

namespace chord {
namespace {

// 16 tokens x 16 rows of W a workgroup, K over WK waves, PF steps of 64 on their way.
template <bool F16, int WK, int PF>
__global__ __launch_bounds__(64 * WK) void linear_stream(LinearArgs a) {
  __shared__ f32x4_t red[WK][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, col = lane & 15;
  const int per = a.gated ? 8 : 16;  // outputs of a workgroup
  const int tiles = (a.N + per - 1) / per;
  const int steps = (a.K + 63) / 64;
  const int c_lo = (int)((int64_t)steps * wave / WK), c_hi = (int)((int64_t)steps * (wave + 1) / WK);
  const int64_t items = (a.M + 15) / 16 * tiles;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t m0 = it / tiles * 16;
    const int n0 = (int)(it % tiles) * per;
    // Rows of this lane; lanes without one read nothing, which is zeros.
    const int mine = a.gated ? col & 7 : col;
    const bool has_w = n0 + mine < a.N, has_x = m0 + col < a.M;
    // (From the first gate row: up rows are N rows further on, so the offset of a
    // lane's row is in the base of its half.)
    const uint16_t* wp = a.w + (int64_t)(n0 + (has_w ? mine : 0) + (a.gated && col >= 8 ? a.N : 0)) * a.ldw;
    const uint16_t* xp = a.x + (m0 + (has_x ? col : 0)) * a.ldx;
    u32x4_t w[PF][2], x[PF][2];
    const u32x4_t zero = {0u, 0u, 0u, 0u};
    auto load = [&](int p, int c) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = c * 64 + j * 32 + q * 8;
        const bool in = k < a.K;
        w[p][j] = in && has_w ? __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(wp + k)) : zero;
        x[p][j] = in && has_x ? *reinterpret_cast<const u32x4_t*>(xp + k) : zero;
      }
    };
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < PF; ++p)
      if (c_lo + p < c_hi) load(p, c_lo + p);
    for (int c = c_lo; c < c_hi; c += PF) {
#pragma unroll
      for (int p = 0; p < PF; ++p) {
        if (c + p < c_hi) {
          acc = mfma16<F16>(w[p][0], x[p][0], acc);
          acc = mfma16<F16>(w[p][1], x[p][1], acc);
        }
        if (c + p + PF < c_hi) load(p, c + p + PF);
      }
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (wave == 0 && has_x && q * 4 < per) {
      f32x4_t z = red[0][lane], up = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 1; u < WK; ++u) z += red[u][lane];
      if (a.gated) {
#pragma unroll
        for (int u = 0; u < WK; ++u) up += red[u][lane + 32];
      }
      store_out4(a, m0 + col, n0 + 4 * q, z, up);
    }
    __syncthreads();
  }
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

// Rows of K values to 16-byte aligned rows of `to` values, the rest of them zeros.
__global__ __launch_bounds__(256) void copy_rows(const uint16_t* __restrict__ src, int64_t ld, int64_t rows, int K,
                                                 int to, uint16_t* __restrict__ dst) {
  const int vecs = to / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * vecs; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / vecs;
    const int k = (int)(i - r * vecs) * 8;
    const uint16_t* p = src + r * ld + k;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k + j < K) w[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
    reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace

hipError_t launch_linear_stream(const LinearArgs& a, hipStream_t stream) {
  const int per = a.gated ? 8 : 16;
  const int64_t items = (a.M + 15) / 16 * ((a.N + per - 1) / per), most = (int64_t)1 << 20;
  const dim3 grid((unsigned)(items < most ? items : most));
  auto run = [&](auto kernel, int waves) {
    hipLaunchKernelGGL(kernel, grid, dim3(64 * waves), 0, stream, a);
    return hipGetLastError();
  };
  return a.f16 ? run(linear_stream<true, 16, 4>, 16) : run(linear_stream<false, 16, 4>, 16);
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
