// Dense product in 16 bits with its epilogue:
//
//   z = x W^T + bias,  h = act(z) or act(z of the gate) * z of the up rows,
//   out = [residual +] scale h
//
// Weights are the A operand of the matrix instruction (16 outputs), tokens the B
// operand, so a lane's four results are four neighbouring outputs of one token.
#include "linear_common.h"

namespace chord {
namespace {

// One wave per 16 tokens x 16 outputs, operands value by value from memory.
template <bool F16>
__global__ __launch_bounds__(64) void linear_plain(LinearArgs a) {
  const int lane = threadIdx.x, q = lane >> 4, col = lane & 15;
  const int64_t tiles = (a.N + 15) / 16, items = (a.M + 15) / 16 * tiles;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t m = it / tiles * 16 + col;
    const int n0 = (int)(it % tiles) * 16;
    const int n = n0 + col;
    f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    for (int k0 = 0; k0 < a.K; k0 += 32) {
      Operand x, w[2];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = k0 + q * 8 + i;
        x.h[i] = m < a.M && k < a.K ? a.x[m * a.ldx + k] : 0;
        w[0].h[i] = n < a.N && k < a.K ? a.w[(int64_t)n * a.ldw + k] : 0;
        w[1].h[i] = a.gated && n < a.N && k < a.K ? a.w[(int64_t)(a.N + n) * a.ldw + k] : 0;
      }
      acc[0] = mfma<F16>(w[0], x, acc[0]);
      if (a.gated) acc[1] = mfma<F16>(w[1], x, acc[1]);
    }
    if (m >= a.M) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int o = n0 + 4 * q + i;
      if (o < a.N) store_out(a, m, o, acc[0][i], acc[1][i]);
    }
  }
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t stream) {
  const int64_t items = (a.M + 15) / 16 * ((a.N + 15) / 16), most = (int64_t)1 << 20;
  const dim3 grid((unsigned)(items < most ? items : most));
  if (a.f16) hipLaunchKernelGGL(linear_plain<true>, grid, dim3(64), 0, stream, a);
  else hipLaunchKernelGGL(linear_plain<false>, grid, dim3(64), 0, stream, a);
  return hipGetLastError();
}

}  // namespace chord
