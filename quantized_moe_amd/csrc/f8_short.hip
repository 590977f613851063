// Down product of a layer whose intermediate size is at most 256 (a
// tensor-parallel slice): K is one or two chunks, so the tokens of an alignment
// block (16 or 32 rows) fit a wave's registers once and for all, and a wave then
// streams weight tiles, 16 output features each, past them.  Nothing is staged
// and no wave waits for another.  Bound by the weights' bytes: four tiles are on
// their way while one is multiplied.
//
// Against the tiled kernel, whose workgroups drain and refill their pipeline for
// every 256 features: 384 experts, 512 tokens, 7168 x 256 weights, 180 -> 160 us.
#include "f8_common.h"

namespace chord {
namespace {

constexpr int kWavesPerBlock = 4;
constexpr int kRing = 4;      // tiles in flight
constexpr int kPart = 28;     // tiles per wave at most

__device__ __forceinline__ i32x8_t operand(u32x4_t a, u32x4_t b) {
  return i32x8_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

template <int NC, int G>
__global__ __launch_bounds__(64 * kWavesPerBlock) void f8_short_down(F8GemmArgs a, int parts) {
  const int lane = threadIdx.x & 63, q = lane >> 4, col = lane & 15;
  const int64_t used = max((int64_t)0, min((int64_t)*a.ntpp, a.max_padded));
  const int64_t items = used / a.block_m * parts;
  const int64_t step = (int64_t)gridDim.x * kWavesPerBlock;
  for (int64_t item = (int64_t)blockIdx.x * kWavesPerBlock +
                      __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
       item < items; item += step) {
    const int blk = (int)(item / parts), part = (int)(item - (int64_t)blk * parts);
    const int e = a.expert_ids[blk];
    if (e < 0 || e >= a.num_experts) continue;
    const int t0 = (int)((int64_t)a.n_tiles * part / parts);
    const int t1 = (int)((int64_t)a.n_tiles * (part + 1) / parts);
    const uint8_t* wbase = a.wq + (int64_t)e * a.n_tiles * NC * kF8BlockBytes + lane * 16;
    u32x4_t w[kRing][NC][2];
    auto load_w = [&](int r, int t) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const uint8_t* p = wbase + (int64_t)f8_block(t, c, a.n_tiles, NC) * kF8BlockBytes;
        w[r][c][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
        w[r][c][1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p + 1024));
      }
    };
#pragma unroll
    for (int r = 0; r < kRing; ++r) load_w(r, min(t0 + r, t1 - 1));
    // This block's tokens: operands and scales.  Lanes of padding rows read row 0
    // and store nothing.
    i32x8_t x[NC][G];
    float sx[NC][G];
    float* out[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int64_t R = (int64_t)blk * a.block_m + g * 16 + col;
      const int64_t f = a.sorted_ids[R];
      const bool live = f >= 0 && f < a.n_flat;
      out[g] = live ? static_cast<float*>(a.out) + f * a.ld + 4 * q : nullptr;
      const int64_t src = live ? R : 0;
      const uint8_t* p = a.aq + src * (NC * kF8Block) + q * 32;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        x[c][g] = operand(*reinterpret_cast<const u32x4_t*>(p + c * kF8Block),
                          *reinterpret_cast<const u32x4_t*>(p + c * kF8Block + 16));
        sx[c][g] = a.as[src * NC + c];
      }
    }
    const float* sw = a.ws + (int64_t)e * a.nb * NC;
    for (int t = t0; t < t1; t += kRing) {
#pragma unroll
      for (int r = 0; r < kRing; ++r) {
        if (t + r >= t1) break;
        f32x4_t acc[G];
#pragma unroll
        for (int g = 0; g < G; ++g) acc[g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float s = sw[(t + r) / 8 * NC + c];
          const i32x8_t wv = operand(w[r][c][0], w[r][c][1]);
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
            const f32x4_t v = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, x[c][g], zero, 0, 0,
                                                                               0, 0, 0, 0);
            const float f = s * sx[c][g];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[g][i] = __builtin_fmaf(v[i], f, acc[g][i]);
          }
        }
        load_w(r, min(t + r + kRing, t1 - 1));
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (out[g] != nullptr) *reinterpret_cast<f32x4_t*>(out[g] + (t + r) * 16) = acc[g];
      }
    }
  }
}

}  // namespace

hipError_t launch_f8_short_down(const F8GemmArgs& a, hipStream_t stream) {
  // Tiles per wave: kPart, fewer where the expected blocks leave SIMDs without a
  // wave (one token, eight experts: 22.7 -> 9 us).
  const int want = (int)((int64_t)4 * 4 * a.num_cus / (a.est_blocks > 0 ? a.est_blocks : 1));
  const int least = (a.n_tiles + kPart - 1) / kPart;
  const int parts = want < least ? least : want > a.n_tiles ? a.n_tiles : want;
  const int64_t items = (a.max_padded / a.block_m + 1) * parts;
  const int64_t blocks = (items + kWavesPerBlock - 1) / kWavesPerBlock;
  const int64_t most = (int64_t)a.num_cus * 16;
  const dim3 grid((unsigned)(blocks < most ? blocks : most)), block(64 * kWavesPerBlock);
  if (a.n_chunks == 1) {
    if (a.block_m <= 16) hipLaunchKernelGGL((f8_short_down<1, 1>), grid, block, 0, stream, a, parts);
    else hipLaunchKernelGGL((f8_short_down<1, 2>), grid, block, 0, stream, a, parts);
  } else {
    if (a.block_m <= 16) hipLaunchKernelGGL((f8_short_down<2, 1>), grid, block, 0, stream, a, parts);
    else hipLaunchKernelGGL((f8_short_down<2, 2>), grid, block, 0, stream, a, parts);
  }
  return hipGetLastError();
}

}  // namespace chord
