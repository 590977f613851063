// Down product of a layer whose intermediate size is at most 256 (a
// tensor-parallel slice): K is one or two chunks, so the tokens of an alignment
// block (16 or 32 rows) fit a wave's registers once and for all, and a wave then
// streams weight tiles, 16 output features each, past them.  Nothing is staged
// and no wave waits for another.  Bound by the weights' bytes: four tiles are on
// their way while one is multiplied.
//
// Against the tiled kernel, whose workgroups drain and refill their pipeline for
// every 256 features: 384 experts, 512 tokens, 7168 x 256 weights, 180 -> 160 us
// with y in fp32, and 150 with y in fp16 (0.83 GB of weights and y, 5.5 TB/s).
#include "f8_common.h"

namespace chord {
namespace {

constexpr int kWavesPerBlock = 4;
constexpr int kRing = 4;      // tiles in flight
// Tiles per wave at most (about: they come in pairs).  Of little weight: with 16, 24,
// 28, 32 and 48 a layer of 512 tokens on 384 experts of 7168 x 256 takes 441, 434, 428,
// 438, 436 us, of 256 tokens on 160 of 5120 x 256 174, 175, 177, 174, 173, on 256 of
// 2048 x 128 67, 67, 68, 68, 67.
constexpr int kPart = 28;

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
    // Pairs of tiles, a block of y each (the tiles' number is a multiple of 8).
    const int t0 = (int)((int64_t)(a.n_tiles / 2) * part / parts) * 2;
    const int t1 = (int)((int64_t)(a.n_tiles / 2) * (part + 1) / parts) * 2;
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
    int64_t out[G];  // slot, or -1
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int64_t R = (int64_t)blk * a.block_m + g * 16 + col;
      const int64_t f = a.sorted_ids[R];
      const bool live = f >= 0 && f < a.n_flat;
      out[g] = live ? f : -1;
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
    uint16_t* y = static_cast<uint16_t*>(a.out) + 16 * (q & 1) + 8 * (q >> 1);
    for (int t = t0; t < t1; t += kRing) {
#pragma unroll
      for (int r0 = 0; r0 < kRing; r0 += 2) {
        if (t + r0 >= t1) break;
        f32x4_t acc[2][G];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int r = r0 + n;
#pragma unroll
          for (int g = 0; g < G; ++g) acc[n][g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
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
              for (int i = 0; i < 4; ++i) acc[n][g][i] = __builtin_fmaf(v[i], f, acc[n][g][i]);
            }
          }
          load_w(r, min(t + r + kRing, t1 - 1));
        }
        const int block = (t + r0) / 2;
        uint32_t e = 0;  // lane quarter q: exponent of group q
#pragma unroll
        for (int g = 0; g < G; ++g) {
          u32x4_t v;
          const uint32_t eg = f8_y_pack(acc[0][g], acc[1][g], v);
          if (out[g] >= 0) *reinterpret_cast<u32x4_t*>(y + out[g] * a.ld + block * kF8YBlock) = v;
          e = q == g ? eg : e;
        }
        const int64_t d = G > 1 && q == 1 ? out[G - 1] : out[0];
        if (q < G && d >= 0) a.yu[d * (a.N / kF8YBlock) + block] = (uint8_t)e;
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
  const int parts = want < least ? least : want > a.n_tiles / 2 ? a.n_tiles / 2 : want;
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
