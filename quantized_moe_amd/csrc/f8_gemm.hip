// 8-bit GEMM with block scales, weight-streaming form: every workgroup streams
// its packed weight tiles from HBM straight into registers; waves split K and
// add up through LDS.
//
// One v_mfma_f32_16x16x128_f8f6f4 covers exactly one block of 128 along K, so
// its result (from a zero accumulator) is the block's partial product, and
// acc += scale_a * scale_w * partial applies both scales in fp32: four
// multiply-adds a lane beside 32 cycles of matrix work.  Weights are the A
// operand (16 output features), tokens the B operand, so a lane's four results
// belong to one token and share its scale.
//
// Bound by memory: weights of 4096 x 7168 for one token in 7.5 us with their
// launch (a launch of nothing is 3.5 us).  Loads stop at the end of a wave's part of
// K: with the last chunk loaded again in the place of those behind it the ring of
// four took 8.5 us here, and 14.2 for 6.9 with two chunks a wave (16 tokens, 7168 x
// 2048).  A weight tile is read again for each 16 tokens, and a wave has few products
// beside its loads, so with long K and wide N the tiled kernel is the faster one
// from about 30 tokens.
#include "f8_common.h"

namespace chord {
namespace {

__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {
  const u32x4_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ i32x8_t operand(uint4 a, uint4 b) {
  return i32x8_t{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// Four neighbouring outputs, as wide as their place allows.
__device__ __forceinline__ void store4(uint16_t* out, int64_t row, int64_t ld, int n, int N,
                                       f32x4_t v, bool wide) {
  uint16_t* p = out + row * ld + n;
  if (wide && n + 4 <= N) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < N) p[i] = to_bf16(v[i]);
}

// NT weight tiles x 16 tokens a workgroup, K over WK waves, PF chunks on their way.
// GATE_UP: a layer's gate_up over alignment blocks (summed by f8_exact_product),
// else the dense product.
template <int NT, int WK, int PF, bool GATE_UP>
__global__ __launch_bounds__(64 * WK) void f8_stream(F8GemmArgs a) {
  __shared__ f32x4_t red[WK][NT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, col = lane & 15;
  const int nc = a.n_chunks;
  const int c_lo = nc * wave / WK, c_hi = nc * (wave + 1) / WK;
  const bool wide = a.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 7) == 0;
  const int groups = (a.n_tiles + NT - 1) / NT;
  const int64_t pitch = (int64_t)nc * kF8Block;
  int64_t ntok;  // token tiles
  if (GATE_UP) {
    const int64_t used = max((int64_t)0, min((int64_t)*a.ntpp, a.max_padded));
    ntok = used / a.block_m;
  } else {
    ntok = (a.a_rows + 15) / 16;
  }
  for (int64_t item = blockIdx.x; item < ntok * groups; item += gridDim.x) {
    const int ti = (int)(item / groups);
    const int tile0 = (int)(item % groups) * NT;
    int e = 0;
    if (GATE_UP) {
      e = a.expert_ids[ti];
      if (e < 0 || e >= a.num_experts) continue;  // uniform
    }
    // Row of this lane's token; lanes without one read row 0 and store nothing
    // (their results touch no other token).
    int64_t src = 0, dst = -1;
    if (GATE_UP) {
      const int64_t r = (int64_t)ti * a.block_m + col;
      if (col < a.block_m) {
        const int64_t f = a.sorted_ids[r];
        if (f >= 0 && f < a.n_flat) {
          src = f / a.topk;
          dst = r;
        }
      }
    } else {
      const int64_t r = (int64_t)ti * 16 + col;
      if (r < a.a_rows) src = dst = r;
    }
    // NT divides 8, so the tiles of an item share their slice and their block(s)
    // of scales.
    const uint8_t* wp[NT];
    const int wstep = f8_slice_width(tile0, a.n_tiles) * kF8BlockBytes;  // chunk to chunk
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = min(tile0 + n, a.n_tiles - 1);
      wp[n] = a.wq + ((int64_t)e * a.n_tiles * nc + f8_block(t, 0, a.n_tiles, nc)) * kF8BlockBytes +
              lane * 16;
    }
    const float* s0;
    const float* s1;
    if (GATE_UP) {
      s0 = a.ws + ((int64_t)e * a.nb + tile0 / 16) * nc;
      s1 = s0 + (int64_t)(a.nb / 2) * nc;
    } else {
      s0 = s1 = a.ws + (int64_t)(tile0 / 8) * nc;
    }
    const uint8_t* xp = a.aq + src * pitch + q * 32;
    const float* sp = a.as + src * nc;
    f32x4_t acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    uint4 w[PF][NT][2], x[PF][2];
    float sx[PF], sw0[PF], sw1[PF];
    auto load = [&](int p, int c) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        w[p][n][0] = load_stream(wp[n] + (int64_t)c * wstep);
        w[p][n][1] = load_stream(wp[n] + (int64_t)c * wstep + 1024);
      }
      x[p][0] = *reinterpret_cast<const uint4*>(xp + c * kF8Block);
      x[p][1] = *reinterpret_cast<const uint4*>(xp + c * kF8Block + 16);
      sx[p] = sp[c];
      sw0[p] = s0[c];
      sw1[p] = s1[c];
    };
    auto compute = [&](int p) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const i32x8_t av = operand(w[p][n][0], w[p][n][1]), bv = operand(x[p][0], x[p][1]);
        const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
        const f32x4_t r = GATE_UP ? f8_exact_product(av, bv)
                                  : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, zero, 0, 0, 0, 0, 0, 0);
        const float f0 = sx[p] * sw0[p], f1 = sx[p] * sw1[p];
        acc[n][0] = __builtin_fmaf(r[0], f0, acc[n][0]);
        acc[n][1] = __builtin_fmaf(r[1], f1, acc[n][1]);
        acc[n][2] = __builtin_fmaf(r[2], f0, acc[n][2]);
        acc[n][3] = __builtin_fmaf(r[3], f1, acc[n][3]);
      }
    };
    if (c_lo < c_hi) {
#pragma unroll
      for (int p = 0; p < PF; ++p)
        if (c_lo + p < c_hi) load(p, c_lo + p);
      for (int c = c_lo; c < c_hi; c += PF) {
#pragma unroll
        for (int p = 0; p < PF; ++p) {
          if (c + p < c_hi) compute(p);
          if (c + p + PF < c_hi) load(p, c + p + PF);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) red[wave][n][lane] = acc[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n != wave) continue;  // (NT <= WK)
      f32x4_t v = red[0][n][lane];
#pragma unroll
      for (int u = 1; u < WK; ++u) v += red[u][n][lane];
      if (dst < 0 || tile0 + n >= a.n_tiles) continue;
      if (GATE_UP) {
        float* h = static_cast<float*>(a.out) + dst * a.ld + (tile0 + n) * 8 + 2 * q;
        *reinterpret_cast<float2*>(h) = make_float2(silu_mul(v[0], v[1]), silu_mul(v[2], v[3]));
      } else {
        store4(static_cast<uint16_t*>(a.out), dst, a.ld, (tile0 + n) * 16 + 4 * q, a.N, v, wide);
      }
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_f8_gemm(const F8GemmArgs& a, hipStream_t stream) {
  auto run = [&](auto kernel, int nt, int wk, int per_cu) {
    const int64_t tiles = a.kind == kF8Plain ? (a.a_rows + 15) / 16 : a.max_padded / a.block_m + 1;
    const int64_t items = tiles * ((a.n_tiles + nt - 1) / nt);
    const int64_t most = (int64_t)a.num_cus * per_cu;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(items < most ? items : most)), dim3(64 * wk), 0, stream, a);
    return hipGetLastError();
  };
  // A product alone has few tiles: one per workgroup, K over 8 waves (M = 1, N =
  // 4096, K = 7168: 12.8 us with two tiles and 4 waves, 7.8 so).
  if (a.kind == kF8Plain) return run(f8_stream<1, 8, 4, false>, 1, 8, 2);
  return run(f8_stream<2, 4, 4, true>, 2, 4, 4);
}

}  // namespace chord
