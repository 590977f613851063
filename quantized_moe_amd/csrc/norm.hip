// Norms in front of and behind a block, with its gate, residual and residual scale:
//
//   u = x or N(x; post),  s = [residual +] scale [gate] u,  y = N(s; pre)
//   N(v; w, b) = (v - m) / sqrt(q + eps) (w + offset) + b
//
// A row lives in the registers of its threads from the one time it is read to the
// one time it is written, so the pass is bound by memory, whichever of the stages
// it has.
#include "f8_common.h"

namespace chord {
namespace {

constexpr int kMaxWaves = 16;
constexpr float kShrink = 0x1p-96f;  // of rows whose squares overflow (2^128 2^-96 squared is far below)

// Eight neighbouring values as they lie in memory: fp32, or 16 bits each in lo.
struct Raw8 {
  u32x4_t lo, hi;
};

template <bool WIDE>
__device__ __forceinline__ Raw8 load_raw(const void* base, int dtype, int64_t at, int n) {
  Raw8 r;
  r.lo = r.hi = u32x4_t{0u, 0u, 0u, 0u};
  if (n <= 0) return r;
  if (dtype == CHORD_DTYPE_F32) {
    const uint32_t* p = static_cast<const uint32_t*>(base) + at;
    if (WIDE) {
      r.lo = *reinterpret_cast<const u32x4_t*>(p);
      r.hi = *reinterpret_cast<const u32x4_t*>(p + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < n) r.lo[i] = p[i];
        if (i + 4 < n) r.hi[i] = p[i + 4];
      }
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if (WIDE) {
      r.lo = *reinterpret_cast<const u32x4_t*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) r.lo[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
  }
  return r;
}
__device__ __forceinline__ void widen(const Raw8& r, int dtype, float (&v)[8]) {
  if (dtype == CHORD_DTYPE_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(r.lo[i]);
      v[i + 4] = __uint_as_float(r.hi[i]);
    }
  } else if (dtype == CHORD_DTYPE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_to_f32(r.lo[i] & 0xFFFFu);
      v[2 * i + 1] = __uint_as_float(r.lo[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const half2_t h = __builtin_bit_cast(half2_t, (uint32_t)r.lo[i]);
      v[2 * i] = (float)h[0];
      v[2 * i + 1] = (float)h[1];
    }
  }
}
__device__ __forceinline__ float one_value(const void* base, int dtype, int64_t at) {
  if (dtype == CHORD_DTYPE_F32) return static_cast<const float*>(base)[at];
  const uint16_t h = static_cast<const uint16_t*>(base)[at];
  return dtype == CHORD_DTYPE_BF16 ? bf16_to_f32(h) : (float)__builtin_bit_cast(_Float16, h);
}
template <bool WIDE>
__device__ __forceinline__ void store8(void* base, int dtype, int64_t at, int n, const float (&v)[8]) {
  if (n <= 0) return;
  if (dtype == CHORD_DTYPE_F32) {
    float* p = static_cast<float*>(base) + at;
    if (WIDE) {
      *reinterpret_cast<f32x4_t*>(p) = f32x4_t{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4_t*>(p + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = v[i];
    }
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = dtype == CHORD_DTYPE_BF16 ? pk_bf16(v[2 * i], v[2 * i + 1]) : pk_f16(v[2 * i], v[2 * i + 1]);
  uint16_t* p = static_cast<uint16_t*>(base) + at;
  if (WIDE) {
    *reinterpret_cast<u32x4_t*>(p) = u32x4_t{w[0], w[1], w[2], w[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}

// Sum over the threads of a row: register moves inside a wave, LDS between waves.
// `slot` alternates, so one barrier a sum is enough.
struct RowSum {
  float (*part)[kMaxWaves];
  int waves, slot;
  __device__ __forceinline__ float operator()(float x) {
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
    if (waves == 1) return x;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) part[slot][wave] = x;
    __syncthreads();
    x = 0.f;
    for (int w = 0; w < waves; ++w) x += part[slot][w];
    slot ^= 1;
    return x;
  }
};

// v (0 from column H on) less its mean (LAYER), times the factor that is returned, is
// the norm without its weights.
template <int V>
__device__ __forceinline__ float centre(float (&v)[V][8], const int (&n)[V], const NormPart& p, int H,
                                        RowSum& sum) {
  float eps = p.eps, total = 0.f;
  for (int round = 0;; ++round) {
    float shift = 0.f;
    if (p.kind == CHORD_NORM_LAYER) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) t += v[i][j];
      shift = sum(t) / (float)H;
    }
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = j < n[i] ? v[i][j] - shift : 0.f;
        t += d * d;
      }
    total = sum(t);
    // (Uniform over the row's threads.  A row with an infinity or NaN stays so.)
    if (round == 1 || __builtin_isfinite(total)) {
      if (p.kind == CHORD_NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = j < n[i] ? v[i][j] - shift : 0.f;
      }
      break;
    }
    eps *= kShrink * kShrink;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= kShrink;
  }
  return 1.f / sqrtf(total / (float)H + eps);
}

// B threads hold a row, V times 8 neighbouring values each; a workgroup has one
// row, or one a wave where a wave is enough.
template <int V, bool WIDE>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a) {
  __shared__ float part[2][kMaxWaves];
  const bool alone = a.threads > 64;  // ... in its workgroup
  const int tid = alone ? threadIdx.x : threadIdx.x & 63;
  RowSum sum{part, alone ? a.threads >> 6 : 1, 0};
  int col[V], n[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    col[i] = (i * a.threads + tid) * 8;
    n[i] = min(8, a.H - col[i]);
  }
  auto load = [&](const void* p, int dtype, int64_t row, Raw8 (&r)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = load_raw<WIDE>(p, dtype, row + col[i], n[i]);
  };
  // (Whole waves leave, where a wave has a row; else the workgroup's rows are there
  // for all of its waves.)
  const int64_t step = alone ? (int64_t)gridDim.x : (int64_t)gridDim.x * (blockDim.x >> 6);
  for (int64_t t = alone ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
       t < a.T; t += step) {
    Raw8 x[V], r[V], w[V], b[V];
    load(a.x, a.dtype, t * a.ldx, x);
    if (a.residual != nullptr) load(a.residual, a.stream_dtype, t * a.ldr, r);
    float v[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) widen(x[i], a.dtype, v[i]);

    auto norm = [&](const NormPart& p) {
      load(p.weight, p.dtype, 0, w);
      if (p.bias != nullptr) load(p.bias, p.dtype, 0, b);
      const float inv = centre<V>(v, n, p, a.H, sum);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float f[8];
        widen(w[i], p.dtype, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * inv * (f[j] + p.offset);
        if (p.bias != nullptr) {
          widen(b[i], p.dtype, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] += f[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = j < n[i] ? v[i][j] : 0.f;
      }
    };
    auto gated = [&](float g) { return a.gate_sigmoid ? 1.f / (1.f + expf(-g)) : g; };

    if (a.post.weight != nullptr) norm(a.post);
    float scale = a.scale;
    if (a.gate != nullptr) {
      if (a.gate_col == 0) {
        scale *= gated(one_value(a.gate, a.gate_dtype, t * a.gate_row));
      } else {
        load(a.gate, a.gate_dtype, t * a.gate_row, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float f[8];
          widen(w[i], a.gate_dtype, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] *= gated(f[j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float f[8];
      if (a.residual != nullptr) {
        widen(r[i], a.stream_dtype, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = __builtin_fmaf(v[i][j], scale, f[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= scale;
      }
      if (a.sum != nullptr) store8<WIDE>(a.sum, a.stream_dtype, t * a.lds + col[i], n[i], v[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = j < n[i] ? v[i][j] : 0.f;  // (0 * an infinite gate)
    }
    if (a.pre.weight == nullptr) continue;
    norm(a.pre);
    const int groups = (a.H + kF8Block - 1) / kF8Block;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (a.out != nullptr) store8<WIDE>(a.out, a.dtype, t * a.ldo + col[i], n[i], v[i]);
      if (a.codes != nullptr) {  // 16 lanes hold a group (by all of them)
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
        const F8Group q = f8_group(row_max16(m));
        float c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = q.inv != 0.f ? f8_value(q, v[i][j]) : 0.f;
        if (col[i] < groups * kF8Block) {
          uint2 o;
          o.x = f8_pack4(c[0], c[1], c[2], c[3]);
          o.y = f8_pack4(c[4], c[5], c[6], c[7]);
          *reinterpret_cast<uint2*>(a.codes + t * groups * kF8Block + col[i]) = o;
          if ((tid & 15) == 0) a.code_scales[t * groups + col[i] / kF8Block] = q.scale;
        }
      }
    }
  }
}

bool wide_rows(const void* p, int64_t ld, int dtype) {
  const int size = dtype == CHORD_DTYPE_F32 ? 4 : 2;
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0);
}
bool wide_part(const NormPart& p) {
  return wide_rows(p.weight, 0, p.dtype) && wide_rows(p.bias, 0, p.dtype);
}

}  // namespace

hipError_t launch_norm(const NormArgs& args, hipStream_t stream) {
  NormArgs a = args;
  const bool wide = a.H % 8 == 0 && wide_rows(a.x, a.ldx, a.dtype) &&
                    wide_rows(a.residual, a.ldr, a.stream_dtype) && wide_rows(a.sum, a.lds, a.stream_dtype) &&
                    wide_rows(a.out, a.ldo, a.dtype) && wide_part(a.post) && wide_part(a.pre) &&
                    (a.gate_col == 0 || wide_rows(a.gate, a.gate_row, a.gate_dtype));
  const int vectors = (a.H + kF8Block - 1) / kF8Block * (kF8Block / 8);  // with those of a group's end
  const int v = vectors <= 256 ? 1 : vectors <= 1024 ? 2 : 4;
  a.threads = ((vectors + v - 1) / v + 63) / 64 * 64;
  const int rows = a.threads == 64 ? 4 : 1;
  // (A launch has fewer than 2^32 threads.)
  const int64_t most = (int64_t)1 << 20, blocks = (a.T + rows - 1) / rows;
  const dim3 grid((unsigned)(blocks < most ? blocks : most)), block(a.threads * rows);
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, a);
    return hipGetLastError();
  };
  if (v == 1) return wide ? run(norm_kernel<1, true>) : run(norm_kernel<1, false>);
  if (v == 2) return wide ? run(norm_kernel<2, true>) : run(norm_kernel<2, false>);
  return wide ? run(norm_kernel<4, true>) : run(norm_kernel<4, false>);
}

}  // namespace chord
