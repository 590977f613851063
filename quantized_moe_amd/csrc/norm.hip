// Norms in front of and behind a block, with its gate, residual and residual scale:
//
//   u = x or N(x; post),  s = [residual +] scale [gate] u,  y = N(s; pre)
//   N(v; w, b) = (v - m) / sqrt(q + eps) (w + offset) + b
//
// A row lives in the registers of its threads from the one time it is read to the
// one time it is written, so the pass is bound by memory, whichever of the stages
// it has: 8192 rows of 7168 in bf16 with a residual (470 MB) take 84 us, 5.6 TB/s, where
// a copy reaches 5.1, with the vector units busy for 31 %; 4099 rows of 7112 between two
// layer norms with a gate and an fp32 stream (350 MB) 88 us, 4.0 TB/s, vector units 41 %.
// There the row's chain bounds it: two norms one after the other, each with sums over its
// waves and an exchange between them, and only the other workgroup's rows to fill the gaps.
// Below some 100 rows it is one row's chain alone: 4 us for one row, 8 with both norms.
#include <type_traits>

#include "f8_common.h"

namespace chord {
namespace {

constexpr int kMaxWaves = 16;
constexpr int kColumnsPerCu = 150 << 10;  // LDS for vectors of columns
constexpr float kShrink = 0x1p-96f;  // of rows whose squares overflow (2^128 2^-96 squared is far below)

// Eight neighbouring values as they lie in memory.  (Vectors that need no more than an
// element's alignment: the instruction is the same as for aligned ones.)
typedef uint32_t u32x4a2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4a4_t __attribute__((ext_vector_type(4), aligned(4)));
template <int DT>
struct Raw8 {
  u32x4_t lo;
};
template <>
struct Raw8<CHORD_DTYPE_F32> {
  u32x4_t lo, hi;
};

// n of the eight values at base[row + at], row being the same for all lanes (n >= 8: all; without TAIL that or none).
template <int DT, bool TAIL>
__device__ __forceinline__ Raw8<DT> load_raw(const void* base, int64_t row, uint32_t at, int n) {
  Raw8<DT> r{};
  if constexpr (DT == CHORD_DTYPE_F32) {
    const uint32_t* p = static_cast<const uint32_t*>(base) + row + at;
    if (n >= 8) {
      r.lo = *reinterpret_cast<const u32x4a4_t*>(p);
      r.hi = *reinterpret_cast<const u32x4a4_t*>(p + 4);
    } else if (TAIL) {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < n) (i < 4 ? r.lo : r.hi)[i & 3] = p[i];
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + row + at;
    if (n >= 8) {
      r.lo = *reinterpret_cast<const u32x4a2_t*>(p);
    } else if (TAIL) {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < n) r.lo[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
  }
  return r;
}
template <int DT>
__device__ __forceinline__ float raw_value(const Raw8<DT>& r, int i) {
  if constexpr (DT == CHORD_DTYPE_F32) return __uint_as_float(i < 4 ? r.lo[i] : r.hi[i & 3]);
  const uint32_t w = r.lo[i >> 1];
  if constexpr (DT == CHORD_DTYPE_BF16) return i & 1 ? __uint_as_float(w & 0xFFFF0000u) : bf16_to_f32(w);
  return (float)__builtin_bit_cast(half2_t, w)[i & 1];
}
template <int DT>
__device__ __forceinline__ float one_value(const void* base, int64_t at) {
  if constexpr (DT == CHORD_DTYPE_F32) return static_cast<const float*>(base)[at];
  const uint16_t h = static_cast<const uint16_t*>(base)[at];
  if constexpr (DT == CHORD_DTYPE_BF16) return bf16_to_f32(h);
  return (float)__builtin_bit_cast(_Float16, h);
}
template <int DT, bool TAIL>
__device__ __forceinline__ void store8(void* base, int64_t row, uint32_t at, int n, const float (&v)[8]) {
  if constexpr (DT == CHORD_DTYPE_F32) {
    float* p = static_cast<float*>(base) + row + at;
    if (n >= 8) {
      *reinterpret_cast<u32x4a4_t*>(p) = u32x4a4_t{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                                   __float_as_uint(v[3])};
      *reinterpret_cast<u32x4a4_t*>(p + 4) = u32x4a4_t{__float_as_uint(v[4]), __float_as_uint(v[5]),
                                                       __float_as_uint(v[6]), __float_as_uint(v[7])};
    } else if (TAIL) {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < n) p[i] = v[i];
    }
  } else {
    u32x4a2_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = DT == CHORD_DTYPE_BF16 ? pk_bf16(v[2 * i], v[2 * i + 1]) : pk_f16(v[2 * i], v[2 * i + 1]);
    uint16_t* p = static_cast<uint16_t*>(base) + row + at;
    if (n >= 8) {
      *reinterpret_cast<u32x4a2_t*>(p) = w;
    } else if (TAIL) {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
  }
}

// Sum over a wave, in every lane: neighbours 1, 2, 4 and 8 away inside the rows of 16
// lanes, then the four rows.
template <int CTRL>
__device__ __forceinline__ float add_step(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float wave_sum(float x) {
  x = add_step<0x118>(add_step<0x114>(add_step<0x112>(add_step<0x111>(x))));
  auto lane = [&](int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), l)); };
  return (lane(15) + lane(31)) + (lane(47) + lane(63));
}

// Sum over the first row of 16 lanes, in every lane.
__device__ __forceinline__ float first_lanes_sum(float x) {
  x = add_step<0x118>(add_step<0x114>(add_step<0x112>(add_step<0x111>(x))));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 15));
}

// Of e^-|g|, as e^-g leaves fp32 below -88, where the sigmoid is still there.  The
// exponential of what is not positive needs one limit (e^-104 is nothing; a NaN passes)
// where expf has two: with that 4096 rows of 7168 with a gate for each value take 66.5 us,
// with expf 68.3, with expf of e^-g 66.4.
__device__ __forceinline__ float sigmoid(float g) {
#pragma clang fp contract(off)  // (whole is the rounded product, rest what it leaves)
  constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0cp-26f;  // of log2 e
  const float x = fabsf(g) > 104.f ? -104.f : -fabsf(g);
  const float whole = x * kLog2e, n = rintf(whole);
  const float rest = __builtin_fmaf(x, kRest, __builtin_fmaf(x, kLog2e, -whole));
  const float e = ldexpf(__builtin_amdgcn_exp2f((whole - n) + rest), (int)n);
  return (g < 0.f ? e : 1.f) / (1.f + e);
}

// x where value j of a thread's eight is one of the row's (n of them are; without TAIL
// all or none), else 0: what stands behind a row is 0 and stays so.
template <bool TAIL>
__device__ __forceinline__ float only(float x, int n, int j) {
  return (TAIL ? j < n : n > 0) ? x : 0.f;
}

// Sums over the threads of a row: register moves inside a wave, LDS between waves.
// `slot` alternates, so one barrier is enough.
struct RowSum {
  float2 (*part)[kMaxWaves];
  int waves, slot;
  float own;    // values of this wave
  float count;  // ... of wave l in lane l

  // x and y of wave l come to lane l (zeros to the lanes behind the waves).
  __device__ __forceinline__ float2 share(float x, float y) {
    slot ^= 1;
    if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = make_float2(x, y);
    // (Fences of LDS alone: __syncthreads would wait for the next row as well.)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    const int lane = threadIdx.x & 63;
    return lane < waves ? part[slot][lane] : make_float2(0.f, 0.f);
  }
  // Sum of squares.
  template <int V>
  __device__ __forceinline__ float squares(const float (&v)[V][8]) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) t += v[i][j] * v[i][j];
    t = wave_sum(t);
    if (waves == 1) return t;
    return first_lanes_sum(share(t, 0.f).x);
  }
  // Mean, and sum of squares from it: of each wave from its own mean, which the
  // distance of that mean from the row's adds to.  (One barrier; nothing cancels.)
  template <int V, bool TAIL>
  __device__ __forceinline__ float spread(const float (&v)[V][8], const int (&n)[V], int H, float* mean) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) t += v[i][j];
    const float m = own > 0.f ? wave_sum(t) / own : 0.f;
    t = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = v[i][j] - only<TAIL>(m, n[i], j);
        t += d * d;
      }
    t = wave_sum(t);
    *mean = m;
    if (waves == 1) return t;
    const float2 p = share(m, t);
    const float centre = first_lanes_sum(p.x * count) / (float)H, d = p.x - centre;
    *mean = centre;
    return first_lanes_sum(p.y + count * d * d);
  }
};

// v (0 from column H on), less its mean (LAYER), times the factor that is returned is
// the norm without its weights.
template <int V, bool TAIL>
__device__ __forceinline__ float centre(float (&v)[V][8], const int (&n)[V], const NormPart& p, int H, RowSum& sum) {
  const bool layer = p.kind == CHORD_NORM_LAYER;
  float mean = 0.f, eps = p.eps;
  float total = layer ? sum.spread<V, TAIL>(v, n, H, &mean) : sum.squares<V>(v);
  if (!__builtin_isfinite(total + mean)) {
    // (Uniform over the row's threads.  A row with an infinity or NaN stays so in small
    // values, too.  A usual eps vanishes beside any row with squares of its own; a row of one
    // value has none, and its zeros stay zeros as long as what they are divided by is not.)
    eps = fmaxf(eps * kShrink * kShrink, 0x1p-126f);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= kShrink;
    total = layer ? sum.spread<V, TAIL>(v, n, H, &mean) : sum.squares<V>(v);
  }
  if (layer) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] -= only<TAIL>(mean, n[i], j);
  }
  return 1.f / sqrtf(total / (float)H + eps);
}

template <int WT, int V, bool TAIL>
__device__ __forceinline__ void load_row(const void* p, int64_t row, const int (&col)[V], const int (&n)[V],
                                         Raw8<WT> (&r)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) r[i] = load_raw<WT, TAIL>(p, row, col[i], n[i]);
}

// A vector of columns (weights, a bias, a gate) of type XT, or fp32 if `wide`, as every
// row needs it.  Each thread keeps its columns in LDS, where waiting for them does not
// wait for the next row; nobody else reads them, so no barrier is needed.
template <int XT, int V, bool TAIL>
struct Columns {
  const void* p;
  bool wide;
  uint8_t* kept;  // 16-byte pieces, this thread's `step` apart; or null: read again every time
  int step;

  __device__ __forceinline__ static int bytes(bool wide, int threads) { return V * (wide ? 32 : 16) * threads; }
  // Takes its place at *at.
  __device__ __forceinline__ void keep(const void* ptr, int dtype, uint8_t** at, int threads, int tid,
                                       const int (&col)[V], const int (&n)[V]) {
    p = ptr;
    wide = XT == CHORD_DTYPE_F32 || dtype == CHORD_DTYPE_F32;
    kept = nullptr;
    if (p == nullptr || *at == nullptr) return;
    kept = *at + tid * 16;
    step = threads * 16;
    *at += bytes(wide, threads);
    u32x4_t* to = reinterpret_cast<u32x4_t*>(kept);
    const int s = threads;
    if (wide) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const auto r = load_raw<CHORD_DTYPE_F32, TAIL>(p, 0, col[i], n[i]);
        to[(2 * i) * s] = r.lo;
        to[(2 * i + 1) * s] = r.hi;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) to[i * s] = load_raw<XT, TAIL>(p, 0, col[i], n[i]).lo;
    }
  }
  // f(i, j, value) for value j of vector i, of row `row` where the vector has rows.
  template <typename F>
  __device__ __forceinline__ void each(int64_t row, const int (&col)[V], const int (&n)[V], F f) const {
    if (wide) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        Raw8<CHORD_DTYPE_F32> r;
        if (kept != nullptr) {
          r.lo = *reinterpret_cast<const u32x4_t*>(kept + (2 * i) * step);
          r.hi = *reinterpret_cast<const u32x4_t*>(kept + (2 * i + 1) * step);
        } else {
          r = load_raw<CHORD_DTYPE_F32, TAIL>(p, row, col[i], n[i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) f(i, j, raw_value<CHORD_DTYPE_F32>(r, j));
      }
    } else if constexpr (XT != CHORD_DTYPE_F32) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        Raw8<XT> r;
        if (kept != nullptr) r.lo = *reinterpret_cast<const u32x4_t*>(kept + i * step);
        else r = load_raw<XT, TAIL>(p, row, col[i], n[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) f(i, j, raw_value<XT>(r, j));
      }
    }
  }
};

// XT: type of x, out, and (unless fp32) of weights and gate; ST: of residual and sum.
// The threads of a row hold V times 8 neighbouring values each; a workgroup has a row
// at a time, or one a wave where a wave is enough.  The next row is on its way while
// one is worked on.
// FULL: with a norm behind the block, a gate or a bias; else the weights stay in
// registers from row to row.  TAIL: H is no multiple of 8.
template <int XT, int ST, int V, bool FULL, bool TAIL>
__global__ __launch_bounds__(1024, TAIL && V == 1 && !FULL ? 8 : 4) void norm_kernel(NormArgs a) {
  __shared__ float2 part[2][kMaxWaves];
  extern __shared__ __attribute__((aligned(16))) uint8_t columns[];
  const bool alone = a.threads > 64;  // ... in its workgroup
  const int tid = alone ? threadIdx.x : threadIdx.x & 63;
  int col[V], n[V], held = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    col[i] = (i * a.threads + tid) * 8;
    n[i] = min(8, a.H - col[i]);
    held += max(n[i], 0);
  }
  RowSum sum{part, alone ? a.threads >> 6 : 1, 0, wave_sum((float)held), 0.f};
  if (alone) sum.count = sum.share(sum.own, 0.f).x;
  auto gated = [&](float g) { return a.gate_sigmoid ? sigmoid(g) : g; };
  // (Whole waves leave, where a wave has a row; else the workgroup's rows are there
  // for all of its waves.)
  const uint32_t of = alone ? 1 : blockDim.x >> 6, mine = alone ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t step = (int64_t)gridDim.x * of;
  int64_t t = (int64_t)blockIdx.x * of + mine;
  if (t >= a.T) return;
  Raw8<XT> x[V];
  Raw8<ST> r[V];
  auto load_x = [&](int64_t row) { load_row<XT, V, TAIL>(a.x, row * a.ldx, col, n, x); };
  auto load_r = [&](int64_t row) {
    if (a.residual != nullptr) load_row<ST, V, TAIL>(a.residual, row * a.ldr, col, n, r);
  };
#pragma unroll
  for (int i = 0; i < V; ++i) r[i] = Raw8<ST>{};
  load_x(t);
  load_r(t);
  typedef Columns<XT, V, TAIL> Vector;
  Vector pre_w, pre_b, post_w, post_b, gate;
  float pre[V][8];
  if (FULL) {
    uint8_t* at = a.columns ? columns + (threadIdx.x - tid) * (a.columns_bytes / a.threads) : nullptr;
    pre_w.keep(a.pre.weight, a.pre.dtype, &at, a.threads, tid, col, n);
    pre_b.keep(a.pre.bias, a.pre.dtype, &at, a.threads, tid, col, n);
    post_w.keep(a.post.weight, a.post.dtype, &at, a.threads, tid, col, n);
    post_b.keep(a.post.bias, a.post.dtype, &at, a.threads, tid, col, n);
    uint8_t* none = nullptr;  // (a gate for each value is read with its row)
    gate.keep(a.gate_col != 0 ? a.gate : nullptr, a.gate_dtype, a.gate_row == 0 ? &at : &none, a.threads, tid, col, n);
  } else if (a.pre.weight != nullptr) {
    uint8_t* none = nullptr;
    pre_w.keep(a.pre.weight, a.pre.dtype, &none, a.threads, tid, col, n);
    pre_w.each(0, col, n, [&](int i, int j, float w) { pre[i][j] = w + a.pre.offset; });
  }
  for (; t < a.T; t += step) {
    float v[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = raw_value<XT>(x[i], j);
    const bool more = t + step < a.T;
    if (more) load_x(t + step);
    auto norm = [&](const NormPart& p, const Vector& w, const Vector& b) {
      const float inv = centre<V, TAIL>(v, n, p, a.H, sum);
      w.each(0, col, n, [&](int i, int j, float f) { v[i][j] = v[i][j] * inv * (f + p.offset); });
      if (p.bias != nullptr) b.each(0, col, n, [&](int i, int j, float f) { v[i][j] += f; });
    };
    if (FULL && a.post.weight != nullptr) norm(a.post, post_w, post_b);
    if (FULL && a.gate != nullptr) {
      const int64_t row = t * a.gate_row;
      if (a.gate_col == 0) {
        // (Before the scale: the product of the two may leave fp32 where what they make of
        // the value does not.)
        const float g = gated(a.gate_dtype == CHORD_DTYPE_F32 ? one_value<CHORD_DTYPE_F32>(a.gate, row)
                                                              : one_value<XT>(a.gate, row));
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] *= g;
      } else {
        gate.each(row, col, n, [&](int i, int j, float g) { v[i][j] *= gated(g); });
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = __builtin_fmaf(v[i][j], a.scale, raw_value<ST>(r[i], j));
    if (more) load_r(t + step);
    if (a.sum != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i) store8<ST, TAIL>(a.sum, t * a.lds, col[i], n[i], v[i]);
    }
    if (a.pre.weight == nullptr) continue;
    if (FULL) {
      norm(a.pre, pre_w, pre_b);
    } else {
      const float inv = centre<V, TAIL>(v, n, a.pre, a.H, sum);
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * inv * pre[i][j];
    }
    if (a.out != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i) store8<XT, TAIL>(a.out, t * a.ldo, col[i], n[i], v[i]);
    }
    if (a.codes != nullptr) {  // 16 lanes hold a group (by all of them)
      const int groups = (a.H + kF8Block - 1) / kF8Block;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
        const F8Group q = f8_group(row_max16(m));
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = q.inv != 0.f ? f8_value(q, v[i][j]) : 0.f;
        if (col[i] < groups * kF8Block) {
          uint2 o;
          o.x = f8_pack4(v[i][0], v[i][1], v[i][2], v[i][3]);
          o.y = f8_pack4(v[i][4], v[i][5], v[i][6], v[i][7]);
          *reinterpret_cast<uint2*>(a.codes + t * groups * kF8Block + (uint32_t)col[i]) = o;
          if ((tid & 15) == 0) (a.code_scales + t * groups)[(uint32_t)col[i] / kF8Block] = q.scale;
        }
      }
    }
  }
}

template <int XT, int ST>
hipError_t launch(const NormArgs& args, hipStream_t stream) {
  NormArgs a = args;
  const bool full = a.post.weight != nullptr || a.gate != nullptr || a.pre.bias != nullptr;
  const int vectors = (a.H + kF8Block - 1) / kF8Block * (kF8Block / 8);  // with those of a group's end
  // Values a thread: 8 up to H = 8192 (with the stages of FULL 4096, whose registers
  // leave one such workgroup a CU), as long as a workgroup's threads reach.  us, 8 / 16 a
  // thread: 8192 x 7168 85 / 90, with a norm behind the block 107 / 89, both of means and an
  // fp32 stream at 4099 x 7112 100 / 86.
  const int v = vectors <= (full ? 512 : 1024) ? 1 : vectors <= 2048 ? 2 : 4;
  a.threads = ((vectors + v - 1) / v + 63) / 64 * 64;
  const int rows = a.threads == 64 ? 4 : 1;
  // 16 waves a CU, the next row of each on its way (32 where rows end inside a vector:
  // their loads take longer), and every workgroup as many rows as the others.  us, 16 /
  // 32 waves: 8192 x 7168 85 / 89, 8191 x 7110 155 / 117.  (A workgroup a row without a
  // next one: 134.)
  const bool tail = a.H % 8 != 0;
  const int waves = a.threads * rows / 64, fit = (tail && v == 1 && !full ? 32 : 16) / waves;
  const int64_t most = (int64_t)a.num_cus * (fit > 1 ? fit : 1), blocks = (a.T + rows - 1) / rows;
  const int64_t each = (blocks + most - 1) / most;
  const dim3 grid((unsigned)((blocks + each - 1) / each)), block(a.threads * rows);
  // What each row of a workgroup keeps in LDS, if a CU's workgroups have room for it.
  size_t lds = 0;
  if (full) {
    auto bytes = [&](const void* p, int dtype) {
      return p == nullptr ? 0 : v * (dtype == CHORD_DTYPE_F32 ? 32 : 16) * a.threads;
    };
    a.columns_bytes = bytes(a.pre.weight, a.pre.dtype) + bytes(a.pre.bias, a.pre.dtype) +
                      bytes(a.post.weight, a.post.dtype) + bytes(a.post.bias, a.post.dtype) +
                      (a.gate_col != 0 && a.gate_row == 0 ? bytes(a.gate, a.gate_dtype) : 0);
    a.columns = (int64_t)a.columns_bytes * rows * (fit > 1 ? fit : 1) <= kColumnsPerCu;
    if (a.columns) lds = (size_t)a.columns_bytes * rows;
  }
  auto run = [&](auto full, auto tail) {
    constexpr bool F = decltype(full)::value, L = decltype(tail)::value;
    auto go = [&](auto kernel) {
      if (lds > 0) {  // (the same limit in every call: calls of several threads set it at once)
        const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                                 kColumnsPerCu);
        if (e != hipSuccess) return e;
      }
      hipLaunchKernelGGL(kernel, grid, block, lds, stream, a);
      return hipGetLastError();
    };
    return v == 1 ? go(norm_kernel<XT, ST, 1, F, L>) : v == 2 ? go(norm_kernel<XT, ST, 2, F, L>) : go(norm_kernel<XT, ST, 4, F, L>);
  };
  const std::true_type yes{};
  const std::false_type no{};
  if (tail) return full ? run(yes, yes) : run(no, yes);
  return full ? run(yes, no) : run(no, no);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  constexpr int F32 = CHORD_DTYPE_F32, BF16 = CHORD_DTYPE_BF16, F16 = CHORD_DTYPE_F16;
  if (a.dtype == F32) return launch<F32, F32>(a, stream);
  if (a.dtype == BF16) return a.stream_dtype == F32 ? launch<BF16, F32>(a, stream) : launch<BF16, BF16>(a, stream);
  return a.stream_dtype == F32 ? launch<F16, F32>(a, stream) : launch<F16, F16>(a, stream);
}

}  // namespace chord
