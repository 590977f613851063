// Balance of the router's choice: counts per expert, the balance loss
//
//   loss = sum over e of f(e) P(e),  f = E c / (k n),  P = mean over rows of p
//
// of each sequence, and its gradient g / n p (f - sum f p) [* (1 - sigmoid)], f
// constant.
//
// f - sum f p is taken as (f - 1) - sum (f - 1) p + (1 - sum p): near balance all of these
// are small and nothing cancels.  The last is 0 for a softmax and 1e-20 / (sum + 1e-20)
// for sigmoids, which counts where a row's are all small (from logits of -36 on with
// eight experts).  No sum depends on an order that changes: counts are whole
// numbers, P is added per wave, wave by wave, and chunk by chunk.
//
// 8192 rows of 384 with the gradient (25 MB, 5.0 us at a copy's rate) take 15.4 us for the
// rows, with the scores once, and 4.4 for the join of P.  A wave takes a row at a time and
// four in all, two waves a SIMD, so a row's chain (a maximum and two sums over the wave, an
// exponential between) waits with little beside it.  One sequence of 8192 rows takes 26.6:
// its join is one workgroup over 256 chunks.  64 rows of 256 are one workgroup and one
// launch, eight rows a wave: 14.6 us.
#include <type_traits>

#include "device_common.h"

namespace chord {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kFinishThreads = 1024;
constexpr float kOff = -INFINITY;

// Over a wave, in every lane: neighbours 1, 2, 4 and 8 away inside the rows of 16
// lanes (a lane without one keeps its own), then the four rows' last lanes.
template <int CTRL, typename F>
__device__ __forceinline__ float with_neighbour(float x, float none, F f) {
  return f(x, __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(none), __float_as_int(x), CTRL, 0xF, 0xF, false)));
}
template <typename F>
__device__ __forceinline__ float over_wave(float x, float none, F f) {
  x = with_neighbour<0x111>(x, none, f);
  x = with_neighbour<0x112>(x, none, f);
  x = with_neighbour<0x114>(x, none, f);
  x = with_neighbour<0x118>(x, none, f);
  auto lane = [&](int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), l)); };
  return f(f(lane(15), lane(31)), f(lane(47), lane(63)));
}
__device__ __forceinline__ float wave_add(float x) {
  return over_wave(x, 0.f, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_top(float x) {
  return over_wave(x, kOff, [](float a, float b) { return fmaxf(a, b); });
}
// As the router has it: -inf and NaN are not available, +inf is the largest number.
__device__ __forceinline__ float clamp_in(float x) {
  return x > kOff ? fminf(x, 3.402823466e38f) : kOff;
}

// Adds the slots of `rows` rows of ids to the counts in LDS, and the rows with an expert
// to *tokens.
__device__ __forceinline__ void count_slots(const BalanceArgs& a, const int32_t* ids, int64_t rows, int32_t* counts,
                                            int32_t* tokens) {
  auto slot = [&](int id) {
    const bool in = (uint32_t)id < (uint32_t)a.E;
    if (in) atomicAdd(&counts[id], 1);
    return in;
  };
  const bool fours = a.k % 4 == 0 && reinterpret_cast<uintptr_t>(ids) % 16 == 0;
  int real = 0;
#pragma unroll 2
  for (int64_t t = threadIdx.x; t < rows; t += kThreads) {
    bool any = false;
    if (fours) {
      const int4* p = reinterpret_cast<const int4*>(ids + t * a.k);
#pragma unroll 2
      for (int j = 0; j < a.k / 4; ++j) {
        const int4 v = p[j];
        any |= slot(v.x);
        any |= slot(v.y);
        any |= slot(v.z);
        any |= slot(v.w);
      }
    } else {
      for (int j = 0; j < a.k; ++j) any |= slot(ids[t * a.k + j]);
    }
    real += any ? 1 : 0;
  }
  if (real > 0) atomicAdd(tokens, real);
}

// Counts of part `blockIdx.x` of sequence `blockIdx.y`.
__global__ __launch_bounds__(kThreads) void balance_count(BalanceArgs a) {
  __shared__ int32_t counts[kMaxExperts + 1];
  for (int e = threadIdx.x; e <= a.E; e += kThreads) counts[e] = 0;
  __syncthreads();
  const int64_t rows = (a.L + a.parts - 1) / a.parts, first = min(a.L, rows * blockIdx.x);
  const int64_t mine = min(rows, a.L - first);
  count_slots(a, a.ids + ((int64_t)blockIdx.y * a.L + first) * a.k, mine, counts, &counts[a.E]);
  __syncthreads();
  int32_t* out = a.part_counts + ((int64_t)blockIdx.y * a.parts + blockIdx.x) * (a.E + 1);
  for (int e = threadIdx.x; e <= a.E; e += kThreads) out[e] = counts[e];
}

// The sum over chunks of P, and the loss, of a sequence, by THREADS threads.  They
// take an expert each; where there are enough for several of each, those share the
// chunks.
template <int THREADS>
__device__ __forceinline__ void finish(const BalanceArgs& a, int s, const float* part, int chunks,
                                       const int32_t* counts, int n, double* tmp) {
  const int wide = (a.E + 63) / 64 * 64, groups = THREADS / wide > 0 ? THREADS / wide : 1;
  const int group = threadIdx.x / wide, me = threadIdx.x % wide;
  const int c0 = chunks * group / groups, c1 = chunks * (group + 1) / groups;
  const double inv = n > 0 ? 1.0 / n : 0.0;
  double loss = 0.0;
  for (int e0 = 0; e0 < a.E; e0 += THREADS) {  // (once, but for E over THREADS)
    const int e = e0 + me;
    double p = 0.0;
    if (group < groups && e < a.E) {
#pragma unroll 8
      for (int c = c0; c < c1; ++c) p += part[(int64_t)c * a.E + e];
    }
    if (groups > 1) {
      if (group < groups) tmp[group * wide + me] = p;
      __syncthreads();
      if (group == 0)
        for (int g = 1; g < groups; ++g) p += tmp[g * wide + me];
      __syncthreads();
    }
    if (group == 0 && e < a.E) {
      p *= inv;
      a.probs[(int64_t)s * a.E + e] = (float)p;
      loss += p * counts[e];
    }
  }
  for (int d = 1; d < 64; d <<= 1) loss += __shfl_xor(loss, d, 64);
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int w = 0; w < THREADS / 64; ++w) t += tmp[w];
    a.loss[s] = (float)(t * a.E / a.k * inv);
  }
}

template <int V, bool SIGMOID>
__global__ __launch_bounds__(kThreads) void balance_rows(BalanceArgs a) {
  __shared__ int32_t counts[kMaxExperts + 1];
  __shared__ float sums[kWaves][V * 64];
  __shared__ double tmp[kThreads];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int s = blockIdx.y, chunk = blockIdx.x;
  const int64_t row0 = (int64_t)s * a.L;
  for (int e = threadIdx.x; e <= a.E; e += kThreads) {
    int c = 0;
    for (int p = 0; p < a.parts; ++p) c += a.part_counts[((int64_t)s * a.parts + p) * (a.E + 1) + e];
    counts[e] = c;
  }
  __syncthreads();
  if (a.parts == 0) {
    count_slots(a, a.ids + row0 * a.k, a.L, counts, &counts[a.E]);
    __syncthreads();
  }
  const int n = counts[a.E];
  const float unit = n > 0 ? (float)((double)a.E / ((double)a.k * n)) : 0.f;
  const float g = n > 0 ? (a.grad_loss != nullptr ? a.grad_loss[s] : 1.f) / (float)n : 0.f;
  float f[V], sum[V];
  bool there[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 64 + lane;
    there[i] = e < a.E && (a.bias == nullptr || a.bias[min(e, a.E - 1)] > kOff);
    f[i] = e < a.E ? unit * (float)counts[e] - 1.f : 0.f;
    sum[i] = 0.f;
  }
  const int64_t first = chunk * a.rows, last = min(a.L, first + a.rows);
  // A row's logits and first 64 ids, one row ahead.
  float raw[V];
  int id = -1;
  auto load = [&](int64_t t) {
    const int64_t row = row0 + t;
    id = lane < a.k ? a.ids[row * a.k + lane] : -1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t at = row * a.ld + min(i * 64 + lane, a.E - 1);
      if (a.dtype == CHORD_DTYPE_F32) raw[i] = static_cast<const float*>(a.logits)[at];
      else raw[i] = __uint_as_float(static_cast<const uint16_t*>(a.logits)[at]);
    }
  };
  int64_t t = first + __builtin_amdgcn_readfirstlane(wave);
  if (t < last) load(t);
  for (; t < last; t += kWaves) {
    const int64_t row = row0 + t;
    bool any = (uint32_t)id < (uint32_t)a.E;
    for (int j = lane + 64; j < a.k; j += 64) any |= (uint32_t)a.ids[row * a.k + j] < (uint32_t)a.E;
    const bool real = __builtin_amdgcn_ballot_w64(any) != 0;
    float* out = a.grad != nullptr ? a.grad + row * a.E : nullptr;
    float l[V], p[V], rest[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t h = __float_as_uint(raw[i]);
      const float x = a.dtype == CHORD_DTYPE_F32 ? raw[i]
                      : a.dtype == CHORD_DTYPE_BF16 ? bf16_to_f32(h) : (float)__builtin_bit_cast(_Float16, (uint16_t)h);
      l[i] = there[i] ? clamp_in(x) : kOff;
    }
    if (t + kWaves < last) load(t + kWaves);
    if (real) {
      float top = 0.f;
      if (!SIGMOID) {
        top = l[0];
#pragma unroll
        for (int i = 1; i < V; ++i) top = fmaxf(top, l[i]);
        top = wave_top(top);
      }
      float total = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        rest[i] = 1.f;
        if (SIGMOID) {
          const float u = expf(-fabsf(l[i])), d = 1.f / (1.f + u);
          p[i] = l[i] > 0.f ? d : u * d;
          rest[i] = l[i] > 0.f ? u * d : d;
        } else {
          p[i] = expf(l[i] - top);
        }
        p[i] = l[i] > kOff ? p[i] : 0.f;
        total += p[i];
      }
      const float inv = 1.f / (wave_add(total) + 1e-20f);
      float mean = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        p[i] *= inv;
        sum[i] += p[i];
        mean += f[i] * p[i];
      }
      if (out != nullptr) {
        mean = wave_add(mean);
        if (SIGMOID) mean -= 1e-20f * inv;  // (1 - sum p)
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i * 64 + lane < a.E) out[i * 64 + lane] = g * p[i] * (f[i] - mean) * rest[i];
      }
    } else if (out != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i * 64 + lane < a.E) out[i * 64 + lane] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) sums[wave][i * 64 + lane] = sum[i];
  __syncthreads();
  const bool only = a.chunks == 1;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    float t = sums[0][e];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) t += sums[w][e];
    if (only) sums[0][e] = t;  // (no other thread reads it before the barrier)
    else a.part_probs[((int64_t)s * a.chunks + chunk) * a.E + e] = t;
  }
  if (chunk == 0) {
    for (int e = threadIdx.x; e < a.E; e += kThreads) a.counts[(int64_t)s * a.E + e] = counts[e];
    if (threadIdx.x == 0) a.tokens[s] = n;
  }
  if (only) {
    __syncthreads();  // (where threads share an expert's chunks, another one takes the sum)
    finish<kThreads>(a, s, sums[0], 1, counts, n, tmp);
  }
}

__global__ __launch_bounds__(kFinishThreads) void balance_finish(BalanceArgs a) {
  __shared__ double tmp[kFinishThreads];
  const int s = blockIdx.x;
  finish<kFinishThreads>(a, s, a.part_probs + (int64_t)s * a.chunks * a.E, a.chunks, a.counts + (int64_t)s * a.E,
                         a.tokens[s], tmp);
}

}  // namespace

hipError_t launch_balance(const BalanceArgs& a, hipStream_t stream) {
  const dim3 block(kThreads);
  if (a.parts > 0) {
    hipLaunchKernelGGL(balance_count, dim3(a.parts, a.n_seq), block, 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid(a.chunks, a.n_seq);
  const int v = (a.E + 63) / 64;
  auto rows = [&](auto sigmoid) {
    constexpr bool S = decltype(sigmoid)::value;
    if (v <= 1) hipLaunchKernelGGL((balance_rows<1, S>), grid, block, 0, stream, a);
    else if (v <= 2) hipLaunchKernelGGL((balance_rows<2, S>), grid, block, 0, stream, a);
    else if (v <= 4) hipLaunchKernelGGL((balance_rows<4, S>), grid, block, 0, stream, a);
    else if (v <= 6) hipLaunchKernelGGL((balance_rows<6, S>), grid, block, 0, stream, a);
    else if (v <= 8) hipLaunchKernelGGL((balance_rows<8, S>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((balance_rows<16, S>), grid, block, 0, stream, a);
    return hipGetLastError();
  };
  const hipError_t e = a.sigmoid ? rows(std::true_type{}) : rows(std::false_type{});
  if (e != hipSuccess || a.chunks == 1) return e;
  hipLaunchKernelGGL(balance_finish, dim3(a.n_seq), dim3(kFinishThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace chord
