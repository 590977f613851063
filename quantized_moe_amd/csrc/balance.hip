// Balance of the router's choice: counts per expert, the balance loss
//
//   loss = sum over e of f(e) P(e),  f = E c / (k n),  P = mean over rows of p
//
// of each sequence, and its gradient g / n p (f - sum f p) [* (1 - sigmoid)], f
// constant.
//
// f - sum f p is taken of f - 1, as sum p = 1: near balance both are small there and
// nothing cancels.  No sum depends on an order that changes: counts are whole
// numbers, P is added per wave, wave by wave, and chunk by chunk.
#include <type_traits>

#include "device_common.h"

namespace chord {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr float kOff = -INFINITY;

__device__ __forceinline__ float wave_add(float x) {
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
  return x;
}
__device__ __forceinline__ float wave_top(float x) {
  for (int d = 1; d < 64; d <<= 1) x = fmaxf(x, __shfl_xor(x, d, 64));
  return x;
}
// As the router has it: -inf and NaN are not available, +inf is the largest number.
__device__ __forceinline__ float clamp_in(float x) {
  return x > kOff ? fminf(x, 3.402823466e38f) : kOff;
}

// Adds the slots first + [0, n) of a sequence's ids, n a multiple of k, to the counts
// in LDS.
__device__ __forceinline__ void count_slots(const BalanceArgs& a, const int32_t* ids, int64_t n, int32_t* counts,
                                            int32_t* tokens) {
  const int64_t rows = n / a.k;
  int real = 0;
  for (int64_t t = threadIdx.x; t < rows; t += kThreads) {
    bool any = false;
    for (int j = 0; j < a.k; ++j) {
      const uint32_t e = (uint32_t)ids[t * a.k + j];
      if (e < (uint32_t)a.E) {
        atomicAdd(&counts[e], 1);
        any = true;
      }
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
  count_slots(a, a.ids + ((int64_t)blockIdx.y * a.L + first) * a.k, mine * a.k, counts, &counts[a.E]);
  __syncthreads();
  int32_t* out = a.part_counts + ((int64_t)blockIdx.y * a.parts + blockIdx.x) * (a.E + 1);
  for (int e = threadIdx.x; e <= a.E; e += kThreads) out[e] = counts[e];
}

// The sum over chunks of P, and the loss, of a sequence.
__device__ __forceinline__ void finish(const BalanceArgs& a, int s, const float* part, int chunks,
                                       const int32_t* counts, int n, double* tmp) {
  const double inv = n > 0 ? 1.0 / n : 0.0;
  double loss = 0.0;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    double p = 0.0;
#pragma unroll 8
    for (int c = 0; c < chunks; ++c) p += part[(int64_t)c * a.E + e];
    p *= inv;
    a.probs[(int64_t)s * a.E + e] = (float)p;
    loss += p * counts[e];
  }
  for (int d = 1; d < 64; d <<= 1) loss += __shfl_xor(loss, d, 64);
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int w = 0; w < kWaves; ++w) t += tmp[w];
    a.loss[s] = (float)(t * a.E / a.k * inv);
  }
}

template <int V, bool SIGMOID>
__global__ __launch_bounds__(kThreads) void balance_rows(BalanceArgs a) {
  __shared__ int32_t counts[kMaxExperts + 1];
  __shared__ float sums[kWaves][V * 64];
  __shared__ double tmp[kWaves];
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
    count_slots(a, a.ids + row0 * a.k, a.L * a.k, counts, &counts[a.E]);
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
  for (int64_t t = first + wave; t < last; t += kWaves) {
    const int64_t row = row0 + t;
    bool any = false;
    for (int j = lane; j < a.k; j += 64) any |= (uint32_t)a.ids[row * a.k + j] < (uint32_t)a.E;
    const bool real = __builtin_amdgcn_ballot_w64(any) != 0;
    float* out = a.grad != nullptr ? a.grad + row * a.E : nullptr;
    float p[V], rest[V];
    if (real) {
      float l[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int64_t at = row * a.ld + min(i * 64 + lane, a.E - 1);
        float x;
        if (a.dtype == CHORD_DTYPE_F32) {
          x = static_cast<const float*>(a.logits)[at];
        } else {
          const uint16_t h = static_cast<const uint16_t*>(a.logits)[at];
          x = a.dtype == CHORD_DTYPE_BF16 ? bf16_to_f32(h) : (float)__builtin_bit_cast(_Float16, h);
        }
        l[i] = there[i] ? clamp_in(x) : kOff;
      }
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
      total = wave_add(total) + 1e-20f;
      float mean = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        p[i] /= total;
        sum[i] += p[i];
        mean += f[i] * p[i];
      }
      if (out != nullptr) {
        mean = wave_add(mean);
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
    if (only) sums[0][e] = t;  // (read by this thread alone until the barrier)
    else a.part_probs[((int64_t)s * a.chunks + chunk) * a.E + e] = t;
  }
  if (chunk == 0) {
    for (int e = threadIdx.x; e < a.E; e += kThreads) a.counts[(int64_t)s * a.E + e] = counts[e];
    if (threadIdx.x == 0) a.tokens[s] = n;
  }
  if (only) finish(a, s, sums[0], 1, counts, n, tmp);
}

__global__ __launch_bounds__(kThreads) void balance_finish(BalanceArgs a) {
  __shared__ double tmp[kWaves];
  const int s = blockIdx.x;
  finish(a, s, a.part_probs + (int64_t)s * a.chunks * a.E, a.chunks, a.counts + (int64_t)s * a.E, a.tokens[s],
         tmp);
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
  hipLaunchKernelGGL(balance_finish, dim3(a.n_seq), block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace chord
