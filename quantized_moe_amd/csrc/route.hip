// Router: the k experts of every token and their weights from router logits.
//
//   score(e)  = softmax or sigmoid of the logits
//   choice(e) = score(e) + bias(e)
//   of E / n_group experts per group, only the topk_group groups with the best
//   group score stay (the sum of a group's two best choices with a bias, its
//   best choice without)
//   ids = the k best choices, descending, ties to the lowest expert
//   weight = score of the chosen (/ their sum + 1e-20) * scaling
//
// One wave per token; lane l holds experts l, l + 64, ... in registers, so the
// logits are read once and nothing is staged.  The result has to be the order
// of the real numbers, not of their 32-bit approximations: among 384 scores
// two neighbours of the order differ by less than the 32-bit error about once
// in a few thousand tokens.
//
//   * Without a bias both scores rise with the logit, so the logits themselves
//     are compared: exact in 32 bits.
//   * With a bias the keys are 32-bit choices with a known error.  The rounds
//     go on past the k-th best while the next key is within that error
//     (usually no further round), the candidates move to one lane each, and a
//     single 64-bit evaluation in all lanes at once orders them.
//   * Group scores whose border is closer than the error, or more than 64
//     candidates, take the 64-bit path for the whole token (`exact`).
#include "device_common.h"

namespace chord {
namespace {

constexpr int kWavesPerBlock = 4;
constexpr float kOff = -INFINITY;  // key and logit of an expert that cannot be chosen
// Error of a 32-bit choice: score within 3e-7 (hardware exp2 and reciprocal),
// one rounding of the sum.  Twice that for a difference, with room to spare.
constexpr float kErrAbs = 2e-6f, kErrRel = 1e-6f;

template <int CTRL>
__device__ __forceinline__ float dpp(float x, float identity, int rows) {
  const int o = __builtin_bit_cast(int, identity), s = __builtin_bit_cast(int, x);
  return __builtin_bit_cast(float, rows == 0xF ? __builtin_amdgcn_update_dpp(o, s, CTRL, 0xF, 0xF, false)
                                   : rows == 0xA ? __builtin_amdgcn_update_dpp(o, s, CTRL, 0xA, 0xF, false)
                                                 : __builtin_amdgcn_update_dpp(o, s, CTRL, 0xC, 0xF, false));
}
__device__ __forceinline__ float lane_f(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

// Reductions over the wave; the result is uniform.  Lanes of a row of 16 add
// their neighbours 1, 2, 4 and 8 places away, then the rows join.
__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, dpp<0x111>(x, kOff, 0xF));
  x = fmaxf(x, dpp<0x112>(x, kOff, 0xF));
  x = fmaxf(x, dpp<0x114>(x, kOff, 0xF));
  x = fmaxf(x, dpp<0x118>(x, kOff, 0xF));
  x = fmaxf(x, dpp<0x142>(x, kOff, 0xA));
  x = fmaxf(x, dpp<0x143>(x, kOff, 0xC));
  return lane_f(x, 63);
}
__device__ __forceinline__ float wave_sum(float x) {
  x += dpp<0x111>(x, 0.f, 0xF);
  x += dpp<0x112>(x, 0.f, 0xF);
  x += dpp<0x114>(x, 0.f, 0xF);
  x += dpp<0x118>(x, 0.f, 0xF);
  x += dpp<0x142>(x, 0.f, 0xA);
  x += dpp<0x143>(x, 0.f, 0xC);
  return lane_f(x, 63);
}
__device__ __forceinline__ double wave_max(double x) {
  for (int d = 1; d < 64; d <<= 1) x = fmax(x, __shfl_xor(x, d, 64));
  return x;
}
__device__ __forceinline__ double wave_sum(double x) {
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
  return x;
}
__device__ __forceinline__ int wave_min(int x) {
  for (int d = 1; d < 64; d <<= 1) x = min(x, __shfl_xor(x, d, 64));
  return __builtin_amdgcn_readfirstlane(x);
}
__device__ __forceinline__ float lane_of(float x, int lane) { return lane_f(x, lane); }
__device__ __forceinline__ double lane_of(double x, int lane) { return __shfl(x, lane, 64); }

// The best key left, and the lowest expert that has it.  Returns -inf if none
// is left.
template <int V, typename F>
__device__ __forceinline__ F best_left(const F (&key)[V], int lane, int* expert) {
  F lm = key[V - 1];
  int li = V - 1;
#pragma unroll
  for (int i = V - 2; i >= 0; --i) {
    const bool up = key[i] >= lm;  // >=: the lowest of equal keys
    lm = up ? key[i] : lm;
    li = up ? i : li;
  }
  const F m = wave_max(lm);
  const uint64_t has = __builtin_amdgcn_ballot_w64(lm == m);
  const int mine = li * 64 + lane;
  if (__builtin_popcountll(has) == 1)
    *expert = __builtin_amdgcn_readlane(mine, __builtin_ctzll(has));
  else
    *expert = wave_min(lm == m ? mine : INT32_MAX);
  return m;
}

template <int V, typename F>
__device__ __forceinline__ void drop(F (&key)[V], int lane, int expert) {
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = i * 64 + lane == expert ? (F)kOff : key[i];
}

// Sets the keys of all groups but the topk_group best to -inf.  Lane g holds
// the score of group g.  False if the border between the last group that stays
// and the first that goes is within the error of 32-bit keys (`approx`).
template <int V, typename F>
__device__ __forceinline__ bool keep_groups(F (&key)[V], const int (&grp)[V], const RouteArgs& a,
                                            int lane, bool approx) {
  const int G = a.n_group;
  F mine = (F)kOff;
  F size = 0;  // magnitude of the two summands
  for (int g = 0; g < G; ++g) {
    F t1 = (F)kOff, t2 = (F)kOff;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const F v = grp[i] == g ? key[i] : (F)kOff;
      t2 = v > t1 ? t1 : (v > t2 ? v : t2);
      t1 = v > t1 ? v : t1;
    }
    // The two best over the wave: the best, then the best without one copy of
    // it (if two lanes hold it, it is also the second).
    const F m1 = wave_max(t1);
    const uint64_t has = __builtin_amdgcn_ballot_w64(t1 == m1);
    const int first = __builtin_ctzll(has);
    const F m2 = wave_max(lane == first ? t2 : t1);
    if (lane == g) {
      const bool two = a.bias != nullptr && m2 > (F)kOff;
      mine = two ? m1 + m2 : m1;
      size = m1 > (F)kOff ? fabs(m1) + (two ? fabs(m2) : (F)0) : (F)0;
    }
  }
  int rank = 0;
  for (int g = 0; g < G; ++g) {
    const F o = lane_of(mine, g);
    rank += (o > mine || (o == mine && g < lane)) ? 1 : 0;
  }
  const uint64_t keep = __builtin_amdgcn_ballot_w64(lane < G && rank < a.topk_group);
  if (approx) {
    const uint64_t last = __builtin_amdgcn_ballot_w64(lane < G && rank == a.topk_group - 1);
    const uint64_t next = __builtin_amdgcn_ballot_w64(lane < G && rank == a.topk_group);
    const F gap = lane_of(mine, __builtin_ctzll(last)) - lane_of(mine, __builtin_ctzll(next));
    // (negated: a NaN gap, from groups without any expert, counts as close)
    if (!(gap > (F)(2 * kErrAbs) + (F)kErrRel * wave_max(size))) return false;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = (keep >> grp[i]) & 1 ? key[i] : (F)kOff;
  return true;
}

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t i) {
  if (a.dtype == CHORD_DTYPE_F32) return static_cast<const float*>(a.logits)[i];
  const uint16_t h = static_cast<const uint16_t*>(a.logits)[i];
  if (a.dtype == CHORD_DTYPE_BF16) return bf16_to_f32(h);
  return (float)__builtin_bit_cast(_Float16, h);
}
// -inf and NaN: not available.  +inf counts as the largest finite number.
__device__ __forceinline__ float clamp_in(float x) {
  return x > kOff ? fminf(x, 3.402823466e38f) : kOff;
}

template <int V>
__global__ __launch_bounds__(64 * kWavesPerBlock) void route_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int t = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * kWavesPerBlock + (threadIdx.x >> 6)));
  if (t >= a.T) return;
  const int64_t row = (int64_t)t * a.ld;
  const bool biased = a.bias != nullptr;
  float l[V], b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 64 + lane;
    l[i] = e < a.E ? load_logit(a, row + e) : kOff;
    b[i] = biased && e < a.E ? a.bias[e] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    l[i] = b[i] > kOff ? clamp_in(l[i]) : kOff;
    b[i] = clamp_in(b[i]);
  }
  // softmax: maximum and sum (64 bits where the sum decides an order)
  float top = 0.f;
  double total = 1.0;
  if (!a.sigmoid) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
    top = wave_max(m);
    if (!(top > kOff)) top = 0.f;  // no expert: every term below is 0
    if (biased) {
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) s += l[i] > kOff ? exp((double)l[i] - (double)top) : 0.0;
      total = wave_sum(s);
    } else {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) s += l[i] > kOff ? expf(l[i] - top) : 0.f;
      total = wave_sum(s);
    }
  }
  auto score64 = [&](float x) {
    return a.sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)top) / total;
  };
  const bool grouped = a.topk_group < a.n_group;
  int grp[V];
  if (grouped) {
#pragma unroll
    for (int i = 0; i < V; ++i) grp[i] = (int)(((uint32_t)(i * 64 + lane) * a.group_magic) >> 20) & 63;
  }

  // The candidates, one a lane: expert and (if biased) 64-bit choice.
  int cand = -1, n = 0;
  bool done = true;
  {
    float key[V];
    if (biased) {
      const float inv = (float)(1.0 / total);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float s = a.sigmoid ? __builtin_amdgcn_rcpf(1.f + __expf(-l[i])) : __expf(l[i] - top) * inv;
        key[i] = l[i] > kOff ? s + b[i] : kOff;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = l[i];
    }
    if (grouped) done = keep_groups<V, float>(key, grp, a, lane, biased);
    float kth = kOff;
    while (done) {
      if (n >= a.k && !biased) break;
      int e;
      const float m = best_left<V, float>(key, lane, &e);
      if (!(m > kOff) || (n >= a.k && m < kth - (kErrAbs + kErrRel * fabsf(kth)))) break;
      if (n == 64) done = false;
      if (lane == n) cand = e;
      if (++n == a.k) kth = m;
      drop<V, float>(key, lane, e);
    }
  }
  if (!done) {  // everything in 64 bits
    double key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = l[i] > kOff ? score64(l[i]) + (double)b[i] : (double)kOff;
    if (grouped) keep_groups<V, double>(key, grp, a, lane, false);
    cand = -1;
    for (n = 0; n < a.k; ++n) {
      int e;
      const double m = best_left<V, double>(key, lane, &e);
      if (!(m > (double)kOff)) break;
      if (lane == n) cand = e;
      drop<V, double>(key, lane, e);
    }
  }

  // One 64-bit evaluation of all candidates; their order if they are biased.
  float x = 0.f, bx = 0.f;
  if (cand >= 0) {
    x = clamp_in(load_logit(a, row + cand));
    if (biased) bx = clamp_in(a.bias[cand]);
  }
  const double score = cand >= 0 ? score64(x) : 0.0;
  int rank = lane;
  if (biased && done) {
    const double choice = cand >= 0 ? score + (double)bx : (double)kOff;
    rank = 0;
    for (int j = 0; j < n; ++j) {
      const double o = lane_of(choice, j);
      const int oe = __builtin_amdgcn_readlane(cand, j);
      rank += (o > choice || (o == choice && oe < cand)) ? 1 : 0;
    }
  }
  const bool chosen = cand >= 0 && rank < a.k;
  float w = chosen ? (float)score : 0.f;
  if (a.renorm) w = w / (wave_sum(w) + 1e-20f);
  w *= a.scaling;
  if (chosen) {
    a.ids[(int64_t)t * a.k + rank] = cand;
    a.weights[(int64_t)t * a.k + rank] = w;
  } else if (lane >= n && lane < a.k) {  // fewer experts than slots
    a.ids[(int64_t)t * a.k + lane] = -1;
    a.weights[(int64_t)t * a.k + lane] = 0.f;
  }
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + kWavesPerBlock - 1) / kWavesPerBlock));
  const dim3 block(64 * kWavesPerBlock);
  const int v = (a.E + 63) / 64;
  if (v <= 1) hipLaunchKernelGGL((route_kernel<1>), grid, block, 0, stream, a);
  else if (v <= 2) hipLaunchKernelGGL((route_kernel<2>), grid, block, 0, stream, a);
  else if (v <= 4) hipLaunchKernelGGL((route_kernel<4>), grid, block, 0, stream, a);
  else if (v <= 6) hipLaunchKernelGGL((route_kernel<6>), grid, block, 0, stream, a);
  else if (v <= 8) hipLaunchKernelGGL((route_kernel<8>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((route_kernel<16>), grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace chord
