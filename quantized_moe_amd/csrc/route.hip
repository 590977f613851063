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
// in a few hundred tokens.
//
//   * Without a bias both scores rise with the logit, so the logits decide;
//     with one, the choices.
//   * The keys of the selection are 32-bit approximations with a known error.
//     The rounds go on past the k-th best while the next key is within that
//     error (usually no further round).  The candidates stand one a lane; if two
//     neighbours among them are within the error, the exact values (logits, or
//     choices in 64 bits), one a lane, order them, else they are in order
//     already.
//   * Group scores whose border is closer than the error, or more than 64
//     candidates, take the 64-bit path for the whole token.
//
// Keys are unsigned integers in the order of the floats (0: not available) whose
// four lowest bits hold the place in the lane, so sorting a lane takes a
// minimum and a maximum per pair, and a round one look at the lanes' heads.
// Bound by instruction issue: 8192 tokens of 384 experts took 16 us with 64-bit
// scores for every candidate, 19 with all keys scanned every round, 15 with
// places sorted beside the keys, 11 so; its bytes would take 2.6 us.  (550 vector and
// 238 scalar instructions a token; the vector units issue in 61 % of the cycles, and
// the waves wait for an issue slot in 38 % of theirs.)
#include <type_traits>

#include "device_common.h"

namespace chord {
namespace {

constexpr int kWavesPerBlock = 4;
constexpr float kOff = -INFINITY;  // logit of an expert that cannot be chosen
// Bound of the difference of two keys' errors.  A sigmoid is within 3e-7 (hardware
// exp2 and reciprocal), a softmax within 2.5e-6 of its value (its sum has up to
// 16 + 6 additions in a row), a choice adds one rounding; a logit is exact.
// The place in the low bits takes 2^-19 of the value.
constexpr float kErrAbs = 6e-6f, kErrRel = 5e-6f;

// Order-preserving integer of a float; 0 for -inf alone.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // (-0 counts as 0)
  return x > kOff ? ((int32_t)b < 0 ? ~b : b | 0x80000000u) : 0u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return k == 0u ? kOff : __uint_as_float((int32_t)k < 0 ? k & 0x7FFFFFFFu : ~k);
}

template <int CTRL>
__device__ __forceinline__ uint32_t row_step(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
}
// Maximum over the wave, uniform: neighbours 1, 2, 4 and 8 away inside the rows
// of 16 lanes, then the four rows' last lanes.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = max(x, row_step<0x111>(x));
  x = max(x, row_step<0x112>(x));
  x = max(x, row_step<0x114>(x));
  x = max(x, row_step<0x118>(x));
  const uint32_t a = __builtin_amdgcn_readlane((int)x, 15), b = __builtin_amdgcn_readlane((int)x, 31);
  const uint32_t c = __builtin_amdgcn_readlane((int)x, 47), d = __builtin_amdgcn_readlane((int)x, 63);
  return max(max(a, b), max(c, d));
}
__device__ __forceinline__ float lane_f(float x, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane(__float_as_int(x), lane));
}
__device__ __forceinline__ float wave_sum(float x) {
  x += __uint_as_float(row_step<0x111>(__float_as_uint(x)));
  x += __uint_as_float(row_step<0x112>(__float_as_uint(x)));
  x += __uint_as_float(row_step<0x114>(__float_as_uint(x)));
  x += __uint_as_float(row_step<0x118>(__float_as_uint(x)));
  return (lane_f(x, 15) + lane_f(x, 31)) + (lane_f(x, 47) + lane_f(x, 63));
}
__device__ __forceinline__ double wave_max(double x) {
  for (int d = 1; d < 64; d <<= 1) x = fmax(x, __shfl_xor(x, d, 64));
  return x;
}
__device__ __forceinline__ double wave_sum(double x) {
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
  return x;
}
__device__ __forceinline__ float lane_of(float x, int lane) { return lane_f(x, lane); }
__device__ __forceinline__ double lane_of(double x, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float as_value(uint32_t k) { return value_of(k); }
__device__ __forceinline__ double as_value(double k) { return k; }
__device__ __forceinline__ uint32_t nothing(uint32_t) { return 0u; }
__device__ __forceinline__ double nothing(double) { return -INFINITY; }

// Sorts a lane's keys, largest first (Batcher's odd-even merge network).
template <int V>
__device__ __forceinline__ void sort_lane(uint32_t (&key)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t x = key[i + j], y = key[i + j + k];
            key[i + j] = max(x, y);
            key[i + j + k] = min(x, y);
          }
}
// Takes the best key left (of equal ones, which have the same place, the lowest
// lane's) and its expert; returns 0 if none is left.
template <int V>
__device__ __forceinline__ uint32_t take_best(uint32_t (&key)[V], int lane, int* expert) {
  const uint32_t m = wave_max(key[0]);
  const int src = __builtin_ctzll(__builtin_amdgcn_ballot_w64(key[0] == m));
  // (By bits: a choice between key[i + 1] and key[i] becomes an index at run time.)
  const uint32_t mine = lane == src ? ~0u : 0u;
#pragma unroll
  for (int i = 0; i + 1 < V; ++i) key[i] = (key[i + 1] & mine) | (key[i] & ~mine);
  key[V - 1] &= ~mine;
  *expert = (15 - (int)(m & 15)) * 64 + src;
  return m;
}
// The best of unsorted 64-bit keys, the lowest expert of equal ones (the rare path).
template <int V>
__device__ __forceinline__ double take_best(double (&key)[V], int lane, int* expert) {
  double m = key[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmax(m, key[i]);
  m = wave_max(m);
  if (!(m > -INFINITY)) return m;
  int e = INT32_MAX;
#pragma unroll
  for (int i = V - 1; i >= 0; --i) {
    const uint64_t has = __builtin_amdgcn_ballot_w64(key[i] == m);
    if (has != 0) e = i * 64 + __builtin_ctzll(has);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = i * 64 + lane == e ? -INFINITY : key[i];
  *expert = e;
  return m;
}

// Drops the keys of all groups but the topk_group best.  Lane g holds the score
// of group g (F: its type).  False if the border between the last group that
// stays and the first that goes is within the error of 32-bit keys (`approx`).
template <int V, bool BIASED, typename K, typename F>
__device__ __forceinline__ bool keep_groups(K (&key)[V], const int (&grp)[V], const RouteArgs& a,
                                            int lane, bool approx) {
  const int G = a.n_group;
  const K none = nothing(key[0]);
  F mine = (F)kOff;
  F size = 0;  // magnitude of the two summands
  for (int g = 0; g < G; ++g) {
    K t1 = none, t2 = none;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const K v = grp[i] == g ? key[i] : none;
      t2 = v > t1 ? t1 : (v > t2 ? v : t2);
      t1 = v > t1 ? v : t1;
    }
    // The two best over the wave: the best, then the best without one copy of
    // it (if two lanes hold it, it is also the second).
    const K m1 = wave_max(t1);
    F score = as_value(m1), mag = score > (F)kOff ? (F)fabs(score) : (F)0;
    if (BIASED) {
      const uint64_t has = __builtin_amdgcn_ballot_w64(t1 == m1);
      const K m2 = wave_max(lane == __builtin_ctzll(has) ? t2 : t1);
      if (m2 > none) {
        score += as_value(m2);
        mag += (F)fabs(as_value(m2));
      }
    }
    if (lane == g) {
      mine = score;
      size = mag;
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
    const float big = value_of(wave_max(key_of((float)size)));
    // (negated: a NaN gap, from groups without any expert, counts as close)
    if (!(gap > (F)(2 * kErrAbs) + (F)kErrRel * (F)big)) return false;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = (keep >> grp[i]) & 1 ? key[i] : none;
  return true;
}

// -inf and NaN: not available.  +inf counts as the largest finite number.
__device__ __forceinline__ float clamp_in(float x) {
  return x > kOff ? fminf(x, 3.402823466e38f) : kOff;
}

template <int V, bool BIASED, bool SIGMOID>
__global__ __launch_bounds__(64 * kWavesPerBlock, V <= 6 ? 8 : 4) void route_kernel(RouteArgs a) {
  __shared__ float ltab[kWavesPerBlock][V * 64];  // a wave's logits, to be read by candidate
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * kWavesPerBlock + wave));
  if (t >= a.T) return;
  const int64_t row = (int64_t)t * a.ld;
  float l[V], b[V];
  if (a.dtype == CHORD_DTYPE_F32) {
    const float* p = static_cast<const float*>(a.logits) + row;
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = p[min(i * 64 + lane, a.E - 1)];
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(a.logits) + row;
    uint16_t h[V];
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = p[min(i * 64 + lane, a.E - 1)];
#pragma unroll
    for (int i = 0; i < V; ++i)
      l[i] = a.dtype == CHORD_DTYPE_BF16 ? bf16_to_f32(h[i]) : (float)__builtin_bit_cast(_Float16, h[i]);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) b[i] = BIASED ? a.bias[min(i * 64 + lane, a.E - 1)] : 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    l[i] = i * 64 + lane < a.E && b[i] > kOff ? clamp_in(l[i]) : kOff;
    ltab[wave][i * 64 + lane] = l[i];
    if (BIASED) b[i] = clamp_in(b[i]);
  }
  // softmax: maximum and sum
  float top = 0.f, total = 1.f;
  if (!SIGMOID) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
    top = value_of(wave_max(key_of(m)));
    if (!(top > kOff)) top = 0.f;  // no expert: every term below is 0
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) s += l[i] > kOff ? expf(l[i] - top) : 0.f;
    total = wave_sum(s);
  }
  auto total64 = [&]() {
    if (SIGMOID) return 1.0;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) s += l[i] > kOff ? exp((double)l[i] - (double)top) : 0.0;
    return wave_sum(s);
  };
  auto score64 = [&](float x, double sum) {
    return SIGMOID ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)top) / sum;
  };
  const bool grouped = a.topk_group < a.n_group;
  int grp[V];
  if (grouped) {
#pragma unroll
    for (int i = 0; i < V; ++i) grp[i] = (int)(((uint32_t)(i * 64 + lane) * a.group_magic) >> 20) & 63;
  }

  // The candidates, one a lane, in descending order of their keys.
  int cand = -1, n = 0;
  bool sure = true;   // ... which is the exact order
  bool whole = true;  // all candidates there are
  {
    uint32_t key[V], ckey = 0u;
    const float inv = 1.f / total;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float v = l[i];
      if (BIASED) {
        const float s = SIGMOID ? __builtin_amdgcn_rcpf(1.f + __expf(-l[i])) : __expf(l[i] - top) * inv;
        v = l[i] > kOff ? s + b[i] : kOff;
      }
      const uint32_t k = key_of(v);
      key[i] = k != 0u ? (k & ~15u) | (15 - i) : 0u;
    }
    if (grouped) whole = keep_groups<V, BIASED, uint32_t, float>(key, grp, a, lane, true);
    sort_lane<V>(key);
    float kth = kOff;
    while (whole) {
      int e;
      const uint32_t m = take_best<V>(key, lane, &e);
      if (m == 0u) break;
      if (n >= a.k) {  // within the error of the k-th best: may belong before it
        const float v = value_of(m);
        if (n == a.k) kth = value_of(__builtin_amdgcn_readlane((int)ckey, n - 1));
        if (v < kth - (kErrAbs + kErrRel * fabsf(v))) break;
        if (n == 64) {
          whole = false;
          break;
        }
      }
      cand = lane == n ? e : cand;
      ckey = lane == n ? m : ckey;
      ++n;
    }
    // A candidate within the error of the one before is not in a sure place.
    const float v = value_of(ckey), before = __shfl_up(v, 1, 64);
    sure = __builtin_amdgcn_ballot_w64(lane > 0 && lane < n &&
                                       !(v < before - (kErrAbs + kErrRel * fabsf(v)))) == 0;
  }
  if (!whole) {  // everything in 64 bits
    const double sum = total64();
    double key[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
      key[i] = !(l[i] > kOff) ? -INFINITY : BIASED ? score64(l[i], sum) + (double)b[i] : (double)l[i];
    if (grouped) keep_groups<V, BIASED, double, double>(key, grp, a, lane, false);
    cand = -1;
    for (n = 0; n < a.k; ++n) {
      int e;
      if (!(take_best<V>(key, lane, &e) > -INFINITY)) break;
      cand = lane == n ? e : cand;
    }
  }

  const float x = cand >= 0 ? ltab[wave][cand] : 0.f;
  int rank = lane;
  if (whole && !sure) {  // order the candidates by their exact values
    double value = (double)x;
    if (BIASED) {
      const double sum = total64();  // (by all lanes)
      value = score64(x, sum) + (double)(cand >= 0 ? clamp_in(a.bias[cand]) : 0.f);
    }
    if (cand < 0) value = -INFINITY;
    rank = 0;
    for (int j = 0; j < n; ++j) {
      const double o = lane_of(value, j);
      const int oe = __builtin_amdgcn_readlane(cand, j);
      rank += (o > value || (o == value && oe < cand)) ? 1 : 0;
    }
  }
  const bool chosen = cand >= 0 && rank < a.k;
  float w = SIGMOID ? 1.f / (1.f + expf(-x)) : expf(x - top) / total;
  w = chosen ? w : 0.f;
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
  auto run = [&](auto biased, auto sigmoid) {
    constexpr bool B = decltype(biased)::value, S = decltype(sigmoid)::value;
    if (v <= 1) hipLaunchKernelGGL((route_kernel<1, B, S>), grid, block, 0, stream, a);
    else if (v <= 2) hipLaunchKernelGGL((route_kernel<2, B, S>), grid, block, 0, stream, a);
    else if (v <= 4) hipLaunchKernelGGL((route_kernel<4, B, S>), grid, block, 0, stream, a);
    else if (v <= 6) hipLaunchKernelGGL((route_kernel<6, B, S>), grid, block, 0, stream, a);
    else if (v <= 8) hipLaunchKernelGGL((route_kernel<8, B, S>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((route_kernel<16, B, S>), grid, block, 0, stream, a);
    return hipGetLastError();
  };
  const std::true_type yes{};
  const std::false_type no{};
  if (a.bias != nullptr) return a.sigmoid ? run(yes, yes) : run(yes, no);
  return a.sigmoid ? run(no, yes) : run(no, no);
}

}  // namespace chord
