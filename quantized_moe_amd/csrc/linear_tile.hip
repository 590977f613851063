// Dense product in 16 bits, LDS-tiled form for many rows: a workgroup of 8 waves
// computes TM tokens x TN rows of W, WM x WN waves of MG x 16 tokens by NT x 16 rows
// each.
//
// Weights go straight from memory into registers, tokens (128-byte row pieces, a
// chunk of 64 along K) straight from memory into LDS by buffer_load ... lds, three
// chunks ahead in four buffers.  With both operands in LDS a chunk would take as long
// to read from there as its products take; with one of them, half of that.
//
// Half a chunk is NT products for each of MG token operands; the next operand is
// read during them.  The one barrier of chunk c stands between its halves: behind it
// every wave knows that chunk c + 1 has landed, so the last step already reads the
// next chunk's first operand, and that chunk c - 1 is read, so its buffer takes chunk
// c + 3.  Weights of a half are loaded where the registers of that half are free: the
// first half's of chunk c + 2 in the second half of c, the second half's of c + 1 in
// the first.
//
// Token rows lie in LDS as eight 16-byte pieces, piece p of row r at p ^ (r & 6):
// 128-bit reads take lanes 0-3 with 20-23, 4-7 with 16-19 and so on, that is piece p
// of four rows with piece p ^ 1 of the next four, and these keys put them, and the 16
// lanes of two such groups, on different banks.
//
// The sums leave through LDS, so that the epilogue is a short loop over neighbouring
// outputs whatever the activation, and gate and up meet there.
#include <type_traits>

#include "linear_common.h"

namespace chord {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kXcds = 8;
constexpr int kStages = 4;  // chunks: one in use, three on their way
constexpr int kChunk = 64;  // values along K
constexpr int kRowBytes = 2 * kChunk;

template <int WM, int WN, int MG, int NT>
struct Shape {
  static constexpr int kTM = WM * MG * 16, kTN = WN * NT * 16;
  static constexpr int kPitch = kTN + 4;  // floats of a token in the epilogue
  static constexpr int kOutRows = kTM > 128 ? 128 : kTM;
  static constexpr size_t kLds = kStages * kTM * kRowBytes > kOutRows * kPitch * 4 ? kStages * kTM * kRowBytes
                                                                                  : kOutRows * kPitch * 4;
};

struct Item {
  int64_t m0;
  int rows;          // of tokens
  int slice, part;
};

template <bool F16, int WM, int WN, int MG, int NT>
__device__ __forceinline__ void run_item(const LinearArgs& a, uint8_t* lds, const Item& it) {
  using S = Shape<WM, WN, MG, NT>;
  constexpr int TM = S::kTM, TN = S::kTN;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int q = lane >> 4, col = lane & 15;
  const int chunks = (a.K + kChunk - 1) / kChunk;
  const int c_lo = (int)((int64_t)chunks * it.part / a.parts);
  const int c_end = (int)((int64_t)chunks * (it.part + 1) / a.parts);
  const int nc = c_end - c_lo;
  // Pieces past K are read as zeros: only the last chunk of all has any.
  const int tail = a.K - (chunks - 1) * kChunk;
  const int last = chunks - 1 - c_lo;

  // Tokens: instruction j brings rows 8 j .. 8 j + 7, one row per 8 lanes.
  constexpr int kDma = TM / 8 / kWaves;
  const __amdgpu_buffer_rsrc_t xres = row_buffer(a.x + it.m0 * a.ldx, it.rows, a.ldx, a.K);
  uint32_t xo[kDma];
  bool xin;
  {
    const int r = lane >> 3, p = (lane & 7) ^ (r & 6);
    xin = p * 8 < tail;
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      const int row = 8 * (wave + kWaves * i) + r;
      xo[i] = row < it.rows ? (uint32_t)(row * a.ldx * 2 + (c_lo * 8 + p) * 16) : kLinNothing;
    }
  }
  // Weights: tile n of this wave, rows past the last one repeat it.
  const int outs = a.gated ? TN / 2 : TN;  // outputs of a slice
  const int first = it.slice * outs;       // ... and its first one
  const __amdgpu_buffer_rsrc_t wres = row_buffer(a.w + (int64_t)first * a.ldw, min(outs, a.N - first), a.ldw, a.K);
  const __amdgpu_buffer_rsrc_t ures =
      a.gated ? row_buffer(a.w + ((int64_t)a.N + first) * a.ldw, min(outs, a.N - first), a.ldw, a.K) : wres;
  uint32_t wo[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = a.gated ? (wn * (NT / 2) + n % (NT / 2)) * 16 : (wn * NT + n) * 16;
    wo[n] = (uint32_t)(min(r + col, a.N - first - 1) * a.ldw * 2 + (c_lo * 8 + q) * 16);
  }
  const bool win[2] = {q * 8 < tail, 32 + q * 8 < tail};

  u32x4_t w[2][NT][2];
  auto load_w = [&](int n, int j, int b, int c) {
    const uint32_t o = c == last && !win[j] ? kLinNothing : wo[n] + j * 64;
    w[b][n][j] = __builtin_amdgcn_raw_buffer_load_b128(n < NT / 2 ? wres : ures, o, c * kRowBytes, 0);
  };
  auto load_x = [&](int i, int b, int c) {
    const uint32_t o = c == last && !xin ? kLinNothing : xo[i];
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        xres, (__attribute__((address_space(3))) void*)(lds + b * (TM * kRowBytes) + (wave + kWaves * i) * 1024), 16,
        o, c * kRowBytes, 0, 0);
  };
  const int x_row = (wm * MG * 16 + col) * kRowBytes;
  const int x_at[2] = {x_row + ((q ^ (col & 6)) * 16), x_row + (((4 + q) ^ (col & 6)) * 16)};
  auto read_x = [&](int b, int j, int g) {
    return *reinterpret_cast<const u32x4_t*>(lds + b * (TM * kRowBytes) + x_at[j] + g * 16 * kRowBytes);
  };

  f32x4_t acc[MG][NT];
#pragma unroll
  for (int g = 0; g < MG; ++g)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[g][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  auto barrier = [&](auto outstanding) {  // ... loads of this wave may be on their way
    constexpr int vm = decltype(outstanding)::value;
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((vm & 15) | (7 << 4) | (15 << 8) | ((vm >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  u32x4_t x[2];
  // Chunk c in buffer b (= c % 4); its first operand is in x[0].  In the loop load
  // indices past the end repeat the last chunk, so every chunk issues the same loads
  // and the counts at the barrier are exact: younger than the tokens of chunk c + 1 are
  // NT weights each of this chunk's second half, the next one's first and second half,
  // and the tokens of chunk c + 2.  Behind the loop no tokens are loaded, and the
  // counts take no weights for granted.
  auto chunk = [&](auto buffer, int c, auto is_last) {
    constexpr int b = decltype(buffer)::value, nb = (b + 1) % kStages, fb = (b + 3) % kStages;
    constexpr bool behind = decltype(is_last)::value;
    const int c1 = min(c + 1, nc - 1), c2 = min(c + 2, nc - 1), c3 = min(c + 3, nc - 1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (j == 1 && !behind) barrier(std::integral_constant<int, 3 * NT + kDma>{});
      if (j == 1 && behind && b == 0) barrier(std::integral_constant<int, kDma>{});
      if (j == 1 && behind && b == 1) barrier(std::integral_constant<int, 0>{});
#pragma unroll
      for (int g = 0; g < MG; ++g) {
        const int s = j * MG + g;
        x[(s + 1) & 1] = s + 1 < 2 * MG ? read_x(b, (s + 1) / MG, (s + 1) % MG) : read_x(nb, 0, 0);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[g][n] = mfma16<F16>(w[b & 1][n][j], x[s & 1], acc[g][n]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (j == 0 && n * MG / NT == g && (!behind || b < 2)) load_w(n, 1, nb & 1, c1);
          if (j == 1 && n * (MG / 2) / NT == g && (!behind || b == 0)) load_w(n, 0, b & 1, c2);
        }
        if (j == 1 && !behind) {
#pragma unroll
          for (int i = 0; i < kDma; ++i)
            if (MG / 2 + i * (MG / 2) / kDma == g) load_x(i, fb, c3);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  auto load_all_w = [&](int j, int b, int c) {
#pragma unroll
    for (int n = 0; n < NT; ++n) load_w(n, j, b, min(c, nc - 1));
    __builtin_amdgcn_sched_barrier(0);
  };
  auto load_all_x = [&](int b) {
#pragma unroll
    for (int i = 0; i < kDma; ++i) load_x(i, b, min(b, nc - 1));
    __builtin_amdgcn_sched_barrier(0);
  };
  load_all_w(0, 0, 0);
  load_all_x(0);
  load_all_x(1);
  load_all_w(1, 0, 0);
  load_all_w(0, 1, 1);
  load_all_x(2);
  barrier(std::integral_constant<int, 2 * kDma + 2 * NT>{});
  x[0] = read_x(0, 0, 0);
  const std::false_type in_loop;
  const std::true_type behind_loop;
  const std::integral_constant<int, 0> b0;
  const std::integral_constant<int, 1> b1;
  const std::integral_constant<int, 2> b2;
  const std::integral_constant<int, 3> b3;
  int c = 0;
  for (; c + 3 < nc; c += 4) {
    chunk(b0, c, in_loop);
    chunk(b1, c + 1, in_loop);
    chunk(b2, c + 2, in_loop);
    chunk(b3, c + 3, in_loop);
  }
  // Weights that no chunk behind the loop needs are read all the same: a load
  // without a reader on some path could be dropped or moved there, and the counts in
  // the loop rely on every one.
  auto used = [&](int b, int j) {
#pragma unroll
    for (int n = 0; n < NT; ++n) asm volatile("" ::"v"(w[b][n][j]));
  };
  if (c < nc) chunk(b0, c, behind_loop);
  else used(0, 0), used(0, 1);
  if (c + 1 < nc) chunk(b1, c + 1, behind_loop);
  else used(1, 0);
  if (c + 2 < nc) chunk(b2, c + 2, behind_loop);
  // The repeated loads at the end land before their buffers are used again.
  __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));

  if (a.parts > 1) {  // fp32 sums of this part, by row of W
    const int half = (a.N + 15) / 16 * 16, pitch = a.gated ? 2 * half : half;
    float* p = a.partials + ((int64_t)it.part * a.M + it.m0) * pitch;
#pragma unroll
    for (int g = 0; g < MG; ++g) {
      const int m = (wm * MG + g) * 16 + col;
      if (m >= it.rows) continue;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int f = first + (a.gated ? (wn * (NT / 2) + n % (NT / 2)) * 16 : (wn * NT + n) * 16);
        if (f < half)
          *reinterpret_cast<f32x4_t*>(p + (int64_t)m * pitch + (a.gated && n >= NT / 2 ? half : 0) + f + 4 * q) =
              acc[g][n];
      }
    }
    return;
  }
  float* sums = reinterpret_cast<float*>(lds);
  constexpr int kPasses = TM / S::kOutRows, kGroups = S::kOutRows / 16;
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    __syncthreads();
#pragma unroll
    for (int g = 0; g < MG; ++g) {
      const int t = wm * MG + g - pass * kGroups;  // token group in this pass
      if (t < 0 || t >= kGroups) continue;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        *reinterpret_cast<f32x4_t*>(sums + (t * 16 + col) * S::kPitch + (wn * NT + n) * 16 + 4 * q) = acc[g][n];
    }
    __syncthreads();
    const int quads = outs / 4;
    for (int i = threadIdx.x; i < S::kOutRows * quads; i += kThreads) {
      const int m = i / quads, o = (i - m * quads) * 4;
      if (pass * S::kOutRows + m >= it.rows) break;
      const float* p = sums + m * S::kPitch;
      // (gated: a wave's NT tiles are NT / 2 of gate rows, then their up rows)
      constexpr int kHalf = NT / 2 * 16;
      const int at = a.gated ? o / kHalf * (2 * kHalf) + o % kHalf : o;
      const f32x4_t z = *reinterpret_cast<const f32x4_t*>(p + at);
      const f32x4_t up = *reinterpret_cast<const f32x4_t*>(p + (a.gated ? at + kHalf : at));
      store_out4(a, it.m0 + pass * S::kOutRows + m, first + o, z, up);
    }
  }
}

// Persistent workgroups; workgroup b runs on XCD b % 8.  Runs of consecutive items go
// to one XCD at a time, and items walk blocks of 8 token tiles slice by slice, so
// those that run together share few token tiles and few slices through their L2.
template <bool F16, int WM, int WN, int MG, int NT, int OCC>
__global__ __launch_bounds__(kThreads, OCC) void linear_tile(LinearArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  using S = Shape<WM, WN, MG, NT>;
  const int outs = a.gated ? S::kTN / 2 : S::kTN;
  const int slices = (a.N + outs - 1) / outs;
  const int64_t tiles = (a.M + S::kTM - 1) / S::kTM, whole = tiles * slices;
  const int run = gridDim.x / kXcds;  // (the grid is a multiple of 8)
  for (int64_t i = (int64_t)(blockIdx.x % kXcds) * run + blockIdx.x / kXcds; i < whole * a.parts; i += gridDim.x) {
    const int64_t u = i % whole, block = u / (8 * slices);
    const int wide = (int)min((int64_t)8, tiles - block * 8);
    const int rest = (int)(u - block * 8 * slices);
    Item it;
    it.part = (int)(i / whole);
    it.slice = rest / wide;
    it.m0 = (block * 8 + rest % wide) * S::kTM;
    it.rows = (int)min((int64_t)S::kTM, a.M - it.m0);
    __syncthreads();  // the last item's epilogue has left LDS
    run_item<F16, WM, WN, MG, NT>(a, lds, it);
  }
}

}  // namespace

hipError_t launch_linear_tile(const LinearArgs& a, int shape, hipStream_t stream) {
  const int cus = a.num_cus >= 8 ? a.num_cus / 8 * 8 : 8;
  auto run = [&](auto kernel, int per_cu, size_t lds) {
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(cus * per_cu)), dim3(kThreads), lds, stream, a);
    return hipGetLastError();
  };
#define CHORD_LINEAR_SHAPE(WM, WN, MG, NT, OCC)                                               \
  return a.f16 ? run(linear_tile<true, WM, WN, MG, NT, OCC>, OCC / 2, Shape<WM, WN, MG, NT>::kLds) \
               : run(linear_tile<false, WM, WN, MG, NT, OCC>, OCC / 2, Shape<WM, WN, MG, NT>::kLds)
  switch (shape) {
    case kLin256x256: CHORD_LINEAR_SHAPE(2, 4, 8, 4, 2);
    case kLin128x256: CHORD_LINEAR_SHAPE(2, 4, 4, 4, 2);
    case kLin128x128: CHORD_LINEAR_SHAPE(2, 4, 4, 2, 4);
    default: CHORD_LINEAR_SHAPE(2, 4, 2, 2, 4);
  }
#undef CHORD_LINEAR_SHAPE
}

}  // namespace chord
