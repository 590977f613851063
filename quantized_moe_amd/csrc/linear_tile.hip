// Dense product in 16 bits, LDS-tiled form for many rows: a workgroup of 8 waves
// computes TM tokens x TN rows of W, WM x WN waves of MG x 16 tokens by NT x 16 rows
// each.
//
// Rows of x and of W come in chunks of 64 along K (128 bytes a row) straight from
// memory into LDS (buffer_load ... lds, eight lanes a row, so that a line is one
// request; weights loaded as operands, 16 rows to an instruction, took 2.1 us a chunk
// for the requests of single lanes).  LDS reads 256 bytes a cycle, three times what the
// operands need.
//
// A chunk is 2 MG steps of NT products; token operands are read kAhead steps before
// theirs, so the barrier of a chunk stands where the next step's reads would leave it,
// kAhead steps before its end: behind it every wave holds the rest of the chunk in
// registers, the next chunk has landed, and the buffer takes the chunk kStages further
// on.  The products of those steps run while the next chunk's first operands come.
//
// Rows lie in LDS as eight 16-byte pieces, piece p of row r at p ^ (r & 6): 128-bit
// reads take lanes 0-3 with 20-23, 4-7 with 16-19 and so on, that is piece p of four
// rows with piece p ^ 1 of the next four, and these keys put them, and the 16 lanes of
// two such groups, on different banks.
//
// The sums leave through LDS, so that the epilogue is a short loop over neighbouring
// outputs whatever the activation, and gate and up meet there.
#include <type_traits>

#include "linear_common.h"

namespace chord {
namespace {

constexpr int kXcds = 8;
constexpr int kChunk = 64;  // values along K
constexpr int kRowBytes = 2 * kChunk;

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

template <int WM, int WN, int MG, int NT, int STAGES>
struct Shape {
  static constexpr int kTM = WM * MG * 16, kTN = WN * NT * 16;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int kStageBytes = (kTM + kTN) * kRowBytes;
  static constexpr int kPitch = kTN + 4;  // floats of a token in the epilogue
  static constexpr int kOutRows = kTM > 128 ? 128 : kTM;
  static constexpr size_t kLds = STAGES * kStageBytes > kOutRows * kPitch * 4 ? STAGES * kStageBytes
                                                                             : kOutRows * kPitch * 4;
};

template <bool F16, int WM, int WN, int MG, int NT, int STAGES>
__device__ __forceinline__ void run_item(const LinearArgs& a, uint8_t* lds, int tile, int slice, int part) {
  using S = Shape<WM, WN, MG, NT, STAGES>;
  constexpr int TM = S::kTM, TN = S::kTN, kWaves = S::kWaves, kThreads = S::kThreads, SB = S::kStageBytes;
  constexpr int kSteps = 2 * MG;
  constexpr int kAhead = MG >= 8 ? 6 : MG >= 4 ? 3 : 2, kRing = MG >= 8 ? 8 : 4;
  static_assert(kSteps % kRing == 0 && kAhead < kRing && kAhead <= MG && NT % 2 == 0);
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int q = lane >> 4, col = lane & 15;
  const int64_t m0 = (int64_t)tile * TM;
  const int rows = (int)min((int64_t)TM, a.M - m0);
  const int chunks = (a.K + kChunk - 1) / kChunk;
  const int c_lo = (int)((int64_t)chunks * part / a.parts);
  const int nc = (int)((int64_t)chunks * (part + 1) / a.parts) - c_lo;
  // Pieces past K are read as zeros: only the last chunk of all has any.
  const int tail = a.K - (chunks - 1) * kChunk;
  const int last = chunks - 1 - c_lo;
  const int outs = a.gated ? TN / 2 : TN;  // outputs of a slice
  const int first = slice * outs;          // ... and its first one

  // Instruction i of a wave brings rows 8 (wave + kWaves i) .. + 7 of the stage, one row
  // per 8 lanes: first x, then the lower half of the slice's rows of W (gated: the gate
  // rows), then the upper half (the up rows).
  constexpr int kX = TM / 8 / kWaves, kW = TN / 2 / 8 / kWaves, kDma = kX + 2 * kW;
  static_assert(kX >= 1 && kW >= 1);
  const int w_lo = min(TN / 2, a.N - first), w_hi = a.gated ? w_lo : max(0, min(TN / 2, a.N - first - TN / 2));
  const __amdgpu_buffer_rsrc_t xres = row_buffer(a.x + m0 * a.ldx, rows, a.ldx, a.K);
  const __amdgpu_buffer_rsrc_t wres = row_buffer(a.w + (int64_t)first * a.ldw, w_lo, a.ldw, a.K);
  const __amdgpu_buffer_rsrc_t ures =
      row_buffer(a.w + ((int64_t)(a.gated ? a.N : TN / 2) + first) * a.ldw, w_hi, a.ldw, a.K);
  uint32_t off[kDma];
  bool in_tail;
  {
    const int r = lane >> 3, p = (lane & 7) ^ (r & 6);
    in_tail = p * 8 < tail;
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      const int k = i < kX ? i : i < kX + kW ? i - kX : i - kX - kW;
      const int row = 8 * (wave + kWaves * k) + r, end = i < kX ? rows : i < kX + kW ? w_lo : w_hi;
      const int64_t ld = i < kX ? a.ldx : a.ldw;
      off[i] = row < end ? (uint32_t)(row * ld * 2 + (c_lo * 8 + p) * 16) : kLinNothing;
    }
  }
  auto load = [&](int i, int at, int c) {
    const uint32_t o = c == last && !in_tail ? kLinNothing : off[i];
    // (x rows, then W rows: kWaves 1 KB pieces an instruction)
    auto to = (__attribute__((address_space(3))) void*)(lds + at + (wave + kWaves * i) * 1024);
    if (i < kX) __builtin_amdgcn_raw_ptr_buffer_load_lds(xres, to, 16, o, c * kRowBytes, 0, 0);
    else if (i < kX + kW) __builtin_amdgcn_raw_ptr_buffer_load_lds(wres, to, 16, o, c * kRowBytes, 0, 0);
    else __builtin_amdgcn_raw_ptr_buffer_load_lds(ures, to, 16, o, c * kRowBytes, 0, 0);
  };
  const int piece[2] = {(q ^ (col & 6)) * 16, ((4 + q) ^ (col & 6)) * 16};
  const int x_at = (wm * MG * 16 + col) * kRowBytes, w_at = (TM + wn * (NT / 2) * 16 + col) * kRowBytes;
  auto read_x = [&](int at, int j, int g) {
    return *reinterpret_cast<const u32x4_t*>(lds + at + (x_at + piece[j]) + g * 16 * kRowBytes);
  };
  auto read_w = [&](int at, int j, int n) {
    const int r = n < NT / 2 ? n * 16 : TN / 2 + (n - NT / 2) * 16;
    return *reinterpret_cast<const u32x4_t*>(lds + at + (w_at + piece[j]) + r * kRowBytes);
  };

  f32x4_t acc[MG][NT];
#pragma unroll
  for (int g = 0; g < MG; ++g)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[g][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // All LDS reads of this wave have arrived, and of its loads all but `vm`.
  auto barrier = [&](auto outstanding) {
    constexpr int vm = decltype(outstanding)::value;
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((vm & 15) | (7 << 4) | ((vm >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  u32x4_t x[kRing], w[2][NT];  // w[j]: of the chunk's half j
#pragma unroll
  for (int c = 0; c < STAGES; ++c) {
    if (c < nc)
#pragma unroll
      for (int i = 0; i < kDma; ++i) load(i, c * SB, c);
    __builtin_amdgcn_sched_barrier(0);
  }
  if (nc >= STAGES) barrier(std::integral_constant<int, (STAGES - 1) * kDma>{});
  else barrier(std::integral_constant<int, 0>{});
#pragma unroll
  for (int n = 0; n < NT; ++n) w[0][n] = read_w(0, 0, n);
#pragma unroll
  for (int r = 0; r < kAhead; ++r) x[r] = read_x(0, 0, r);
  int at = 0;
  for (int c = 0; c < nc; ++c) {
    const int next = at + SB == STAGES * SB ? 0 : at + SB;
    const bool more = c + STAGES < nc;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int j = s / MG, g = s % MG, r = s + kAhead, past = s - (kSteps - kAhead);
      if (past == 0) {
        // (The loads of chunks c + 2 .. c + STAGES - 1 are younger than those of c + 1.)
        if (STAGES > 2 && c + STAGES <= nc) barrier(std::integral_constant<int, (STAGES - 2) * kDma>{});
        else barrier(std::integral_constant<int, 0>{});
      }
      x[r % kRing] = r < kSteps ? read_x(at, r / MG, r % MG) : read_x(next, 0, r - kSteps);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n * (MG / 2) / NT == s) w[1][n] = read_w(at, 1, n);
        if (past >= 0 && n * kAhead / NT == past) w[0][n] = read_w(next, 0, n);
      }
      if (past >= 0 && more) {
#pragma unroll
        for (int i = 0; i < kDma; ++i)
          if (i * kAhead / kDma == past) load(i, at, c + STAGES);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[g][n] = mfma16<F16>(w[j][n], x[s % kRing], acc[g][n]);
      __builtin_amdgcn_sched_barrier(0);
    }
    at = next;
  }

  // Row of W (inside the slice's two halves) of tile n.
  auto w_row = [&](int n) { return (n < NT / 2 ? 0 : TN / 2) + (wn * (NT / 2) + n % (NT / 2)) * 16; };
  if (a.parts > 1) {  // fp32 sums of this part, by row of W
    const int half = (a.N + 15) / 16 * 16, pitch = a.gated ? 2 * half : half;
    float* p = a.partials + ((int64_t)part * a.M + m0) * pitch;
#pragma unroll
    for (int g = 0; g < MG; ++g) {
      const int m = (wm * MG + g) * 16 + col;
      if (m >= rows) continue;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const bool up = a.gated && n >= NT / 2;
        const int f = first + w_row(n) - (up ? TN / 2 : 0);
        if (f < half) *reinterpret_cast<f32x4_t*>(p + (int64_t)m * pitch + (up ? half : 0) + f + 4 * q) = acc[g][n];
      }
    }
    return;
  }
  float* sums = reinterpret_cast<float*>(lds);
  // (Opaque, so that addresses of the epilogue hold no registers during the loop.)
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
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
        *reinterpret_cast<f32x4_t*>(sums + (t * 16 + (tid & 15)) * S::kPitch + w_row(n) + (tid >> 4 & 3) * 4) =
            acc[g][n];
    }
    __syncthreads();
    // A thread has four neighbouring outputs of every kThreads / quads-th row, kBatch of
    // them at a time, so that their residuals are on their way together.
    constexpr int kBatch = 4;
    const int quads = outs / 4, step = kThreads / quads;
    const int o = (tid & (quads - 1)) * 4;
    const float* p = sums + o;
    const OutQuad out = out_quad(a, first + o);
    const int mine = min(rows - pass * S::kOutRows, S::kOutRows);
    if (out.left > 0) {
      for (int r = tid / quads; r < mine; r += kBatch * step) {
        f32x4_t res[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (r + u * step < mine) res[u] = out_residual(a, out, m0 + pass * S::kOutRows + r + u * step);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (r + u * step >= mine) continue;
          const float* v = p + (r + u * step) * S::kPitch;
          const f32x4_t z = *reinterpret_cast<const f32x4_t*>(v);
          const f32x4_t up = *reinterpret_cast<const f32x4_t*>(a.gated ? v + TN / 2 : v);
          out_store(a, out, m0 + pass * S::kOutRows + r + u * step, z, up, res[u]);
        }
      }
    }
  }
}

// Persistent workgroups; workgroup b runs on XCD b % 8.  Runs of consecutive items go
// to one XCD at a time, and items walk blocks of 8 token tiles slice by slice, so
// those that run together share few token tiles and few slices through their L2.
template <bool F16, int WM, int WN, int MG, int NT, int STAGES, int OCC>
__global__ __launch_bounds__(64 * WM * WN, OCC) void linear_tile(LinearArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  using S = Shape<WM, WN, MG, NT, STAGES>;
  const int outs = a.gated ? S::kTN / 2 : S::kTN;
  const int slices = (a.N + outs - 1) / outs;
  const int64_t tiles = (a.M + S::kTM - 1) / S::kTM, whole = tiles * slices;
  // (The grid is a multiple of 8.  Fewer items than workgroups spread over all XCDs.)
  const int run = (int)min((int64_t)gridDim.x / kXcds, (whole * a.parts + kXcds - 1) / kXcds);
  if ((int)(blockIdx.x / kXcds) >= run) return;
  for (int64_t i = (int64_t)(blockIdx.x % kXcds) * run + blockIdx.x / kXcds; i < whole * a.parts; i += kXcds * run) {
    const int64_t u = i % whole, block = u / (8 * slices);
    const int wide = (int)min((int64_t)8, tiles - block * 8);
    const int rest = (int)(u - block * 8 * slices);
    __syncthreads();  // the last item's epilogue has left LDS
    run_item<F16, WM, WN, MG, NT, STAGES>(a, lds, uniform((int)(block * 8) + rest % wide), uniform(rest / wide),
                                  uniform((int)(i / whole)));
  }
}

}  // namespace

hipError_t launch_linear_tile(const LinearArgs& a, int shape, hipStream_t stream) {
  const int cus = a.num_cus >= 8 ? a.num_cus / 8 * 8 : 8;
  auto run = [&](auto kernel, int waves, int per_cu, size_t lds) {
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(cus * per_cu)), dim3(64 * waves), lds, stream, a);
    return hipGetLastError();
  };
// (PER: workgroups of a CU)
#define CHORD_LINEAR_SHAPE(WM, WN, MG, NT, STAGES, PER)                                                      \
  return a.f16 ? run(linear_tile<true, WM, WN, MG, NT, STAGES, PER * WM * WN / 4>, WM * WN, PER,              \
                     Shape<WM, WN, MG, NT, STAGES>::kLds)                                                    \
               : run(linear_tile<false, WM, WN, MG, NT, STAGES, PER * WM * WN / 4>, WM * WN, PER,             \
                     Shape<WM, WN, MG, NT, STAGES>::kLds)
  switch (shape) {
    case kLin256x256: CHORD_LINEAR_SHAPE(2, 4, 8, 4, 2, 1);
    case kLin128x256: CHORD_LINEAR_SHAPE(2, 4, 4, 4, 3, 1);
    case kLin128x128: CHORD_LINEAR_SHAPE(2, 4, 4, 2, 4, 1);
    default: CHORD_LINEAR_SHAPE(2, 4, 2, 2, 3, 2);
  }
#undef CHORD_LINEAR_SHAPE
}

}  // namespace chord
