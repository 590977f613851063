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

// XS, WS: chunks of x and of W that LDS holds.
template <int WM, int WN, int MG, int NT, int XS, int WS>
struct Shape {
  static constexpr int kTM = WM * MG * 16, kTN = WN * NT * 16;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int kXBytes = kTM * kRowBytes, kWBytes = kTN * kRowBytes;  // of a chunk
  static constexpr int kRing = XS * kXBytes + WS * kWBytes;
  static constexpr int kPitch = kTN + 4;  // floats of a token in the epilogue
  static constexpr int kOutRows = kTM > 128 ? 128 : kTM;
  static constexpr size_t kLds = kRing > kOutRows * kPitch * 4 ? kRing : kOutRows * kPitch * 4;
};

template <bool F16, int WM, int WN, int MG, int NT, int XS, int WS>
__device__ __forceinline__ void run_item(const LinearArgs& a, uint8_t* lds, int tile, int slice, int part) {
  using S = Shape<WM, WN, MG, NT, XS, WS>;
  constexpr int TM = S::kTM, TN = S::kTN, kWaves = S::kWaves, kThreads = S::kThreads, XB = S::kXBytes, WB = S::kWBytes;
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

  // Instruction i of a wave for x brings rows 8 (wave + kWaves i) .. + 7, one row per 8
  // lanes.  W: the same of the lower half of the slice's rows (gated: the gate rows)
  // for the first kW / 2, then of the upper half (the up rows).
  constexpr int kX = TM / 8 / kWaves, kW = TN / 8 / kWaves;
  static_assert(kX >= 1 && kW >= 2);
  const int w_lo = min(TN / 2, a.N - first), w_hi = a.gated ? w_lo : max(0, min(TN / 2, a.N - first - TN / 2));
  const __amdgpu_buffer_rsrc_t xres = row_buffer(a.x + m0 * a.ldx, rows, a.ldx, a.K);
  const __amdgpu_buffer_rsrc_t wres = row_buffer(a.w + (int64_t)first * a.ldw, w_lo, a.ldw, a.K);
  const __amdgpu_buffer_rsrc_t ures =
      row_buffer(a.w + ((int64_t)(a.gated ? a.N : TN / 2) + first) * a.ldw, w_hi, a.ldw, a.K);
  uint32_t xo[kX], wo[kW];
  bool in_tail;
  {
    const int r = lane >> 3, p = (lane & 7) ^ (r & 6);
    in_tail = p * 8 < tail;
#pragma unroll
    for (int i = 0; i < kX; ++i) {
      const int row = 8 * (wave + kWaves * i) + r;
      xo[i] = row < rows ? (uint32_t)(row * a.ldx * 2 + (c_lo * 8 + p) * 16) : kLinNothing;
    }
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      const int row = 8 * (wave + kWaves * (i % (kW / 2))) + r;
      wo[i] = row < (i < kW / 2 ? w_lo : w_hi) ? (uint32_t)(row * a.ldw * 2 + (c_lo * 8 + p) * 16) : kLinNothing;
    }
  }
  typedef __attribute__((address_space(3))) void* Lds;
  uint8_t* const w_lds = lds + XS * XB;
  auto load_x = [&](int i, int at, int c) {
    const uint32_t o = c == last && !in_tail ? kLinNothing : xo[i];
    __builtin_amdgcn_raw_ptr_buffer_load_lds(xres, (Lds)(lds + at + (wave + kWaves * i) * 1024), 16, o, c * kRowBytes,
                                             0, 0);
  };
  auto load_w = [&](int i, int at, int c) {
    const uint32_t o = c == last && !in_tail ? kLinNothing : wo[i];
    const Lds to = (Lds)(w_lds + at + (wave + kWaves * i) * 1024);
    if (i < kW / 2) __builtin_amdgcn_raw_ptr_buffer_load_lds(wres, to, 16, o, c * kRowBytes, 0, 0);
    else __builtin_amdgcn_raw_ptr_buffer_load_lds(ures, to, 16, o, c * kRowBytes, 0, 0);
  };
  const int piece[2] = {(q ^ (col & 6)) * 16, ((4 + q) ^ (col & 6)) * 16};
  const int x_at = (wm * MG * 16 + col) * kRowBytes, w_at = (wn * (NT / 2) * 16 + col) * kRowBytes;
  auto read_x = [&](int at, int j, int g) {
    return *reinterpret_cast<const u32x4_t*>(lds + at + (x_at + piece[j]) + g * 16 * kRowBytes);
  };
  auto read_w = [&](int at, int j, int n) {
    const int r = n < NT / 2 ? n * 16 : TN / 2 + (n - NT / 2) * 16;
    return *reinterpret_cast<const u32x4_t*>(w_lds + at + (w_at + piece[j]) + r * kRowBytes);
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
  // Chunk c loads x of chunk c + XS - 1 before its barrier and W of chunk c + WS behind
  // it (each where its buffer is free), so the loads are spread over the chunk; here
  // those of the chunks before the first.
  constexpr int kMost = XS - 1 > WS ? XS - 1 : WS;
#pragma unroll
  for (int c = -kMost; c < 0; ++c) {
    if (c + XS - 1 >= 0 && c + XS - 1 < nc) {
#pragma unroll
      for (int i = 0; i < kX; ++i) load_x(i, (c + XS - 1) * XB, c + XS - 1);
    }
    if (c + WS >= 0 && c + WS < nc) {
#pragma unroll
      for (int i = 0; i < kW; ++i) load_w(i, (c + WS) * WB, c + WS);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  if (nc >= kMost) barrier(std::integral_constant<int, (XS - 2) * kX + (WS - 1) * kW>{});
  else barrier(std::integral_constant<int, 0>{});
#pragma unroll
  for (int n = 0; n < NT; ++n) w[0][n] = read_w(0, 0, n);
#pragma unroll
  for (int r = 0; r < kAhead; ++r) x[r] = read_x(0, 0, r);
  int xat = 0, wat = 0, xfar = (XS - 1) * XB;  // buffers of chunk c, and x's of chunk c + XS - 1
  // Younger than x and W of chunk c + 1, at the barrier of chunk c (steady: none is left
  // out near the end).
  constexpr int kFromX = (XS - 2) * (kX + kW), kFromW = (WS - 1) * kX + (WS - 2) * kW;
  constexpr int kYounger = kFromX < kFromW ? kFromX : kFromW;
  auto chunk = [&](int c, auto is_steady) {
    constexpr bool steady = decltype(is_steady)::value;
    const int xnext = xat + XB == XS * XB ? 0 : xat + XB, wnext = wat + WB == WS * WB ? 0 : wat + WB;
    const bool more_x = steady || c + XS - 1 < nc, more_w = steady || c + WS < nc;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      constexpr int kBefore = kSteps - kAhead;
      const int j = s / MG, g = s % MG, r = s + kAhead, past = s - kBefore;
      if (past == 0) barrier(std::integral_constant<int, steady ? kYounger : 0>{});
      x[r % kRing] = r < kSteps ? read_x(xat, r / MG, r % MG) : read_x(xnext, 0, r - kSteps);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n * (MG / 2) / NT == s) w[1][n] = read_w(wat, 1, n);
        if (past >= 0 && n * kAhead / NT == past) w[0][n] = read_w(wnext, 0, n);
      }
      if (past < 0 && more_x) {
#pragma unroll
        for (int i = 0; i < kX; ++i)
          if (i * kBefore / kX == s) load_x(i, xfar, c + XS - 1);
      }
      if (past >= 0 && more_w) {
#pragma unroll
        for (int i = 0; i < kW; ++i)
          if (i * kAhead / kW == past) load_w(i, wat, c + WS);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[g][n] = mfma16<F16>(w[j][n], x[s % kRing], acc[g][n]);
      __builtin_amdgcn_sched_barrier(0);
    }
    xfar = xat;  // (chunk c + XS lies where chunk c did)
    xat = xnext;
    wat = wnext;
  };
  int c = 0;
  for (; c + (XS - 1 > WS ? XS - 1 : WS) < nc; ++c) chunk(c, std::true_type{});
  for (; c < nc; ++c) chunk(c, std::false_type{});

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
template <bool F16, int WM, int WN, int MG, int NT, int XS, int WS, int OCC>
__global__ __launch_bounds__(64 * WM * WN, OCC) void linear_tile(LinearArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  using S = Shape<WM, WN, MG, NT, XS, WS>;
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
    run_item<F16, WM, WN, MG, NT, XS, WS>(a, lds, uniform((int)(block * 8) + rest % wide), uniform(rest / wide),
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
#define CHORD_LINEAR_SHAPE(WM, WN, MG, NT, XS, WS, PER)                                                      \
  return a.f16 ? run(linear_tile<true, WM, WN, MG, NT, XS, WS, PER * WM * WN / 4>, WM * WN, PER,              \
                     Shape<WM, WN, MG, NT, XS, WS>::kLds)                                                    \
               : run(linear_tile<false, WM, WN, MG, NT, XS, WS, PER * WM * WN / 4>, WM * WN, PER,             \
                     Shape<WM, WN, MG, NT, XS, WS>::kLds)
  switch (shape) {
    case kLin256x256: CHORD_LINEAR_SHAPE(2, 4, 8, 4, 3, 2, 1);
    case kLin128x256: CHORD_LINEAR_SHAPE(2, 4, 4, 4, 3, 3, 1);
    case kLin128x128: CHORD_LINEAR_SHAPE(2, 4, 4, 2, 4, 4, 1);
    default: CHORD_LINEAR_SHAPE(2, 4, 2, 2, 6, 6, 1);
  }
#undef CHORD_LINEAR_SHAPE
}

}  // namespace chord
