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
// Sums leave from registers, rounded, 16 bytes a lane.  Outputs that do not lie so, and
// the long code of GELU, go through LDS to a short loop over neighbouring outputs.
//
// 8192 tokens through 4096 x 7168 take 346 us (1.39 PFLOP/s; the library's plain product
// 345), with the matrix units busy for 71 % of a clock that they hold to 1.8 GHz; 8192
// through 7168 x 2048 with a residual 223 us (1.08 PFLOP/s; the library's plain product
// 186): 32 chunks an item leave the epilogue, 670 MB in all, little to hide
// behind.
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
  static constexpr int kOutRows = 64;  // tokens that pass through LDS at a time
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
  if (a.direct) {
    // From registers to memory: a lane's four outputs of a tile, or eight of two
    // neighbouring tiles after a swap between quarters of the wave (quarter q then has
    // outputs 16 (q & 1) + 8 (q >> 1) on of the 32).
    constexpr bool kPair = NT == 4;
    constexpr int kWide = kPair ? 8 : 4;
    auto store = [&](auto is_gated, auto is_f32) {
      constexpr bool gated = decltype(is_gated)::value, F32 = decltype(is_f32)::value;
      constexpr int kTiles = gated ? NT / 2 : NT;         // of outputs,
      constexpr int kUnits = kPair ? kTiles / 2 : kTiles;  // stored at a time
      constexpr int kWords = kWide * (F32 ? 4 : 2) / 4;
      constexpr int kBatch = F32 ? 2 : MG < 4 ? MG : 4;    // token groups whose residuals come together
      f32x4_t bias[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int f = first + w_row(n) - (gated && n >= NT / 2 ? TN / 2 : 0) + 4 * q;
        bias[n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if (a.bias != nullptr && f < a.N)
          bias[n] = load4(a.bias, (gated && n >= NT / 2 ? a.N : 0) + f, a.bias_f32, F16, false, 4);
      }
      typedef uint32_t Words __attribute__((ext_vector_type(kWords)));
      const int64_t size = F32 ? 4 : 2;
      int64_t column[kUnits];
      bool in[kUnits];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int c = first + (kPair ? w_row(2 * u) + 16 * (q & 1) + 8 * (q >> 1) : w_row(u) + 4 * q);
        column[u] = c;
        in[u] = c < a.N;
      }
      const int64_t m = m0 + wm * MG * 16 + col;
      const int left = rows - wm * MG * 16 - col;  // rows from this lane's first on
      uint8_t* const out = static_cast<uint8_t*>(a.out) + m * a.ldo * size;
      const uint8_t* const more = static_cast<const uint8_t*>(a.residual) + m * a.ldr * size;
#pragma unroll
      for (int g0 = 0; g0 < MG; g0 += kBatch) {
        Words res[kBatch][kUnits];
        if (a.residual != nullptr) {
#pragma unroll
          for (int g = 0; g < kBatch; ++g)
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
              if ((g0 + g) * 16 < left && in[u])
                res[g][u] = *reinterpret_cast<const Words*>(more + ((g0 + g) * 16 * a.ldr + column[u]) * size);
        }
#pragma unroll
        for (int g = 0; g < kBatch; ++g) {
          f32x4_t h[kTiles];
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            f32x4_t z = acc[g0 + g][n] + bias[n];
            if (a.act != CHORD_ACT_NONE) {
#pragma unroll
              for (int i = 0; i < 4; ++i) z[i] = activate_short(a.act, z[i]);
            }
            if constexpr (gated) z *= acc[g0 + g][n + NT / 2] + bias[n + NT / 2];
            h[n] = z * a.scale;
          }
#pragma unroll
          for (int u = 0; u < kUnits; ++u) {
            float v[kWide];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if constexpr (kPair) {
                const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(h[2 * u][i]),
                                                                __float_as_uint(h[2 * u + 1][i]), false, false);
                v[i] = __uint_as_float(w[0]);
                v[i + 4] = __uint_as_float(w[1]);
              } else {
                v[i] = h[u][i];
              }
            }
            if (a.residual != nullptr) {
#pragma unroll
              for (int i = 0; i < kWide; ++i)
                v[i] += F32 ? __uint_as_float(res[g][u][i]) : value16(res[g][u][i / 2] >> (16 * (i & 1)) & 0xFFFF, F16);
            }
            Words w;
#pragma unroll
            for (int i = 0; i < kWords; ++i)
              w[i] = F32 ? __float_as_uint(v[i]) : F16 ? pack16<true>(v[2 * i], v[2 * i + 1]) : pack16<false>(v[2 * i], v[2 * i + 1]);
            if ((g0 + g) * 16 < left && in[u])
              *reinterpret_cast<Words*>(out + ((g0 + g) * 16 * a.ldo + column[u]) * size) = w;
          }
        }
      }
    };
    const std::true_type yes{};
    const std::false_type no{};
    if (a.out_f32) a.gated ? store(yes, yes) : store(no, yes);
    else a.gated ? store(yes, no) : store(no, no);
    return;
  }
  float* sums = reinterpret_cast<float*>(lds);
  // (Opaque, so that addresses of the epilogue hold no registers during the loop.)
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  constexpr int kPasses = TM / S::kOutRows, kGroups = S::kOutRows / 16;
  // A thread has four neighbouring outputs of every kThreads / quads-th row.  Their
  // residuals are on their way while the sums pass through LDS.
  const int quads = outs / 4, step = kThreads / quads;
  const int o = (tid & (quads - 1)) * 4;
  const OutQuad out = out_quad(a, first + o);
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    const int mine = out.left > 0 ? min(rows - pass * S::kOutRows, S::kOutRows) : 0;
    const int64_t top = m0 + pass * S::kOutRows;
    // (As many as a thread has where nothing is gated: the fewest rows are there then.)
    constexpr int kBatch = S::kOutRows * (TN / 4) / kThreads;
    const bool early = a.residual != nullptr && out.wide_res && mine > 0;
    u32x4_t res[kBatch];
    if (early && a.out_f32) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) res[u] = raw_residual<true>(a, out, top + min(tid / quads + u * step, mine - 1));
    } else if (early) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) res[u] = raw_residual<false>(a, out, top + min(tid / quads + u * step, mine - 1));
    }
    lds_barrier();
#pragma unroll
    for (int g = 0; g < MG; ++g) {
      const int t = wm * MG + g - pass * kGroups;  // token group in this pass
      if (t < 0 || t >= kGroups) continue;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        *reinterpret_cast<f32x4_t*>(sums + (t * 16 + (tid & 15)) * S::kPitch + w_row(n) + (tid >> 4 & 3) * 4) =
            acc[g][n];
    }
    lds_barrier();
    constexpr int kRead = kBatch < 4 ? kBatch : 4;
#pragma unroll
    for (int u0 = 0; u0 < kBatch; u0 += kRead) {
      f32x4_t z[kRead], up[kRead];
#pragma unroll
      for (int u = 0; u < kRead; ++u) {
        // (gated: half of the rows are behind the last)
        const float* v = sums + o + ((tid / quads + (u0 + u) * step) & (S::kOutRows - 1)) * S::kPitch;
        z[u] = *reinterpret_cast<const f32x4_t*>(v);
        up[u] = *reinterpret_cast<const f32x4_t*>(a.gated ? v + TN / 2 : v);
      }
#pragma unroll
      for (int u = 0; u < kRead; ++u) {
        const int r = tid / quads + (u0 + u) * step;
        if (r >= mine) continue;
        f32x4_t more = {0.f, 0.f, 0.f, 0.f};
        if (early) more = residual_value(a, res[u0 + u]);
        else if (a.residual != nullptr) more = out_residual(a, out, top + r);
        out_store(a, out, top + r, z[u], up[u], more);
      }
    }
  }
}

// Persistent workgroups; workgroup b runs on XCD b % 8.  Runs of consecutive items go
// to one XCD at a time, and items walk blocks of 8 token tiles slice by slice, so
// those that run together share few token tiles and few slices through their L2.
// CUT: items that fill no more than half a round are cut by rows into two (8192 x 7168
// outputs are 3.5 rounds).
template <bool F16, int WM, int WN, int MG, int NT, int XS, int WS, int OCC, bool CUT>
__global__ __launch_bounds__(64 * WM * WN, OCC) void linear_tile(LinearArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  using S = Shape<WM, WN, MG, NT, XS, WS>;
  const int outs = a.gated ? S::kTN / 2 : S::kTN;
  const int slices = (a.N + outs - 1) / outs;
  const int64_t tiles = (a.M + S::kTM - 1) / S::kTM, whole = tiles * slices, items = whole * a.parts;
  // (The grid is a multiple of 8.  Fewer items than workgroups spread over all XCDs.)
  const int64_t last = items / gridDim.x * gridDim.x, rest = items - last;
  const bool cut = CUT && rest > 0 && 2 * rest <= gridDim.x;
  const int xcd = blockIdx.x % kXcds, local = blockIdx.x / kXcds;
  for (int64_t begin = 0; begin < items; begin += gridDim.x) {
    const bool halves = cut && begin == last;
    const int64_t here = min((int64_t)gridDim.x, halves ? 2 * rest : items - begin);
    const int run = (int)((here + kXcds - 1) / kXcds), mine = xcd * run + local;
    if (local >= run || mine >= here) continue;  // (a last round: uniform over the workgroup)
    const int64_t i = begin + (halves ? mine >> 1 : mine);
    const int64_t u = i % whole, block = u / (8 * slices);
    const int wide = (int)min((int64_t)8, tiles - block * 8);
    const int at = (int)(u - block * 8 * slices);
    const int tile = uniform((int)(block * 8) + at % wide), slice = uniform(at / wide), part = uniform((int)(i / whole));
    lds_barrier();  // the last item's epilogue has left LDS
    if constexpr (CUT) {
      if (halves) {
        if ((int64_t)(2 * tile + (mine & 1)) * (S::kTM / 2) < a.M)
          run_item<F16, WM, WN, MG / 2, NT, XS, WS>(a, lds, 2 * tile + (mine & 1), slice, part);
        continue;
      }
    }
    run_item<F16, WM, WN, MG, NT, XS, WS>(a, lds, tile, slice, part);
  }
}

}  // namespace

hipError_t launch_linear_tile(const LinearArgs& a, int shape, hipStream_t stream) {
  const int cus = a.num_cus >= 8 ? a.num_cus / 8 * 8 : 8;
  auto run = [&](auto kernel, int waves, size_t lds) {
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)cus), dim3(64 * waves), lds, stream, a);
    return hipGetLastError();
  };
#define CHORD_LINEAR_SHAPE(WM, WN, MG, NT, XS, WS, CUT)                                                      \
  return a.f16 ? run(linear_tile<true, WM, WN, MG, NT, XS, WS, WM * WN / 4, CUT>, WM * WN,                    \
                     Shape<WM, WN, MG, NT, XS, WS>::kLds)                                                    \
               : run(linear_tile<false, WM, WN, MG, NT, XS, WS, WM * WN / 4, CUT>, WM * WN,                   \
                     Shape<WM, WN, MG, NT, XS, WS>::kLds)
  switch (shape) {
    case kLin256x256: CHORD_LINEAR_SHAPE(2, 4, 8, 4, 3, 2, true);
    case kLin128x256: CHORD_LINEAR_SHAPE(2, 4, 4, 4, 3, 3, false);
    case kLin128x128: CHORD_LINEAR_SHAPE(2, 4, 4, 2, 4, 4, false);
    default: CHORD_LINEAR_SHAPE(2, 4, 2, 2, 6, 6, false);
  }
#undef CHORD_LINEAR_SHAPE
}

}  // namespace chord
