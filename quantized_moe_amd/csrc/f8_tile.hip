// 8-bit GEMM with block scales, LDS-tiled form for many rows: a workgroup of 8
// waves computes 256 weight rows x up to 256 tokens.
//
// Wave w owns weight tiles 2 w and 2 w + 1 (16 rows each) and every token.  Its
// weights go straight from memory into registers; the tokens' 128-byte row pieces
// and their scales go straight from memory into LDS (buffer_load ... lds), three
// chunks of 128 along K ahead, in four buffers.  (With weights in LDS too only
// one chunk fits in flight, and the loads alone took as long as the products.)
// 8192 x 4096 x 7168 takes 203 to 212 us, 2.3 PFLOP/s, matrix units busy for 57 to 60 %
// of 1.85 GHz, to which the clock falls under them; weights of 48 experts of 4096 x 7168
// with 170 rows each 330 us, 4.5 TB/s of them.
//
// A matrix instruction covers the chunk; its result is scaled into the fp32
// accumulators one token group later, so the multiply-adds run beside the next
// matrix instructions.  Nothing drains at the end of a chunk: the one barrier of
// chunk c stands in its middle.  Behind it every wave knows that chunk c + 1 has
// landed, so the last group already reads the next chunk's first operand, and
// that chunk c - 1 is read, so its buffer takes chunk c + 3.
//
// Token rows lie in LDS as eight 16-byte pieces, piece p of row r at p ^ key(r).
// A 128-bit read takes 8 lanes at a time, four neighbours of one operand
// quarter and four of the next (lanes 0-3 with 20-23, 4-7 with 16-19, ...), so
// four rows' piece p and the next four's piece p + 2: the key (r % 8 with its two
// low bits swapped) puts those, and also the 16 lanes of two such groups over
// 64 banks, on different banks.
//
// gate_up: 256 interleaved rows are one block of 128 features of h, gate and up,
// so the epilogue quantises that block (maximum over the eight waves through
// LDS) and stores codes: h never exists in memory in more bits.  Where rows are few it
// sums its products in fp32 (f8_exact_product says why): over alignment blocks each
// product widens its operands, over large tiles the chunk's weights are widened once.
#include <type_traits>

#include "f8_common.h"

namespace chord {
namespace {

constexpr int kRsrcWord3 = 0x00020000;
constexpr uint32_t kNoRow = 0xC0000000u;  // byte offset past any row buffer
constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kTiles = 16;                // weight tiles per workgroup
constexpr int kStages = 4;                // chunks: one in use, three on their way
constexpr int kXcds = 8;
constexpr int kStreamAux = 2;             // non-temporal
constexpr int kEvery = 16;                // EXACT: every group of a tall tile

typedef const __attribute__((address_space(4))) float ConstFloat;

// ROWS: tokens per workgroup at most.
template <int ROWS>
struct Smem {
  uint8_t x[kStages][ROWS * kF8Block];
  uint32_t xoff[ROWS];  // byte offset of the row's codes, or kNoRow
  uint32_t soff[ROWS];  // byte offset of the row's scales, or kNoRow
  int32_t dst[ROWS];    // output row, or -1
  uint32_t amax[kWaves][ROWS];
};

__device__ __forceinline__ i32x8_t operand(u32x4_t a, u32x4_t b) {
  return i32x8_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// Scales of four chunks, and of the next four: the buffer changes at run time,
// so it is an object of its own, which no other load can be taken to touch.
template <int ROWS>
struct Scales {
  float s[2][ROWS][4];
};

// Memory straight to LDS, lane l's 4 bytes to `lds` + 4 l.  Written out because
// the compiler, which sees that such a load writes LDS but not which half of
// the scales, would wait for it before reading the other half; the barrier's
// count covers it.  Nothing is returned in registers.  (s_nop 4: m0, and
// scalars that a vector instruction wrote, have to be old enough for a memory
// instruction; the compiler does not look in here.)
typedef __attribute__((ext_vector_type(4))) int Rsrc;
__device__ __forceinline__ void load_lds4(uint32_t lds, uint32_t voff, Rsrc r, int soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :: "s"(lds), "v"(voff), "s"(r), "s"(soff) : "memory", "m0");
}
__device__ __forceinline__ Rsrc make_rsrc(const void* p, int64_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(p);
  return Rsrc{__builtin_amdgcn_readfirstlane((int)b),
              __builtin_amdgcn_readfirstlane((int)((b >> 32) & 0xFFFF)),
              __builtin_amdgcn_readfirstlane((int)bytes), kRsrcWord3};
}

__device__ __forceinline__ int swz(int r) { return (r & 4) | ((r & 1) << 1) | ((r >> 1) & 1); }

struct Item {
  int expert, slice, nrows;
  int64_t row0;  // first row (plain: of the activations; else: aligned row)
  int part;      // plain: part of K (of a.parts)
};

// One item with G = 2 MG token groups of 16.
template <int MG, int KIND, int ROWS, int EXACT>
__device__ __forceinline__ void run_item(const F8GemmArgs& a, Smem<ROWS>& sm, Scales<ROWS>& scales,
                                         const Item& it, __amdgpu_buffer_rsrc_t xres, Rsrc sres) {
  constexpr int G = 2 * MG;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, col = lane & 15;
  // Chunks c_lo .. c_lo + nc of the row's n_chunks.
  const int c_lo = KIND == kF8Plain ? (int)((int64_t)a.n_chunks * it.part / a.parts) : 0;
  const int nc = KIND == kF8Plain ? (int)((int64_t)a.n_chunks * (it.part + 1) / a.parts) - c_lo : a.n_chunks;
  const int64_t expert_bytes = (int64_t)a.n_tiles * a.n_chunks * kF8BlockBytes;
  const __amdgpu_buffer_rsrc_t wres = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(a.wq + it.expert * expert_bytes), 0, (int)expert_bytes, kRsrcWord3);

  // Token loads: instruction j brings rows 8 j .. 8 j + 7, one row per 8 lanes.
  // Surplus slots repeat the last rows (the same bytes to the same place), so
  // that every wave issues the same number of loads.
  constexpr int kDma = (2 * G + kWaves - 1) / kWaves;
  uint32_t xo[kDma];
  int jx[kDma];
#pragma unroll
  for (int i = 0; i < kDma; ++i) {
    jx[i] = min(wave + kWaves * i, 2 * G - 1);
    const int row = 8 * jx[i] + (lane >> 3);
    xo[i] = sm.xoff[row] + (uint32_t)(c_lo * kF8Block + ((lane & 7) ^ swz(row)) * 16);
  }
  // Scales come for four chunks at a time, 16 rows x 4 chunks per instruction:
  // fetched chunk by chunk, every row's 4 bytes are a memory request of their own,
  // more of them than the rows themselves take (gate_up of 8192 tokens on 48
  // experts: 381 us so, 340 without a request a row).
  // (Fewer than 256 rows: the surplus waves repeat rows, to the same places.)
  uint32_t so[2];
  uint32_t ls[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = (8 * i + wave) % (ROWS / 16);
    so[i] = sm.soff[m * 16 + (lane >> 2)] + (c_lo + (lane & 3)) * 4;
    ls[i] = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) float*)&scales.s[0][m * 16][0];
  }
  // Weights: tiles past the last one of a partial slice repeat it.
  const int t0 = min(it.slice * kTiles + 2 * wave, a.n_tiles - 1);
  const int t1 = min(it.slice * kTiles + 2 * wave + 1, a.n_tiles - 1);
  const int o0 = f8_block(t0, c_lo, a.n_tiles, a.n_chunks) * kF8BlockBytes;
  const int o1 = f8_block(t1, c_lo, a.n_tiles, a.n_chunks) * kF8BlockBytes;
  const int wstep = f8_slice_width(t0, a.n_tiles) * kF8BlockBytes;  // chunk to chunk
  // Weight registers: as far ahead as the tokens where the accumulators leave
  // room, else one chunk; two where weights are widened when a chunk begins, which
  // frees their registers for those of the next but one.
  constexpr bool kWiden = EXACT == kEvery;
  constexpr int WR = G <= 12 && !kWiden ? 4 : 2;
  constexpr int kAhead = WR == 4 ? 3 : kWiden ? 2 : 1;
  u32x4_t w[WR][2][2];
  constexpr int kW = 4;  // loads of weights per chunk
  auto load_x = [&](int j, int b, int c) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        xres, (__attribute__((address_space(3))) void*)(sm.x[b] + jx[j] * 1024), 16, xo[j],
        c * kF8Block, 0, 0);
  };
  // Half i of the scales of chunks c0 .. c0 + 3.  (Past a row's end: other rows',
  // never used, or zeros.)
  auto load_s = [&](int i, int half, int c0) {
    load_lds4(ls[i] + half * (ROWS * 16), so[i], sres, c0 * 4);
  };
  auto load_w = [&](int j, int b, int c) {
    w[b][j >> 1][j & 1] = __builtin_amdgcn_raw_buffer_load_b128(
        wres, lane * 16 + (j & 1) * 1024, (j >> 1 ? o1 : o0) + c * wstep, kStreamAux);
  };

  // Weight scales of this wave's two tiles (a gate and an up block, or one).
  // (Constant address space: uniform scalar loads, although the kernel writes.)
  const int blk = KIND == kF8GateUp ? it.slice : min(2 * it.slice + (wave >> 2), a.nb - 1);
  const ConstFloat* s0 = (const ConstFloat*)(a.ws + ((int64_t)it.expert * a.nb + blk) * a.n_chunks + c_lo);
  const ConstFloat* s1 = KIND == kF8GateUp ? s0 + (int64_t)(a.nb / 2) * a.n_chunks : s0;

  f32x4_t acc[2][G];
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int g = 0; g < G; ++g) acc[n][g] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const int x0 = col * kF8Block + (((2 * q) ^ swz(col)) * 16);
  const int x1 = col * kF8Block + (((2 * q + 1) ^ swz(col)) * 16);

  auto read_x = [&](int b, int g) {
    const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(sm.x[b] + x0 + g * 16 * kF8Block);
    const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(sm.x[b] + x1 + g * 16 * kF8Block);
    return operand(lo, hi);
  };
  auto read_s = [&](int half, int ph, int g) { return scales.s[half][g * 16 + col][ph]; };
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  // EXACT: f8_exact_product for this many groups, the rest of a block being empty
  // (kEvery: for all, below).
  // (With a constant 1 the widened weights of the next products would be kept, and
  // spill.)
  auto product = [&](i32x8_t wv, i32x8_t x, int g) {
    if constexpr (EXACT > 0) {
      if (g >= EXACT) return zero;
      float one = 1.f;
      asm volatile("" : "+s"(one));
      return f8_exact_product(wv, x, one);
    } else {
      return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, x, zero, 0, 0, 0, 0, 0, 0);
    }
  };
  i32x8_t xv[2];
  float sx[2];
  f32x4_t r[2][2] = {{zero, zero}, {zero, zero}};
  float f0 = 0.f, f1 = 0.f;  // factors of the results in r
  auto scale_in = [&](int n, int g) {
    if (EXACT > 0 && g >= EXACT) return;
    acc[n][g][0] = __builtin_fmaf(r[g & 1][n][0], f0, acc[n][g][0]);
    acc[n][g][1] = __builtin_fmaf(r[g & 1][n][1], f1, acc[n][g][1]);
    acc[n][g][2] = __builtin_fmaf(r[g & 1][n][2], f0, acc[n][g][2]);
    acc[n][g][3] = __builtin_fmaf(r[g & 1][n][3], f1, acc[n][g][3]);
  };
  auto barrier = [&](auto outstanding) {  // ... loads of this wave may be on their way
    constexpr int vm = decltype(outstanding)::value;
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((vm & 15) | (7 << 4) | (15 << 8) | ((vm >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  float sw0 = s0[0], sw1 = s1[0];

  // Chunk c in buffer b (= c % 4; its group 0 and that group's scales are in
  // registers; half: which of the scales are its own).
  // In the loop, load indices past the end repeat the last chunk, so every chunk
  // issues the same loads and the counts are exact.  At the barrier only these
  // may be younger than the tokens of chunk c + 1: a chunk's weights, the tokens
  // of chunk c + 2 with (in two chunks of four) half of the next scales in front
  // of them, and this chunk's weights.
  // Behind the loop (last) nothing is loaded any more, but for the weights that a
  // chunk there needs where they are one or two chunks ahead; the counts there take
  // no weights for granted, since the compiler drops loads whose registers nobody
  // reads.
  // (With one chunk ahead the chunk's own weights, already waited for, are
  // younger than the tokens of chunk c + 1.)
  constexpr int kBehind = 2 * kW + kDma;
  constexpr int kBehindLast = kAhead == 3 ? 0 : kW;
  auto chunk = [&](int b, int c, int half, auto is_last) {
    constexpr bool last = decltype(is_last)::value;
    const int nb = (b + 1) % kStages, fb = (b + 3) % kStages;
    const int c1 = min(c + 1, nc - 1), c3 = min(c + 3, nc - 1), cw = min(c + kAhead, nc - 1);
    const float n0 = s0[c1], n1 = s1[c1];
    const i32x8_t w0 = operand(w[b % WR][0][0], w[b % WR][0][1]);
    const i32x8_t w1 = operand(w[b % WR][1][0], w[b % WR][1][1]);
    half8_t h[2][4];
    if constexpr (kWiden) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[0][j] = f8_widen(w0[2 * j], w0[2 * j + 1], 1.f);
        h[1][j] = f8_widen(w1[2 * j], w1[2 * j + 1], 1.f);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (EXACT > 0) {
      if (!last || (kWiden && b == 0))
#pragma unroll
        for (int j = 0; j < kW; ++j) load_w(j, (b + kAhead) % WR, cw);
      __builtin_amdgcn_sched_barrier(0);
    }
    // Fences after every matrix instruction keep this order: one matrix
    // instruction, then the multiply-adds of the one two places before it (left
    // alone, the compiler puts those right behind their own instruction, with
    // waits for its result).
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (g == G / 2 && !last && (b == 1 || b == 2)) barrier(std::integral_constant<int, kBehind + 1>{});
      if (g == G / 2 && !last && (b == 0 || b == 3)) barrier(std::integral_constant<int, kBehind>{});
      if (g == G / 2 && last && b == 0) barrier(std::integral_constant<int, kBehindLast + kDma>{});
      if (g == G / 2 && last && b == 1) barrier(std::integral_constant<int, kWiden ? 0 : kBehindLast>{});
      if constexpr (kWiden) {
        const i32x8_t x = xv[g & 1];
        xv[(g + 1) & 1] = g + 1 < G ? read_x(b, g + 1) : read_x(nb, 0);
        f32x4_t p0 = zero, p1 = zero;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const half8_t xh = f8_widen(x[2 * j], x[2 * j + 1], 1.f);
          p0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(h[0][j], xh, p0, 0, 0, 0);
          p1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(h[1][j], xh, p1, 0, 0, 0);
          if (j == 0) scale_in(0, (g + G - 1) % G);
          if (j == 1) scale_in(1, (g + G - 1) % G);
        }
        r[g & 1][0] = p0;
        r[g & 1][1] = p1;
        f0 = sx[g & 1] * sw0;
        f1 = sx[g & 1] * sw1;
      } else if constexpr (EXACT > 0) {
        // (Scaled at once: the registers that hold results over a group would spill.)
        r[g & 1][0] = product(w0, xv[g & 1], g);
        r[g & 1][1] = product(w1, xv[g & 1], g);
        xv[(g + 1) & 1] = g + 1 < G ? read_x(b, g + 1) : read_x(nb, 0);
        f0 = sx[g & 1] * sw0;
        f1 = sx[g & 1] * sw1;
        scale_in(0, g);
        scale_in(1, g);
      } else {
        r[g & 1][0] = product(w0, xv[g & 1], g);
        xv[(g + 1) & 1] = g + 1 < G ? read_x(b, g + 1) : read_x(nb, 0);
        scale_in(0, (g + G - 1) % G);
        __builtin_amdgcn_sched_barrier(0);
        r[g & 1][1] = product(w1, xv[g & 1], g);
        scale_in(1, (g + G - 1) % G);
        f0 = sx[g & 1] * sw0;
        f1 = KIND == kF8GateUp ? sx[g & 1] * sw1 : f0;
      }
      sx[(g + 1) & 1] = g + 1 < G ? read_s(half, b, g + 1) : read_s(b == 3 ? 1 - half : half, nb, 0);
#pragma unroll
      for (int j = 0; j < kW; ++j)
        if (EXACT == 0 && (!last || WR == 2) && g < G / 2 && j * (G / 2) / kW == g) load_w(j, (b + kAhead) % WR, cw);
      if (!last && g == G / 2 && b < 2) load_s(b, 1 - half, c - b + 4);
#pragma unroll
      for (int j = 0; j < kDma; ++j)
        if (!last && g >= G / 2 && j * (G / 2) / kDma == g - G / 2) load_x(j, fb, c3);
      __builtin_amdgcn_sched_barrier(0);
    }
    sw0 = n0;
    sw1 = n1;
  };

  auto load_all_x = [&](int c) {
#pragma unroll
    for (int j = 0; j < kDma; ++j) load_x(j, c, min(c, nc - 1));
  };
  auto load_all_w = [&](int c) {
#pragma unroll
    for (int j = 0; j < kW; ++j) load_w(j, c, min(c, nc - 1));
  };
  // (Weights stand between the tokens of chunks 1 and 2, as the count at the
  // barrier has it.)
#pragma unroll
  for (int c = 0; c + 1 < kAhead; ++c) load_all_w(c);
  load_s(0, 0, 0);
  load_s(1, 0, 0);
  load_all_x(0);
  __builtin_amdgcn_sched_barrier(0);
  load_all_x(1);
  __builtin_amdgcn_sched_barrier(0);
  load_all_w(kAhead - 1);
  __builtin_amdgcn_sched_barrier(0);
  load_all_x(2);
  barrier(std::integral_constant<int, kW + 2 * kDma>{});
  xv[0] = read_x(0, 0);
  sx[0] = read_s(0, 0, 0);
  int c = 0, half = 0;
  const std::false_type in_loop;
  const std::true_type behind_loop;
  for (; c + 3 < nc; c += 4) {
    chunk(0, c, half, in_loop);
    chunk(1, c + 1, half, in_loop);
    chunk(2, c + 2, half, in_loop);
    chunk(3, c + 3, half, in_loop);
    half = 1 - half;
  }
  // Where a chunk behind the loop is missing its weights (repeats of the last
  // chunk's) are read all the same: a load without a reader on some path could be
  // dropped or moved there, and the counts in the loop rely on every one.
  auto used = [&](int b) {
#pragma unroll
    for (int j = 0; j < kW; ++j) asm volatile("" ::"v"(w[b % WR][j >> 1][j & 1]));
  };
  if (c < nc) chunk(0, c, half, behind_loop);
  else used(0);
  if (c + 1 < nc) chunk(1, c + 1, half, behind_loop);
  else used(1);
  if (c + 2 < nc) chunk(2, c + 2, half, behind_loop);
  else used(2);
  if (EXACT == 0 || kWiden) {
    scale_in(0, G - 1);
    scale_in(1, G - 1);
  }
  // The repeated loads at the end land before their buffers are used again.
  __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));

  if (KIND == kF8GateUp) {
    // h of this lane: features 8 (2 wave + n) + 2 q + {0, 1} of token col in group g.
#pragma unroll
    for (int g = 0; g < G; ++g) {
      uint32_t m = 0;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        acc[n][g][0] = silu_mul(acc[n][g][0], acc[n][g][1]);
        acc[n][g][1] = silu_mul(acc[n][g][2], acc[n][g][3]);
        m = max(m, __float_as_uint(acc[n][g][0]) & 0x7FFFFFFFu);
        m = max(m, __float_as_uint(acc[n][g][1]) & 0x7FFFFFFFu);
      }
      m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
      if (q == 0) sm.amax[wave][g * 16 + col] = m;
    }
    __syncthreads();  // also: every wave is done with the token buffers
    uint8_t* codes = sm.x[0];  // [tokens][128]
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int t = g * 16 + col;
      uint32_t m = sm.amax[0][t];
#pragma unroll
      for (int u = 1; u < kWaves; ++u) m = max(m, sm.amax[u][t]);
      const F8Group f = f8_group(m);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float v0 = f.inv != 0.f ? f8_value(f, acc[n][g][0]) : 0.f;
        const float v1 = f.inv != 0.f ? f8_value(f, acc[n][g][1]) : 0.f;
        *reinterpret_cast<uint16_t*>(codes + t * kF8Block + 8 * (2 * wave + n) + 2 * q) =
            (uint16_t)__builtin_amdgcn_cvt_pk_fp8_f32(v0, v1, 0, false);
      }
      if (wave == 0 && q == 0 && sm.dst[t] >= 0)
        a.hs[(int64_t)sm.dst[t] * (a.nb / 2) + it.slice] = f.scale;
    }
    __syncthreads();
    uint8_t* hq = static_cast<uint8_t*>(a.out);
    for (int i = threadIdx.x; i < 16 * G * 8; i += kThreads) {
      const int t = i >> 3;
      if (sm.dst[t] >= 0)
        *reinterpret_cast<uint4*>(hq + (int64_t)sm.dst[t] * a.ld + it.slice * kF8Block + (i & 7) * 16) =
            *reinterpret_cast<const uint4*>(codes + t * kF8Block + (i & 7) * 16);
    }
    return;
  }

  if constexpr (KIND == kF8Down) {
    // A wave's two tiles are one block of y: no wave waits for another.  (8192
    // tokens on 48 experts, 117 MB of y: 205 us; 218 staged through LDS in units
    // per 256 outputs, 231 in fp32.  About 35 us of it are the stores, which all
    // workgroups issue at the same time and the next item's loads queue behind.)
    if ((it.slice * kTiles + 2 * wave) * 16 >= a.N) return;  // (N is a multiple of 128)
    const int block = it.slice * (kTiles / 2) + wave, blocks = a.N / kF8YBlock;
    uint16_t* y = static_cast<uint16_t*>(a.out) + block * kF8YBlock + 16 * (q & 1) + 8 * (q >> 1);
#pragma unroll
    for (int g0 = 0; g0 < G; g0 += 4) {
      uint32_t e = 0;  // lane quarter q: exponent of group g0 + q
#pragma unroll
      for (int g = g0; g < g0 + 4 && g < G; ++g) {
        u32x4_t v;
        const uint32_t eg = f8_y_pack(acc[0][g], acc[1][g], v);
        const int64_t d = sm.dst[g * 16 + col];
        if (d >= 0) *reinterpret_cast<u32x4_t*>(y + d * a.ld) = v;
        e = q == g - g0 ? eg : e;
      }
      const int64_t d = g0 + q < G ? sm.dst[(g0 + q) * 16 + col] : -1;
      if (d >= 0) a.yu[d * blocks + block] = (uint8_t)e;
    }
    return;
  }

  const int n_base = (it.slice * kTiles + 2 * wave) * 16 + 4 * q;
  const bool wide = a.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 7) == 0;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t d = sm.dst[g * 16 + col];
    if (d < 0) continue;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int f = n_base + 16 * n;
      if (KIND == kF8Plain && a.parts > 1) {
        if (f < a.n_tiles * 16)
          *reinterpret_cast<f32x4_t*>(a.partials + ((int64_t)it.part * a.a_rows + it.row0 + d) * (a.n_tiles * 16) +
                                      f) = acc[n][g];
      } else {
        uint16_t* p = static_cast<uint16_t*>(a.out) + (it.row0 + d) * a.ld + f;
        if (wide && f + 4 <= a.N) {
          *reinterpret_cast<uint2*>(p) =
              make_uint2(pk_bf16(acc[n][g][0], acc[n][g][1]), pk_bf16(acc[n][g][2], acc[n][g][3]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (f + i < a.N) p[i] = to_bf16(acc[n][g][i]);
        }
      }
    }
  }
}

template <int KIND, int ROWS, int EXACT>
__device__ __forceinline__ void do_item(const F8GemmArgs& a, Smem<ROWS>& sm, Scales<ROWS>& scales,
                                        const Item& it) {
  const int64_t pitch = (int64_t)a.n_chunks * kF8Block, spitch = (int64_t)a.n_chunks * 4;
  __syncthreads();  // the last item's epilogue is done with the tables
  const uint8_t* xbase = a.aq;
  const uint8_t* sbase = reinterpret_cast<const uint8_t*>(a.as);
  int64_t xrows = a.a_rows;
  if (KIND == kF8Plain) {  // rows of a tile from its own base: any number of rows
    xbase += it.row0 * pitch;
    sbase += it.row0 * spitch;
    xrows = it.nrows;
  }
  if (threadIdx.x < ROWS) {
    const int m = threadIdx.x;
    int64_t src = -1, dst = -1;
    if (m < it.nrows) {
      if (KIND == kF8Plain) {
        src = dst = m;
      } else {
        const int64_t R = it.row0 + m;
        const int64_t f = a.sorted_ids[R];
        if (f >= 0 && f < a.n_flat) {
          src = KIND == kF8GateUp ? f / a.topk : R;
          dst = KIND == kF8GateUp ? R : f;
        }
      }
    }
    sm.xoff[m] = src >= 0 ? (uint32_t)(src * pitch) : kNoRow;
    sm.soff[m] = src >= 0 ? (uint32_t)(src * spitch) : kNoRow;
    sm.dst[m] = (int32_t)dst;
  }
  __syncthreads();
  const __amdgpu_buffer_rsrc_t xres =
      __builtin_amdgcn_make_buffer_rsrc((void*)xbase, 0, (int)(xrows * pitch), kRsrcWord3);
  const Rsrc sres = make_rsrc(sbase, xrows * spitch);
  if constexpr (ROWS == kF8SmallRows) {
    run_item<1, KIND, ROWS, EXACT>(a, sm, scales, it, xres, sres);
  } else {
    switch ((it.nrows + 31) / 32) {
      case 1: run_item<1, KIND, ROWS, EXACT>(a, sm, scales, it, xres, sres); break;
      case 2: run_item<2, KIND, ROWS, EXACT>(a, sm, scales, it, xres, sres); break;
      case 3: run_item<3, KIND, ROWS, EXACT>(a, sm, scales, it, xres, sres); break;
      case 4: run_item<4, KIND, ROWS, EXACT>(a, sm, scales, it, xres, sres); break;
      case 5: run_item<5, KIND, ROWS, EXACT>(a, sm, scales, it, xres, sres); break;
      case 6: run_item<6, KIND, ROWS, EXACT>(a, sm, scales, it, xres, sres); break;
      case 7: run_item<7, KIND, ROWS, EXACT>(a, sm, scales, it, xres, sres); break;
      default:
        if constexpr (KIND == kF8Plain) run_item<8, KIND, ROWS, EXACT>(a, sm, scales, it, xres, sres);
    }
  }
}

// out[m, n] = bf16(sum of the K parts, ascending).
__global__ __launch_bounds__(256) void f8_add_parts(F8GemmArgs a) {
  const int pitch = a.n_tiles * 16, quads = pitch / 4;
  const bool wide = a.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 7) == 0;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.a_rows * quads;
       i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / quads;
    const int n = (int)(i - m * quads) * 4;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int p = 0; p < a.parts; ++p)
      v += *reinterpret_cast<const f32x4_t*>(a.partials + ((int64_t)p * a.a_rows + m) * pitch + n);
    uint16_t* o = static_cast<uint16_t*>(a.out) + m * a.ld + n;
    if (wide && n + 4 <= a.N) {
      *reinterpret_cast<uint2*>(o) = make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (n + u < a.N) o[u] = to_bf16(v[u]);
    }
  }
}

// Persistent workgroups.  Workgroup b runs on XCD b % 8.  OCC: waves per SIMD.
// EXACT: token groups whose products are summed in fp32 (gate_up: 1 or 2 over
// alignment blocks, kEvery over tall tiles).
template <int KIND, int ROWS, int OCC, int EXACT>
__global__ __launch_bounds__(kThreads, OCC) void f8_tile(F8GemmArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  Smem<ROWS>& sm = *reinterpret_cast<Smem<ROWS>*>(smem);
  __shared__ __attribute__((aligned(16))) Scales<ROWS> scales;
  const int slices = (a.n_tiles + kTiles - 1) / kTiles;
  const int xcd = blockIdx.x % kXcds, local = blockIdx.x / kXcds;
  const int run = gridDim.x / kXcds;  // (the grid is a multiple of 8)
  if (KIND == kF8Plain) {
    // Runs of `run` consecutive items go to one XCD at a time.  Items walk
    // blocks of 8 token tiles slice by slice, so those that run together share
    // few token tiles and few slices through their L2.
    const int rows = a.tile_rows;
    const int64_t tiles = (a.a_rows + rows - 1) / rows;
    const int64_t whole = tiles * slices;
    for (int64_t i = (int64_t)xcd * run + local; i < whole * a.parts; i += gridDim.x) {
      const int64_t u = i % whole, block = u / (8 * slices);
      const int wide = (int)min((int64_t)8, tiles - block * 8);
      const int rest = (int)(u - block * 8 * slices);
      Item it;
      it.expert = 0;
      it.part = (int)(i / whole);
      it.slice = rest / wide;
      it.row0 = (block * 8 + rest % wide) * rows;
      it.nrows = (int)min((int64_t)rows, a.a_rows - it.row0);
      do_item<KIND, ROWS, EXACT>(a, sm, scales, it);
    }
  } else if (ROWS == kF8SmallRows) {
    // Tiles are the alignment blocks (at most ROWS rows), block t and all its
    // slices on XCD t % 8.
    const int64_t used = max((int64_t)0, min((int64_t)*a.ntpp, a.max_padded));
    const int blocks = (int)(used / a.block_m);
    const int mine = xcd < blocks ? (blocks - xcd + kXcds - 1) / kXcds : 0;
    for (int64_t j = local; j < (int64_t)mine * slices; j += run) {
      const int t = (int)(j / slices) * kXcds + xcd;
      Item it;
      it.expert = a.expert_ids[t];
      it.slice = (int)(j % slices);
      it.row0 = (int64_t)t * a.block_m;
      it.nrows = a.block_m;
      if (it.expert < 0 || it.expert >= a.num_experts) continue;  // uniform
      do_item<KIND, ROWS, EXACT>(a, sm, scales, it);
    }
  } else {
    // The tile list comes in 8 groups of balanced size, one per XCD; all slices
    // of a tile stay on one XCD, which reads its token rows once.  Items that
    // fill no whole round of the XCD's workgroups are cut by rows into as many
    // pieces as fill one.
    const int t0 = a.status->group_start[xcd];
    const int n = (a.status->group_start[xcd + 1] - t0) * slices;
    const int whole = n / run * run, rest = n - whole;
    const int pieces = rest > 0 ? run / rest : 1;
    for (int j = local; j < whole + rest * pieces; j += run) {
      const int u = j - whole, i = u < 0 ? j : whole + u / pieces;
      const TileDesc td = a.tiles[t0 + i / slices];
      Item it;
      it.expert = td.expert;
      it.slice = i % slices;
      it.row0 = td.row_begin;
      it.nrows = min(td.nrows, kF8MoeTileRows);
      if (u >= 0) {
        const int rows = ((it.nrows + pieces - 1) / pieces + 31) / 32 * 32;
        const int begin = u % pieces * rows;
        if (begin >= it.nrows) continue;  // uniform
        it.row0 += begin;
        it.nrows = min(rows, it.nrows - begin);
      }
      do_item<KIND, ROWS, EXACT>(a, sm, scales, it);
    }
  }
}

}  // namespace

hipError_t launch_f8_tile(const F8GemmArgs& a, bool small, hipStream_t stream) {
  // A multiple of 8 workgroups, so that every XCD gets the same share: one per
  // CU, and two in the small form.
  const int cus = a.num_cus >= 8 ? a.num_cus / 8 * 8 : 8;
  auto run = [&](auto kernel, int per_cu, size_t lds) {
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(cus * per_cu)), dim3(kThreads), lds, stream, a);
    return hipGetLastError();
  };
  constexpr int R = kF8TileRows, S = kF8SmallRows;
  if (a.kind == kF8Plain) {
    const hipError_t e = run(f8_tile<kF8Plain, R, 2, 0>, 1, sizeof(Smem<R>));
    if (e != hipSuccess || a.parts <= 1) return e;
    const int64_t n = (a.a_rows * (a.n_tiles * 4) + 255) / 256, most = (int64_t)a.num_cus * 16;
    hipLaunchKernelGGL(f8_add_parts, dim3((unsigned)(n < most ? n : most)), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  if (a.kind == kF8GateUp)
    return !small             ? a.exact ? run(f8_tile<kF8GateUp, R, 2, kEvery>, 1, sizeof(Smem<R>))
                                         : run(f8_tile<kF8GateUp, R, 2, 0>, 1, sizeof(Smem<R>))
           : a.block_m <= 16 ? run(f8_tile<kF8GateUp, S, 4, 1>, 2, sizeof(Smem<S>))
                             : run(f8_tile<kF8GateUp, S, 4, 2>, 2, sizeof(Smem<S>));
  return small ? run(f8_tile<kF8Down, S, 4, 0>, 2, sizeof(Smem<S>))
               : run(f8_tile<kF8Down, R, 2, 0>, 1, sizeof(Smem<R>));
}

}  // namespace chord
