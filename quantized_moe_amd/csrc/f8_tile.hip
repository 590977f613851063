// 8-bit GEMM with block scales, LDS-tiled form for many rows: a workgroup of 8
// waves computes 256 weight rows x up to 256 tokens.
//
// Per 128-wide K chunk the workgroup stages 32 KB of packed weights, the
// tokens' 128-byte row pieces and their scales in LDS, straight from memory
// (buffer_load ... lds), double-buffered: chunk c + 1 lands while chunk c is
// multiplied.  Waves form a 2 x 4 grid (token halves x row quarters); a wave
// owns 64 rows x 16 MG tokens and holds its four weight operands for the whole
// chunk, so LDS reads stay below the matrix time (24 KB per wave and chunk at
// MG = 8, 94 of 128 bytes per clock).  A matrix instruction covers the chunk, its
// result is scaled into the fp32 accumulators one token group later, so the
// four multiply-adds run beside the next matrix instructions.
//
// Token rows lie in LDS as eight 16-byte pieces, piece p of row r at p ^ (r / 2 %
// 8): 128-bit reads go in halves of 8 bytes for 16 lanes (16 rows, one piece) at
// a time, and this key puts them on 16 different bank pairs.
//
// gate_up: 256 interleaved rows are one block of 128 features of h, gate and up,
// so the epilogue quantises that block (maximum over the four row quarters
// through LDS) and stores codes: h never exists in memory in more bits.
#include "f8_common.h"

namespace chord {
namespace {

constexpr int kRsrcWord3 = 0x00020000;
constexpr uint32_t kNoRow = 0xC0000000u;  // byte offset past any row buffer
constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kTiles = 16;                // weight tiles per workgroup
constexpr int kRows = kF8TileRows;        // tokens per workgroup
constexpr int kWBuf = kTiles * kF8BlockBytes;
constexpr int kXBuf = kRows * kF8Block;
constexpr int kXcds = 8;

typedef const __attribute__((address_space(4))) float ConstFloat;

struct Smem {
  uint8_t w[2][kWBuf];
  uint8_t x[2][kXBuf];
  float s[2][kRows];
  uint32_t xoff[kRows];  // byte offset of the row's codes, or kNoRow
  uint32_t soff[kRows];  // byte offset of the row's scales, or kNoRow
  int32_t dst[kRows];    // output row, or -1
  uint32_t amax[4][kRows];
};

__device__ __forceinline__ i32x8_t operand(const uint4& a, const uint4& b) {
  return i32x8_t{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// Buffer resource (raw, out-of-range offsets read as zero) in four scalars.
typedef __attribute__((ext_vector_type(4))) int Rsrc;
__device__ __forceinline__ Rsrc make_rsrc(const void* p, int64_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(p);
  return Rsrc{__builtin_amdgcn_readfirstlane((int)b),
              __builtin_amdgcn_readfirstlane((int)((b >> 32) & 0xFFFF)),
              __builtin_amdgcn_readfirstlane((int)bytes), kRsrcWord3};
}

// Memory straight to LDS: lane l's 16 (4) bytes go to `lds` + 16 (4) l.  Written
// out because the compiler, which sees that such a load writes LDS but not
// which part of it, waits for all of them before the next LDS read; the waits
// here are the explicit ones in run_item.  Nothing is returned in registers.
// (s_nop 4: m0, and scalars that a vector instruction wrote, have to be old
// enough for a memory instruction; the compiler does not look in here.)
__device__ __forceinline__ void load_lds16(uint32_t lds, uint32_t voff, Rsrc r, int soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(lds), "v"(voff), "s"(r), "s"(soff) : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(uint32_t lds, uint32_t voff, Rsrc r, int soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :: "s"(lds), "v"(voff), "s"(r), "s"(soff) : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

struct Item {
  int expert, slice, nrows;
  int64_t row0;  // first row (plain: of the activations; else: aligned row)
};

template <int MG, int KIND>
__device__ __forceinline__ void run_item(const F8GemmArgs& a, Smem& sm, const Item& it,
                                         Rsrc xres, Rsrc sres) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, col = lane & 15;
  const int wm = wave >> 2, wn = wave & 3;
  const int nc = a.n_chunks;
  const int64_t expert_bytes = (int64_t)a.n_tiles * nc * kF8BlockBytes;
  const Rsrc wres = make_rsrc(a.wq + it.expert * expert_bytes, expert_bytes);

  // Token loads: instruction j brings rows 8 j .. 8 j + 7, one row per 8 lanes.
  // Surplus slots repeat the last rows (the same bytes to the same place).
  constexpr int kDma = (4 * MG + kWaves - 1) / kWaves;
  uint32_t xo[kDma];
  int jx[kDma];
#pragma unroll
  for (int i = 0; i < kDma; ++i) {
    jx[i] = min(wave + kWaves * i, 4 * MG - 1);
    const int row = 8 * jx[i] + (lane >> 3);
    xo[i] = sm.xoff[row] + (uint32_t)(((lane & 7) ^ ((row >> 1) & 7)) * 16);
  }
  const int js = min(wave, (32 * MG + 63) / 64 - 1);
  const uint32_t so = sm.soff[js * 64 + lane];
  // Weight loads: two tiles per wave, 1 KB per instruction.
  const int t0 = min(it.slice * kTiles + 2 * wave, a.n_tiles - 1);
  const int t1 = min(it.slice * kTiles + 2 * wave + 1, a.n_tiles - 1);
  const uint32_t lx = lds_address(sm.x[0]), lw = lds_address(sm.w[0] + 2 * wave * kF8BlockBytes);
  const uint32_t ls = lds_address(sm.s[0] + js * 64);
  auto fill = [&](int b, int c) {
#pragma unroll
    for (int i = 0; i < kDma; ++i)
      load_lds16(lx + b * kXBuf + jx[i] * 1024, xo[i], xres, c * kF8Block);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      load_lds16(lw + b * kWBuf + i * 1024, lane * 16 + (i & 1) * 1024, wres,
                 ((i < 2 ? t0 : t1) * nc + c) * kF8BlockBytes);
    load_lds4(ls + b * (kRows * 4), so, sres, c * 4);
  };

  // Weight scales of this wave's four tiles (a gate and an up block, or one).
  // (Constant address space: uniform scalar loads, although the kernel writes.)
  const int blk = KIND == kF8GateUp ? it.slice : min(2 * it.slice + (wn >> 1), a.nb - 1);
  const ConstFloat* s0 = (const ConstFloat*)(a.ws + ((int64_t)it.expert * a.nb + blk) * nc);
  const ConstFloat* s1 = KIND == kF8GateUp ? s0 + (int64_t)(a.nb / 2) * nc : s0;

  f32x4_t acc[4][MG];
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int g = 0; g < MG; ++g) acc[n][g] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const int xrow = (wm * MG * 16 + col) * kF8Block;
  const int x0 = xrow + (((2 * q) ^ ((col >> 1) & 7)) * 16);
  const int x1 = xrow + (((2 * q + 1) ^ ((col >> 1) & 7)) * 16);
  const int w0 = 4 * wn * kF8BlockBytes + lane * 16;

  auto compute = [&](int b, float sw0, float sw1) {
    const uint8_t* xb = sm.x[b];
    const uint8_t* wb = sm.w[b] + w0;
    const float* sb = sm.s[b] + wm * MG * 16 + col;
    auto read_x = [&](int g) {
      return operand(*reinterpret_cast<const uint4*>(xb + x0 + g * 16 * kF8Block),
                     *reinterpret_cast<const uint4*>(xb + x1 + g * 16 * kF8Block));
    };
    i32x8_t wv[4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
      wv[n] = operand(*reinterpret_cast<const uint4*>(wb + n * kF8BlockBytes),
                      *reinterpret_cast<const uint4*>(wb + n * kF8BlockBytes + 1024));
    i32x8_t xv[2];
    float sx[2];
    xv[0] = read_x(0);
    sx[0] = sb[0];
    f32x4_t r[2][4];
    auto scale_in = [&](int g, float s) {
      const float f0 = s * sw0, f1 = KIND == kF8GateUp ? s * sw1 : f0;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        acc[n][g][0] = __builtin_fmaf(r[g & 1][n][0], f0, acc[n][g][0]);
        acc[n][g][1] = __builtin_fmaf(r[g & 1][n][1], f1, acc[n][g][1]);
        acc[n][g][2] = __builtin_fmaf(r[g & 1][n][2], f0, acc[n][g][2]);
        acc[n][g][3] = __builtin_fmaf(r[g & 1][n][3], f1, acc[n][g][3]);
      }
    };
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < MG; ++g) {
      const float sprev = sx[(g + 1) & 1];
      if (g + 1 < MG) {
        xv[(g + 1) & 1] = read_x(g + 1);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n)
        r[g & 1][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv[n], xv[g & 1], zero, 0, 0,
                                                                      0, 0, 0, 0);
      if (g > 0) scale_in(g - 1, sprev);
      if (g + 1 < MG) sx[(g + 1) & 1] = sb[(g + 1) * 16];
      __builtin_amdgcn_sched_barrier(0);
    }
    scale_in(MG - 1, sx[(MG - 1) & 1]);
  };

  fill(0, 0);
  float sw0 = s0[0], sw1 = s1[0];
  for (int c = 0; c < nc; ++c) {
    // Everything issued one chunk ago has landed, in every wave; and no wave
    // reads the other buffer any more.
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));  // vmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    const int cn = c + 1 < nc ? c + 1 : c;
    if (c + 1 < nc) fill((c + 1) & 1, c + 1);
    const float n0 = s0[cn], n1 = s1[cn];
    compute(c & 1, sw0, sw1);
    sw0 = n0;
    sw1 = n1;
  }

  if (KIND == kF8GateUp) {
    // h of this lane: features 8 (4 wn + n) + 2 q + {0, 1} of token col in group g.
    uint32_t m[MG];
#pragma unroll
    for (int g = 0; g < MG; ++g) {
      m[g] = 0;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        acc[n][g][0] = silu_mul(acc[n][g][0], acc[n][g][1]);
        acc[n][g][1] = silu_mul(acc[n][g][2], acc[n][g][3]);
        m[g] = max(m[g], __float_as_uint(acc[n][g][0]) & 0x7FFFFFFFu);
        m[g] = max(m[g], __float_as_uint(acc[n][g][1]) & 0x7FFFFFFFu);
      }
      m[g] = max(m[g], (uint32_t)__shfl_xor((int)m[g], 16, 64));
      m[g] = max(m[g], (uint32_t)__shfl_xor((int)m[g], 32, 64));
      if (q == 0) sm.amax[wn][(wm * MG + g) * 16 + col] = m[g];
    }
    __syncthreads();  // also: every wave is done with the stage buffers
    uint8_t* codes = sm.x[0];  // [tokens][128]
#pragma unroll
    for (int g = 0; g < MG; ++g) {
      const int t = (wm * MG + g) * 16 + col;
      const F8Group f = f8_group(max(max(sm.amax[0][t], sm.amax[1][t]), max(sm.amax[2][t], sm.amax[3][t])));
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float v0 = f.inv != 0.f ? f8_value(f, acc[n][g][0]) : 0.f;
        const float v1 = f.inv != 0.f ? f8_value(f, acc[n][g][1]) : 0.f;
        *reinterpret_cast<uint16_t*>(codes + t * kF8Block + 8 * (4 * wn + n) + 2 * q) =
            (uint16_t)__builtin_amdgcn_cvt_pk_fp8_f32(v0, v1, 0, false);
      }
      if (wn == 0 && q == 0 && sm.dst[t] >= 0)
        a.hs[(int64_t)sm.dst[t] * (a.nb / 2) + it.slice] = f.scale;
    }
    __syncthreads();
    uint8_t* hq = static_cast<uint8_t*>(a.out);
    for (int i = threadIdx.x; i < 32 * MG * 8; i += kThreads) {
      const int t = i >> 3;
      if (sm.dst[t] >= 0)
        *reinterpret_cast<uint4*>(hq + (int64_t)sm.dst[t] * a.ld + it.slice * kF8Block + (i & 7) * 16) =
            *reinterpret_cast<const uint4*>(codes + t * kF8Block + (i & 7) * 16);
    }
    return;
  }

  const int n_base = (it.slice * kTiles + 4 * wn) * 16 + 4 * q;
  const bool wide = a.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 7) == 0;
#pragma unroll
  for (int g = 0; g < MG; ++g) {
    const int64_t d = sm.dst[(wm * MG + g) * 16 + col];
    if (d < 0) continue;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int f = n_base + 16 * n;
      if (KIND == kF8Down) {
        if (f < a.N) *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + d * a.ld + f) = acc[n][g];
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

template <int KIND>
__device__ __forceinline__ void do_item(const F8GemmArgs& a, Smem& sm, const Item& it) {
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
  if (threadIdx.x < kRows) {
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
  const Rsrc xres = make_rsrc(xbase, xrows * pitch), sres = make_rsrc(sbase, xrows * spitch);
  switch ((it.nrows + 31) / 32) {
    case 1: run_item<1, KIND>(a, sm, it, xres, sres); break;
    case 2: run_item<2, KIND>(a, sm, it, xres, sres); break;
    case 3: run_item<3, KIND>(a, sm, it, xres, sres); break;
    case 4: run_item<4, KIND>(a, sm, it, xres, sres); break;
    case 5: run_item<5, KIND>(a, sm, it, xres, sres); break;
    case 6: run_item<6, KIND>(a, sm, it, xres, sres); break;
    case 7: run_item<7, KIND>(a, sm, it, xres, sres); break;
    default: run_item<8, KIND>(a, sm, it, xres, sres); break;
  }
}

// Persistent workgroups.  Workgroup b runs on XCD b % 8.
template <int KIND>
__global__ __launch_bounds__(kThreads, 2) void f8_tile(F8GemmArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  Smem& sm = *reinterpret_cast<Smem*>(smem);
  const int slices = (a.n_tiles + kTiles - 1) / kTiles;
  const int xcd = blockIdx.x % kXcds, local = blockIdx.x / kXcds;
  const int per_xcd = (gridDim.x + kXcds - 1 - xcd) / kXcds;
  if (KIND == kF8Plain) {
    // Runs of `per_xcd` consecutive items go to one XCD at a time.  Items walk
    // blocks of 8 token tiles slice by slice, so those that run together share
    // few token tiles and few slices through their L2.
    const int64_t tiles = (a.a_rows + kRows - 1) / kRows;
    const int64_t total = tiles * slices;
    const int run = gridDim.x / kXcds;  // (the grid is a multiple of 8)
    for (int64_t i = (int64_t)xcd * run + local; i < total; i += gridDim.x) {
      const int64_t block = i / (8 * slices);
      const int wide = (int)min((int64_t)8, tiles - block * 8);
      const int rest = (int)(i - block * 8 * slices);
      Item it;
      it.expert = 0;
      it.slice = rest / wide;
      it.row0 = (block * 8 + rest % wide) * kRows;
      it.nrows = (int)min((int64_t)kRows, a.a_rows - it.row0);
      do_item<KIND>(a, sm, it);
    }
  } else {
    // The tile list comes in 8 groups of balanced size, one per XCD; all slices
    // of a tile stay on one XCD, which reads its token rows once.
    const int G = gridDim.x < kXcds ? (int)gridDim.x : kXcds;
    for (int g = xcd; g < kTileGroups; g += G) {
      const int t0 = a.status->group_start[g];
      const int n = (a.status->group_start[g + 1] - t0) * slices;
      for (int j = local; j < n; j += per_xcd) {
        const TileDesc td = a.tiles[t0 + j / slices];
        Item it;
        it.expert = td.expert;
        it.slice = j % slices;
        it.row0 = td.row_begin;
        it.nrows = min(td.nrows, kRows);
        do_item<KIND>(a, sm, it);
      }
    }
  }
}

}  // namespace

hipError_t launch_f8_tile(const F8GemmArgs& a, hipStream_t stream) {
  // One workgroup per CU (LDS); a multiple of 8 so that every XCD gets a share.
  const int grid = a.num_cus >= 8 ? a.num_cus / 8 * 8 : 8;
  const dim3 g((unsigned)grid), b(kThreads);
  auto run = [&](auto kernel) {
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)sizeof(Smem));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, g, b, sizeof(Smem), stream, a);
    return hipGetLastError();
  };
  if (a.kind == kF8Plain) return run(f8_tile<kF8Plain>);
  if (a.kind == kF8GateUp) return run(f8_tile<kF8GateUp>);
  return run(f8_tile<kF8Down>);
}

}  // namespace chord
