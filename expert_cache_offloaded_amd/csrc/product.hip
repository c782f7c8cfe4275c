// mc_mxfp4_matmul and mc_grouped_matmul: products of rows (bf16 or MXFP4) with expert matrices
// (bf16 or MXFP4), grouped by expert.
//
// The weights are the MFMA's A operand and the rows its B operand, so a lane's four results
// of one instruction are four consecutive output columns of one row.  bf16 operands: MFMA
// 16x16x32, lane l holds 8 elements of row l % 16 from k = 8 (l / 16).  MXFP4 operands: the
// scaled MFMA 16x16x128, lane l holds the whole 32-element block l / 16 of row l % 16 and its
// scale byte, so both formats read 16 bytes per lane and 64 per row.
#include "mxfp4_dev.h"
#include "product.h"

namespace mc {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kMaxGroups = 1024;

// One tile of a group: nrows sorted rows from row0, column block nb.
struct Tile {
  int entry, row0, nrows, nb;
};

// Group e's first row and row count (offsets clamped into [0, M], 0 rows if its entry is
// outside the matrices).
__device__ __forceinline__ int group_rows(const ProductArgs& a, int e, int* lo) {
  const int b = min(max(a.offsets[e], 0), a.M), t = min(max(a.offsets[e + 1], 0), a.M);
  const int en = a.entry_of ? a.entry_of[e] : e;
  *lo = b;
  return en >= 0 && en < a.n ? max(t - b, 0) : 0;
}

// Consecutive tiles L on the same XCD: workgroup b runs on XCD b % 8; `total` tiles are dealt
// out in eight runs whose lengths differ by at most one.
__device__ __forceinline__ int xcd_order(int b, int total) {
  const int x = b & 7, q = total >> 3, r = total & 7;
  return x * q + min(x, r) + (b >> 3);
}

// Place of tile p of a group with m row tiles and n_nb column blocks: bands of 8 row tiles,
// column block by column block within a band, so that tiles running at the same time share
// both the weights of a few column blocks and the rows of a few row tiles.
__device__ __forceinline__ void tile_place(int p, int m, int n_nb, int* mt, int* nb) {
  const int band = p / (8 * n_nb), in = p - band * 8 * n_nb;
  const int h = min(8, m - band * 8);              // row tiles of this band
  *nb = in / h;
  *mt = band * 8 + in - *nb * h;
}

// Tile of workgroup `b` (XCD: dealt out by xcd_order): row tiles of BM rows, group by group.
// Every wave runs the search by itself: lane l looks at group 64 c + l, a prefix sum over the
// lanes gives each group's first tile.
template <int BM, bool XCD>
__device__ __forceinline__ bool find_tile(const ProductArgs& a, int b, int n_nb, Tile* t) {
  if (!a.offsets) {
    const int m = (a.M + BM - 1) / BM;
    if (b >= m * n_nb) return false;
    int mt;
    tile_place(XCD ? xcd_order(b, m * n_nb) : b, m, n_nb, &mt, &t->nb);
    t->entry = 0;
    t->row0 = mt * BM;
    t->nrows = min(BM, a.M - t->row0);
    return true;
  }
  const int lane = threadIdx.x & 63;
  int L = b;
  if (XCD) {
    int m = 0;
    for (int e = lane; e < a.E; e += 64) {
      int lo;
      m += (group_rows(a, e, &lo) + BM - 1) / BM;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m += __shfl_xor(m, o, 64);
    const int total = __builtin_amdgcn_readfirstlane(m) * n_nb;
    if (b >= total) return false;
    L = xcd_order(b, total);
  }
  const int j = L / n_nb;
  int before = 0;
  for (int base = 0; base < a.E; base += 64) {
    const int e = base + lane;
    int lo = 0;
    const int rows = e < a.E ? group_rows(a, e, &lo) : 0;
    const int m = (rows + BM - 1) / BM;
    int incl = m;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, 64);
      if (lane >= o) incl += v;
    }
    const uint64_t past = __ballot(before + incl > j);
    if (past) {
      const int src = __ffsll((unsigned long long)past) - 1;
      const int first = before + __builtin_amdgcn_readlane(incl - m, src);
      const int me = __builtin_amdgcn_readlane(m, src), lo_e = __builtin_amdgcn_readlane(lo, src);
      const int rows_e = __builtin_amdgcn_readlane(rows, src);
      int mt;
      tile_place(L - first * n_nb, me, n_nb, &mt, &t->nb);
      t->row0 = lo_e + mt * BM;
      t->nrows = min(BM, rows_e - mt * BM);
      t->entry = a.entry_of ? a.entry_of[base + src] : base + src;
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// Row of x of sorted row i whose route is r; -1 if it is outside x.
__device__ __forceinline__ int x_row(const ProductArgs& a, int i, int r) {
  if (!a.x_perm) return i < a.x_rows ? i : -1;
  const int xr = a.x_div == 1 ? r : r / a.x_div;
  return r >= 0 && xr < a.x_rows ? xr : -1;
}

// Four results v of columns col .. col + 3 of row y_row of y.
__device__ __forceinline__ void store4(const ProductArgs& a, int64_t row, int col, int n_out, const f32x4_t& v) {
  if (a.y_fmt == MC_F32) {
    float* p = reinterpret_cast<float*>(a.y) + row * a.ldy + col;
    if (col + 4 <= n_out && (a.ldy & 3) == 0) {
      *reinterpret_cast<f32x4_t*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < n_out) p[i] = v[i];
    }
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(a.y) + row * a.ldy + col;
    uint16_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = f32_to_bf16_rne(v[i]);
    if (col + 4 <= n_out && (a.ldy & 3) == 0) {
      *reinterpret_cast<uint2*>(p) = make_uint2(o[0] | ((uint32_t)o[1] << 16), o[2] | ((uint32_t)o[3] << 16));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < n_out) p[i] = o[i];
    }
  }
}

// Where sorted row i goes: its row of y (-1: nowhere) and its gate.
struct RowOut {
  int64_t y;
  float gate;
};

__device__ __forceinline__ RowOut row_out(const ProductArgs& a, int i, bool on) {
  const int r = a.perm ? a.perm[i] : i;
  const int yr = a.y_perm ? r : i;
  on = on && r >= 0 && x_row(a, i, r) >= 0 && yr < a.y_rows && (!a.gate || r < a.n_gate);
  return RowOut{on ? yr : -1, a.gate && on ? a.gate[r] : 1.0f};
}

// Two 16-column fragments v (32 neighbouring columns from col0) of one 16-row fragment: v[f][i] is
// column col0 + 16 f + 4 (lane / 16) + i of the lane's row (lane % 16 of the fragment).
__device__ __forceinline__ void store_pair(const ProductArgs& a, const RowOut& o, int col0, int n_out, f32x4_t v0,
                                           f32x4_t v1) {
  const int g = (threadIdx.x & 63) >> 4;
  if (a.gate) {
    v0 *= o.gate;
    v1 *= o.gate;
  }
  if (a.y_fmt == MC_MXFP4) {
    // the block's 8 quarters of four columns meet by lane exchanges over lane bits 4 and 5
    float e[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[i] = v0[i];
      e[4 + i] = v1[i];
      m = max(m, max(abs_bits(v0[i]), abs_bits(v1[i])));
    }
    m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
    const uint32_t X = block_exponent(m);
    const uint32_t c = fp4x8_codes(e, X);
    if (o.y >= 0 && col0 < n_out) {
      uint8_t* p = a.y + o.y * (int64_t)(n_out / 2) + (col0 >> 1) + 2 * g;
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)c;
      *reinterpret_cast<uint16_t*>(p + 8) = (uint16_t)(c >> 16);
      if (g == 0) a.ys[o.y * (int64_t)(n_out / 32) + (col0 >> 5)] = (uint8_t)X;
    }
  } else if (o.y >= 0) {
    const int col = col0 + 4 * g;
    if (col < n_out) store4(a, o.y, col, n_out, v0);
    if (col + 16 < n_out) store4(a, o.y, col + 16, n_out, v1);
  }
}

// One 16-column fragment (bf16 or fp32 y).
__device__ __forceinline__ void store_one(const ProductArgs& a, const RowOut& o, int col0, int n_out, f32x4_t v) {
  const int col = col0 + 4 * ((threadIdx.x & 63) >> 4);
  if (o.y >= 0 && col < n_out) store4(a, o.y, col, n_out, a.gate ? o.gate * v : v);
}

__device__ __forceinline__ f32x4_t swiglu4(const f32x4_t& g, const f32x4_t& u) {
  f32x4_t h;
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = silu(g[i]) * u[i];
  return h;
}

// ---------------------------------------------------------------- operands from memory

__device__ __forceinline__ f32x4_t mfma_bf16(u32x4_t w, u32x4_t x, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w), __builtin_bit_cast(bf16x8_t, x), c, 0,
                                                 0, 0);
}

// Scaled product of two MXFP4 operands: the low byte of sw / sx is the lane's block scale.
__device__ __forceinline__ f32x4_t mfma_fp4(u32x4_t w, uint32_t sw, u32x4_t x, uint32_t sx, f32x4_t c) {
  const i32x8_t a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  const i32x8_t b = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, 0, (int)sw, 0, (int)sx);
}

// ---------------------------------------------------------------- few rows
//
// Tiles of 16 MF rows x 16 NT weight rows (SwiGLU: NT / 2 fragments of gate rows and the matching
// up rows), NT x KW waves: a wave multiplies one 16-row weight fragment over every KW-th
// step of K (64 bytes of each weight row per step), operands straight from memory, and the KW
// partial sums meet in LDS in a fixed order.  With few rows the weights are read once and bound
// the product; what counts is that all of a wave's loads are on their way at once (kFewSteps steps
// per round) and that even a small matrix fills the chip, hence the split of K over waves
// and the narrow tiles.

constexpr int kFewSteps = 4;

template <int XF, int WF, int MF, int NT, int KW>
__global__ void __launch_bounds__(64 * NT * KW)
product_few_kernel(ProductArgs a, int n_nb) {
  __shared__ f32x4_t part[KW][NT][MF][64];
  Tile t;
  if (!find_tile<16 * MF, false>(a, blockIdx.x, n_nb, &t)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const int f = wave % NT, kw = wave / NT;
  const int n_out = a.swiglu ? a.N / 2 : a.N;
  const int c0 = t.nb * (a.swiglu ? 8 * NT : 16 * NT);
  const int64_t K = a.K;
  const int64_t wrow_b = WF == MC_BF16 ? 2 * K : K / 2, xrow_b = XF == MC_BF16 ? 2 * a.ldx : K / 2;
  const int nblk = a.K / 32;
  const int steps = WF == MC_BF16 ? nblk : (nblk + 3) / 4;
  const int wrow = a.swiglu ? min(c0 + (f % (NT / 2)) * 16 + l16, n_out - 1) + (f >= NT / 2 ? n_out : 0)
                            : min(c0 + f * 16 + l16, n_out - 1);
  const uint8_t* wp = a.w + ((int64_t)t.entry * a.N + wrow) * wrow_b;
  const uint8_t* wsp = a.ws + ((int64_t)t.entry * a.N + wrow) * (K / 32);
  const uint8_t* xp[MF];
  const uint8_t* xsp[MF];
#pragma unroll
  for (int m = 0; m < MF; ++m) {
    const int i = t.row0 + min(16 * m + l16, t.nrows - 1);
    const int64_t xr = max(x_row(a, i, a.perm ? a.perm[i] : i), 0);
    xp[m] = a.x + xr * xrow_b;
    xsp[m] = a.xs + xr * (K / 32);
  }

  f32x4_t acc[MF];
#pragma unroll
  for (int m = 0; m < MF; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int s0 = kw; s0 < steps; s0 += KW * kFewSteps) {
    u32x4_t w[kFewSteps];
    uint32_t sw[kFewSteps];
    // steps and blocks past the end re-read the last ones and count as zeros
#pragma unroll
    for (int u = 0; u < kFewSteps; ++u) {
      const int s = min(s0 + u * KW, steps - 1);
      if (WF == MC_BF16) {
        w[u] = *reinterpret_cast<const u32x4_t*>(wp + (int64_t)s * 64 + 16 * g);
      } else {
        const int b = min(4 * s + g, nblk - 1);
        w[u] = *reinterpret_cast<const u32x4_t*>(wp + (int64_t)b * 16);
        sw[u] = wsp[b];
      }
    }
#pragma unroll
    for (int u = 0; u < kFewSteps; ++u) {
      const int s = min(s0 + u * KW, steps - 1);
      const bool in = s0 + u * KW < steps && (WF == MC_BF16 || 4 * s + g < nblk);
      const int b = WF == MC_BF16 ? s : min(4 * s + g, nblk - 1);
      if (!in) w[u] = u32x4_t{0, 0, 0, 0};
      if (WF == MC_BF16) {
#pragma unroll
        for (int m = 0; m < MF; ++m) {
          u32x4_t x = *reinterpret_cast<const u32x4_t*>(xp[m] + (int64_t)b * 64 + 16 * g);
          if (!in) x = u32x4_t{0, 0, 0, 0};       // a zero times an infinity is no zero
          acc[m] = mfma_bf16(w[u], x, acc[m]);
        }
      } else if (XF == MC_MXFP4) {
        if (!in) sw[u] = 127u;
#pragma unroll
        for (int m = 0; m < MF; ++m) {
          const u32x4_t x = *reinterpret_cast<const u32x4_t*>(xp[m] + (int64_t)b * 16);
          const uint32_t sx = in ? xsp[m][b] : 127u;
          acc[m] = mfma_fp4(w[u], sw[u], x, sx, acc[m]);
        }
      } else {
        // the K order of the four products is permuted: lane group g holds block b of its row
        const float s32 = in ? e8m0_or_nan(sw[u]) : 1.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4_t wj = __builtin_bit_cast(u32x4_t, fp4x8_bf16(w[u][j], s32));
#pragma unroll
          for (int m = 0; m < MF; ++m) {
            u32x4_t x = *reinterpret_cast<const u32x4_t*>(xp[m] + (int64_t)b * 64 + 16 * j);
            if (!in) x = u32x4_t{0, 0, 0, 0};
            acc[m] = mfma_bf16(wj, x, acc[m]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MF; ++m) part[kw][f][m][lane] = acc[m];
  __syncthreads();
  // the partial sums of a row fragment: wave m < MF takes row fragment m (and all columns)
  for (int m = wave; m < MF; m += NT * KW) {
    const int r = 16 * m + l16;
    if (16 * m >= t.nrows) break;
    f32x4_t v[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      v[q] = part[0][q][m][lane];
#pragma unroll
      for (int k = 1; k < KW; ++k) v[q] += part[k][q][m][lane];
    }
    const RowOut o = row_out(a, t.row0 + min(r, t.nrows - 1), r < t.nrows);
    if (a.swiglu) {
      if (NT == 4) store_pair(a, o, c0, n_out, swiglu4(v[0], v[2]), swiglu4(v[1], v[3]));
      else store_one(a, o, c0, n_out, swiglu4(v[0], v[1]));
    } else {
#pragma unroll
      for (int q = 0; q < NT; q += 2) store_pair(a, o, c0 + 16 * q, n_out, v[q], v[q + 1]);
    }
  }
}

// ---------------------------------------------------------------- many rows
//
// 256 rows x 256 weight rows (SwiGLU: 128 gate and the matching 128 up rows) per workgroup of 8
// waves, 2 along the rows x 4 along the weight rows: a wave multiplies MF 16-row fragments
// (rows 32 f + 16 wm of the tile, so that a tile of fewer rows runs fewer fragments in every
// wave alike) with 64 weight rows (32 at 32 wn of each half of the weight tile: with SwiGLU
// the gate rows and their up rows).  K moves in stages of 64 bytes per row through a ring of
// four LDS buffers (global_load_lds, no registers): stage s + 3 is requested when stage s
// begins, one barrier per stage.  A row's four 16-byte chunks are stored at chunk
// c ^ (row / 2 % 4), with which the operand reads run at the LDS's full rate (221 of
// 256 B/clk measured, 120 without it).
//
// kBf16: bf16 x bf16, 32 elements per stage.  kFp4: MXFP4 x MXFP4, 128 elements per stage, the
// four scale bytes of each row's stage in a small ring of their own.  kA16W4: bf16 rows in
// stages of 32 elements; the weights' codes and scales come in every four stages (64 bytes per
// row) into a ring of two and become bf16 when a wave reads its fragment.

enum { kBf16 = 0, kA16W4 = 1, kFp4 = 2 };

constexpr int kWideThreads = 512, kWideBM = 256, kWideBN = 256;
constexpr int kRing = 4;
constexpr int kTileBytes = 256 * 64;              // one operand's tile of a stage

template <int VM>
__device__ __forceinline__ void wait_stage() {
  // at most VM loads outstanding, every LDS access done, then the workgroup's barrier
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((VM & 15) | (7 << 4) | ((VM >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

typedef __attribute__((address_space(3))) void* lds_ptr;

// 16 (4) bytes per lane from src into LDS at dst + 16 (4) lane, dst the same for the wave.  Written
// as an instruction with no register result: the compiler's builtin makes every later LDS read
// wait for all such loads, those for other ring buffers among them.  The reader's wait is
// wait_stage's; the compiler's own waits for other loads count these as unknown older or newer
// ones, which can only make them longer.
__device__ __forceinline__ void load_lds16(const uint8_t* src, void* dst) {
  const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_ptr)dst);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(src) : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(const uint8_t* src, void* dst) {
  const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_ptr)dst);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(at), "v"(src) : "memory", "m0");
}

// Four scale bytes of blocks b .. b + 3 of a row of n blocks, at any alignment (blocks past the
// last count as 2^0).
__device__ __forceinline__ uint32_t load_scales(const uint8_t* row, int b, int n) {
  uint32_t v = 0x7F7F7F7Fu;
  if (b + 4 <= n) {
    __builtin_memcpy(&v, row + b, 4);
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (b + i < n) v = (v & ~(0xFFu << (8 * i))) | ((uint32_t)row[b + i] << (8 * i));
  }
  return v;
}

struct WideLds {
  uint8_t x[kRing][kTileBytes];
  uint8_t w[kRing][kTileBytes];
  uint32_t s[kRing][512];                         // scales: weight rows, then rows (MXFP4)
};
struct WideLdsBf16 {
  uint8_t x[kRing][kTileBytes];
  uint8_t w[kRing][kTileBytes];
};
struct WideLdsA16 {
  uint8_t x[kRing][kTileBytes];
  uint8_t w[2][kTileBytes];
  uint32_t s[2][256];
};
template <int MODE> struct WideLdsOf { typedef WideLds type; };
template <> struct WideLdsOf<kBf16> { typedef WideLdsBf16 type; };
template <> struct WideLdsOf<kA16W4> { typedef WideLdsA16 type; };

// SDMA: the scales of a row start at a multiple of four bytes and K is a multiple of 128, so they
// go straight into LDS like the operands; otherwise they pass through a register, whose wait
// also drains the loads on their way.
template <int MODE, bool SDMA, int MF>
__device__ __forceinline__ void wide_tile(const ProductArgs& a, const Tile& t, typename WideLdsOf<MODE>::type& lds) {
  constexpr int XQ = MF > 4 ? 2 : 1;              // x loads per thread and stage: 128 rows each
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, l16 = lane & 15;
  const int wm = wave & 1, wn = wave >> 1;
  const int n_out = a.swiglu ? a.N / 2 : a.N;
  const int c0 = t.nb * (a.swiglu ? kWideBN / 2 : kWideBN);
  const int64_t K = a.K;
  const int64_t wrow_b = MODE == kBf16 ? 2 * K : K / 2, xrow_b = MODE == kFp4 ? K / 2 : 2 * a.ldx;
  const int xb = MODE == kFp4 ? a.K / 2 : 2 * a.K, wb = MODE == kBf16 ? 2 * a.K : a.K / 2;   // bytes of a row in use
  const int stages = (xb + 63) / 64;

  // this thread's 16 bytes of a stage: rows tid / 4 and 128 + tid / 4, logical chunk ch
  const int ch = (tid & 3) ^ ((tid >> 3) & 3);
  const uint8_t *wp[2], *xp[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int row = a.swiglu ? min(c0 + (tid >> 2), n_out - 1) + q * n_out : min(c0 + q * 128 + (tid >> 2), n_out - 1);
    wp[q] = a.w + ((int64_t)t.entry * a.N + row) * wrow_b + ch * 16;
    const int i = t.row0 + min(q * 128 + (tid >> 2), t.nrows - 1);
    xp[q] = a.x + (int64_t)max(x_row(a, i, a.perm ? a.perm[i] : i), 0) * xrow_b + ch * 16;
  }
  const uint8_t* sp = nullptr;                    // scales of weight row tid, and of row tid - 256
  if (MODE != kBf16) {
    if (tid < 256) {
      const int r = tid & 127, q = tid >> 7;
      const int row = a.swiglu ? min(c0 + r, n_out - 1) + q * n_out : min(c0 + tid, n_out - 1);
      sp = a.ws + ((int64_t)t.entry * a.N + row) * (K / 32);
    } else if (MODE == kFp4) {
      const int i = t.row0 + min(tid - 256, t.nrows - 1);
      sp = a.xs + (int64_t)max(x_row(a, i, a.perm ? a.perm[i] : i), 0) * (K / 32);
    }
  }
  const int nblk = a.K / 32;
  uint32_t sc = 0;
  // 64 bytes of every weight row and the scales of their blocks: stage s (kA16W4: four stages)
  auto request_w = [&](int s) {
    const int b = MODE == kA16W4 ? s & 1 : s & (kRing - 1);
    // a chunk past the row's end (only in the last stage) re-reads the row's first bytes
    const int64_t off = s * 64 + ch * 16 < wb ? (int64_t)s * 64 : -(int64_t)(ch * 16);
    if constexpr (MODE != kBf16) {
      if (MODE == kFp4 || wave < 4) {
        if (SDMA) load_lds4(sp + s * 4, &lds.s[b][wave * 64]);
        else sc = load_scales(sp, s * 4, nblk);
      }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) load_lds16(wp[q] + off, &lds.w[b][q * 8192 + wave * 1024]);
  };
  auto request_x = [&](int s) {
    const int b = s & (kRing - 1);
    const int64_t off = s * 64 + ch * 16 < xb ? (int64_t)s * 64 : -(int64_t)(ch * 16);
#pragma unroll
    for (int q = 0; q < XQ; ++q) load_lds16(xp[q] + off, &lds.x[b][q * 8192 + wave * 1024]);
  };
  auto put_scales = [&](int s) {
    if constexpr (MODE != kBf16 && !SDMA) {
      if (MODE == kFp4 || wave < 4) lds.s[MODE == kA16W4 ? s & 1 : s & (kRing - 1)][tid] = sc;
    }
  };

  f32x4_t acc[4][MF];
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int m = 0; m < MF; ++m) acc[f][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const int swz = (l16 >> 1) & 3;
  const int frag = l16 * 64 + ((g ^ swz) << 4);
  const int xfrag = wm * 16 * 64 + frag;
  auto compute = [&](int s) {
    const int b = s & (kRing - 1);
    u32x4_t w[4];
    uint32_t sw[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int row = (f >> 1) * 128 + (f & 1) * 16 + wn * 32;
      if constexpr (MODE == kA16W4) {
        // element 8 g of block s of the row: a dword of its 16-byte chunk
        const int c = (s >> 2) & 1, j = s & 3;
        const uint32_t code =
            *reinterpret_cast<const uint32_t*>(&lds.w[c][(row + l16) * 64 + ((j ^ swz) << 4) + g * 4]);
        const uint32_t X = reinterpret_cast<const uint8_t*>(lds.s[c])[(row + l16) * 4 + j];
        w[f] = __builtin_bit_cast(u32x4_t, fp4x8_bf16(code, e8m0_or_nan(X)));
      } else {
        w[f] = *reinterpret_cast<const u32x4_t*>(&lds.w[b][row * 64 + frag]);
        if constexpr (MODE == kFp4) sw[f] = lds.s[b][row + l16] >> (8 * g);
      }
    }
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      const u32x4_t x = *reinterpret_cast<const u32x4_t*>(&lds.x[b][xfrag + m * 32 * 64]);
      if constexpr (MODE == kFp4) {
        const uint32_t sx = lds.s[b][256 + m * 32 + wm * 16 + l16] >> (8 * g);
#pragma unroll
        for (int f = 0; f < 4; ++f) acc[f][m] = mfma_fp4(w[f], sw[f], x, sx, acc[f][m]);
      } else {
#pragma unroll
        for (int f = 0; f < 4; ++f) acc[f][m] = mfma_bf16(w[f], x, acc[f][m]);
      }
    }
  };

  if (MODE == kA16W4) {
    request_w(0);
    put_scales(0);
  }
  for (int s = 0; s < kRing - 1 && s < stages; ++s) {
    if (MODE != kA16W4) {
      request_w(s);
      put_scales(s);
    }
    request_x(s);
  }
  int s = 0;
  for (; s + kRing - 1 < stages; ++s) {
    // stage s is in; s + 1 and s + 2 (and with s % 4 = 1, 2 the weights of the next four stages,
    // requested with or after stage s + 1) may be on their way
    if (MODE != kA16W4) wait_stage<2 * (2 + XQ + (MODE == kFp4 && SDMA))>();
    else if (((s - 1) & 3) < 2) wait_stage<2 * XQ + 2>();
    else wait_stage<2 * XQ>();
    if (MODE != kA16W4) request_w(s + kRing - 1);
    else if ((s & 3) == 0 && (s + 4) < stages) request_w((s >> 2) + 1);
    request_x(s + kRing - 1);
    compute(s);
    if (MODE != kA16W4) put_scales(s + kRing - 1);
    else if ((s & 3) == 0 && (s + 4) < stages) put_scales((s >> 2) + 1);
  }
  for (; s < stages; ++s) {
    if (MODE == kFp4 && !SDMA && s + 1 == stages && (xb & 63)) {
      // the last stage's chunks past the row's end count as zeros: of one operand, since every
      // e2m1 code is finite
      __builtin_amdgcn_s_waitcnt(0 | (7 << 4) | (15 << 8));
      asm volatile("" ::: "memory");
      if (s * 64 + ch * 16 >= wb) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
          *reinterpret_cast<u32x4_t*>(&lds.w[s & (kRing - 1)][q * 8192 + tid * 16]) = u32x4_t{0, 0, 0, 0};
      }
    }
    wait_stage<0>();
    compute(s);
  }

  RowOut o[MF];
#pragma unroll
  for (int m = 0; m < MF; ++m) {
    const int r = m * 32 + wm * 16 + l16;
    o[m] = row_out(a, t.row0 + min(r, t.nrows - 1), r < t.nrows);
  }
#pragma unroll
  for (int m = 0; m < MF; ++m) {
    if (a.swiglu) {
      store_pair(a, o[m], c0 + wn * 32, n_out, swiglu4(acc[0][m], acc[2][m]), swiglu4(acc[1][m], acc[3][m]));
    } else {
      store_pair(a, o[m], c0 + wn * 32, n_out, acc[0][m], acc[1][m]);
      store_pair(a, o[m], c0 + 128 + wn * 32, n_out, acc[2][m], acc[3][m]);
    }
  }
}

template <int MODE, bool SDMA>
__global__ void __launch_bounds__(kWideThreads, 2)
product_wide_kernel(ProductArgs a, int n_nb) {
  __shared__ __attribute__((aligned(16))) typename WideLdsOf<MODE>::type lds;
  Tile t;
  if (!find_tile<kWideBM, true>(a, blockIdx.x, n_nb, &t)) return;
  // 32-row steps of the tile, the same for the whole workgroup
  const int steps = (t.nrows + 31) >> 5;
  if constexpr (SDMA) {
    switch (steps) {
      case 1: wide_tile<MODE, SDMA, 1>(a, t, lds); break;
      case 2: wide_tile<MODE, SDMA, 2>(a, t, lds); break;
      case 3: wide_tile<MODE, SDMA, 3>(a, t, lds); break;
      case 4: wide_tile<MODE, SDMA, 4>(a, t, lds); break;
      case 5: wide_tile<MODE, SDMA, 5>(a, t, lds); break;
      case 6: wide_tile<MODE, SDMA, 6>(a, t, lds); break;
      case 7: wide_tile<MODE, SDMA, 7>(a, t, lds); break;
      default: wide_tile<MODE, SDMA, 8>(a, t, lds); break;
    }
  } else {
    if (steps <= 2) wide_tile<MODE, SDMA, 2>(a, t, lds);
    else if (steps <= 4) wide_tile<MODE, SDMA, 4>(a, t, lds);
    else wide_tile<MODE, SDMA, 8>(a, t, lds);
  }
}

// ---------------------------------------------------------------- launch

int check_product(const char* fn, const ProductArgs& a) {
  MC_REQUIRE((a.x_fmt == MC_BF16 && (a.w_fmt == MC_BF16 || a.w_fmt == MC_MXFP4)) ||
                 (a.x_fmt == MC_MXFP4 && a.w_fmt == MC_MXFP4),
             "%s: no product of x format %d with w format %d", fn, a.x_fmt, a.w_fmt);
  MC_REQUIRE(a.y_fmt == MC_BF16 || a.y_fmt == MC_F32 || a.y_fmt == MC_MXFP4, "%s: unknown y format %d", fn, a.y_fmt);
  MC_REQUIRE(a.M >= 0 && a.N >= 0 && a.K >= 32 && a.K % 32 == 0, "%s: M=%d N=%d K=%d (K must be a positive multiple of 32)",
             fn, a.M, a.N, a.K);
  MC_REQUIRE(a.E >= 1 && a.E <= kMaxGroups, "%s: E=%d must be in [1, %d]", fn, a.E, kMaxGroups);
  MC_REQUIRE(a.swiglu == 0 || a.swiglu == 1, "%s: swiglu=%d", fn, a.swiglu);
  MC_REQUIRE(!a.swiglu || a.N % 2 == 0, "%s: N=%d must be even with swiglu", fn, a.N);
  const int n_out = a.swiglu ? a.N / 2 : a.N;
  MC_REQUIRE(a.y_fmt != MC_MXFP4 || n_out % 32 == 0, "%s: MXFP4 rows of %d columns (must be a multiple of 32)", fn, n_out);
  MC_REQUIRE(!a.gate || a.n_gate >= 0, "%s: n_gate=%d", fn, a.n_gate);
  MC_REQUIRE(a.x_div >= 1 && a.x_rows >= 0 && a.y_rows >= 0 && a.n >= 0, "%s: x_div=%d x_rows=%d y_rows=%d n=%lld", fn,
             a.x_div, a.x_rows, a.y_rows, (long long)a.n);
  MC_REQUIRE((a.x_perm == 0 || a.x_perm == 1) && (a.y_perm == 0 || a.y_perm == 1), "%s: x_perm=%d y_perm=%d", fn, a.x_perm,
             a.y_perm);
  MC_REQUIRE(a.perm || a.M == 0 || (!a.x_perm && !a.y_perm), "%s: x_perm and y_perm need perm", fn);
  if (a.x_fmt == MC_BF16)
    MC_REQUIRE(a.ldx >= a.K && a.ldx % 8 == 0, "%s: ldx=%lld must be at least K=%d and a multiple of 8", fn,
               (long long)a.ldx, a.K);
  if (a.y_fmt != MC_MXFP4) MC_REQUIRE(a.ldy >= n_out, "%s: ldy=%lld < %d columns", fn, (long long)a.ldy, n_out);
  const int64_t most = (int64_t)1 << 31;
  MC_REQUIRE(a.ldx < most && a.ldy < most && a.n < most, "%s: ldx=%lld ldy=%lld n=%lld too large", fn, (long long)a.ldx,
             (long long)a.ldy, (long long)a.n);
  if (a.M == 0 || a.N == 0) return MC_OK;
  MC_REQUIRE(a.x && a.w && a.y, "%s: NULL pointer", fn);
  MC_REQUIRE(a.x_fmt != MC_MXFP4 || a.xs, "%s: MXFP4 x needs scales", fn);
  MC_REQUIRE(a.w_fmt != MC_MXFP4 || a.ws, "%s: MXFP4 w needs scales", fn);
  MC_REQUIRE(a.y_fmt != MC_MXFP4 || a.ys, "%s: MXFP4 y needs scales", fn);
  MC_REQUIRE(((uintptr_t)a.x | (uintptr_t)a.w | (uintptr_t)a.y) % 16 == 0, "%s: x, w and y must be 16-byte aligned", fn);
  MC_REQUIRE(((uintptr_t)a.offsets | (uintptr_t)a.perm | (uintptr_t)a.entry_of | (uintptr_t)a.gate) % 4 == 0,
             "%s: index and gate arrays must be 4-byte aligned", fn);
  return MC_OK;
}

// Row tiles of all groups together, at most: sum over groups of ceil(rows / bm).
static int64_t most_row_tiles(const ProductArgs& a, int64_t bm) {
  return a.offsets ? a.M / bm + (a.E < a.M ? a.E : a.M) : (a.M + bm - 1) / bm;
}

template <int XF, int WF, int MF, int NT>
static void launch_few_k(const ProductArgs& a, unsigned grid, int n_nb, int steps, hipStream_t s) {
  // enough waves along K that a wave has at most 4 steps, up to 16 waves per workgroup
  if (steps <= 16 || NT == 4)
    hipLaunchKernelGGL((product_few_kernel<XF, WF, MF, NT, 4>), dim3(grid), dim3(64 * NT * 4), 0, s, a, n_nb);
  else if constexpr (NT == 2)
    hipLaunchKernelGGL((product_few_kernel<XF, WF, MF, NT, 8>), dim3(grid), dim3(64 * NT * 8), 0, s, a, n_nb);
}

template <int XF, int WF>
static int launch_few(const ProductArgs& a, hipStream_t s) {
  const int nt = a.swiglu && a.y_fmt == MC_MXFP4 ? 4 : 2;
  const int64_t n_out = a.swiglu ? a.N / 2 : a.N, cols = a.swiglu ? 8 * nt : 16 * nt;
  const int64_t n_nb = (n_out + cols - 1) / cols;
  const int mf = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
  const int64_t tiles = most_row_tiles(a, 16 * mf) * n_nb;
  MC_REQUIRE(tiles <= 0x7FFFFFFF, "product of %d rows with %d columns is too large", a.M, a.N);
  const int steps = WF == MC_BF16 ? a.K / 32 : (a.K + 127) / 128;
  const unsigned grid = (unsigned)tiles;
  if (nt == 4) {
    if (mf == 1) launch_few_k<XF, WF, 1, 4>(a, grid, (int)n_nb, steps, s);
    else if (mf == 2) launch_few_k<XF, WF, 2, 4>(a, grid, (int)n_nb, steps, s);
    else launch_few_k<XF, WF, 4, 4>(a, grid, (int)n_nb, steps, s);
  } else {
    if (mf == 1) launch_few_k<XF, WF, 1, 2>(a, grid, (int)n_nb, steps, s);
    else if (mf == 2) launch_few_k<XF, WF, 2, 2>(a, grid, (int)n_nb, steps, s);
    else launch_few_k<XF, WF, 4, 2>(a, grid, (int)n_nb, steps, s);
  }
  MC_LAUNCH_CHECK();
  return MC_OK;
}

static int launch_wide(const ProductArgs& a, hipStream_t s) {
  const int64_t n_out = a.swiglu ? a.N / 2 : a.N, cols = a.swiglu ? kWideBN / 2 : kWideBN;
  const int64_t n_nb = (n_out + cols - 1) / cols, tiles = most_row_tiles(a, kWideBM) * n_nb;
  MC_REQUIRE(tiles <= 0x7FFFFFFF, "product of %d rows with %d columns is too large", a.M, a.N);
  const bool sdma = a.K % 128 == 0 && ((uintptr_t)a.xs | (uintptr_t)a.ws) % 4 == 0;
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)tiles), dim3(kWideThreads), 0, s, a, (int)n_nb);
  };
  if (a.w_fmt == MC_BF16) run(product_wide_kernel<kBf16, true>);
  else if (a.x_fmt == MC_BF16 && sdma) run(product_wide_kernel<kA16W4, true>);
  else if (a.x_fmt == MC_BF16) run(product_wide_kernel<kA16W4, false>);
  else if (sdma) run(product_wide_kernel<kFp4, true>);
  else run(product_wide_kernel<kFp4, false>);
  MC_LAUNCH_CHECK();
  return MC_OK;
}

int launch_product(const ProductArgs& a, hipStream_t s) {
  if (a.M == 0 || a.N == 0 || a.x_rows == 0 || a.y_rows == 0 || a.n == 0) return MC_OK;
  if (a.M > 64) return launch_wide(a, s);
  if (a.x_fmt == MC_MXFP4) return launch_few<MC_MXFP4, MC_MXFP4>(a, s);
  if (a.w_fmt == MC_MXFP4) return launch_few<MC_BF16, MC_MXFP4>(a, s);
  return launch_few<MC_BF16, MC_BF16>(a, s);
}

}  // namespace mc

using namespace mc;

extern "C" int mc_mxfp4_matmul(const void* x, const void* x_scale, int32_t x_fmt, int64_t ldx, const void* w,
                               const void* w_scale, int32_t M, int32_t N, int32_t K, void* y, int32_t y_fmt,
                               int64_t ldy, hipStream_t s) {
  clear_error();
  ProductArgs a{};
  a.x = static_cast<const uint8_t*>(x);
  a.xs = static_cast<const uint8_t*>(x_scale);
  a.w = static_cast<const uint8_t*>(w);
  a.ws = static_cast<const uint8_t*>(w_scale);
  a.y = static_cast<uint8_t*>(y);
  a.x_fmt = x_fmt;
  a.w_fmt = MC_MXFP4;
  a.y_fmt = y_fmt;
  a.ldx = x_fmt == MC_BF16 ? ldx : K;
  a.ldy = ldy;
  a.E = 1;
  a.n = 1;
  a.M = a.x_rows = a.y_rows = M;
  a.N = N;
  a.K = K;
  a.x_div = 1;
  MC_REQUIRE(y_fmt != MC_MXFP4, "mc_mxfp4_matmul: y is bf16 or fp32");
  int rc;
  if ((rc = check_product("mc_mxfp4_matmul", a)) != MC_OK) return rc;
  return launch_product(a, s);
}

extern "C" int mc_grouped_matmul(const mc_grouped* g, hipStream_t s) {
  clear_error();
  MC_REQUIRE(g != nullptr, "mc_grouped_matmul: descriptor is NULL");
  ProductArgs a{};
  a.x = static_cast<const uint8_t*>(g->x);
  a.xs = static_cast<const uint8_t*>(g->x_scale);
  a.w = static_cast<const uint8_t*>(g->w);
  a.ws = static_cast<const uint8_t*>(g->w_scale);
  a.y = static_cast<uint8_t*>(g->y);
  a.ys = static_cast<uint8_t*>(g->y_scale);
  a.offsets = g->offsets;
  a.perm = g->perm;
  a.entry_of = g->entry_of;
  a.gate = g->gate;
  a.n_gate = g->n_gate;
  a.ldx = g->x_fmt == MC_MXFP4 ? g->K : g->ldx;
  a.ldy = g->y_fmt == MC_MXFP4 ? 0 : g->ldy;
  a.n = g->n;
  a.x_fmt = g->x_fmt;
  a.w_fmt = g->w_fmt;
  a.y_fmt = g->y_fmt;
  a.swiglu = g->swiglu;
  a.E = g->E;
  a.M = g->M;
  a.N = g->N;
  a.K = g->K;
  a.x_rows = g->x_rows;
  a.x_div = g->x_div;
  a.x_perm = g->x_perm;
  a.y_rows = g->y_rows;
  a.y_perm = g->y_perm;
  int rc;
  if ((rc = check_product("mc_grouped_matmul", a)) != MC_OK) return rc;
  MC_REQUIRE(a.offsets || a.M == 0, "mc_grouped_matmul: offsets is NULL");
  return launch_product(a, s);
}
