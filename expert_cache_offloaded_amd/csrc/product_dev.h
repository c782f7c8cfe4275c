// Kernels of mc_mxfp4_matmul and mc_grouped_matmul: products of rows (bf16 or MXFP4) with expert matrices
// (bf16 or MXFP4), grouped by expert.
//
// The weights are the MFMA's A operand and the rows its B operand, so a lane's four results
// of one instruction are four consecutive output columns of one row.  bf16 operands: MFMA
// 16x16x32, lane l holds 8 elements of row l % 16 from k = 8 (l / 16).  MXFP4 operands: the
// scaled MFMA 16x16x128, lane l holds the whole 32-element block l / 16 of row l % 16 and its
// scale byte, so both formats read 16 bytes per lane and 64 per row.
#pragma once

#include <type_traits>

#include "mxfp4_dev.h"
#include "product.h"

namespace mc {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// One tile of a group: nrows sorted rows from row0, column block nb.
struct Tile {
  int entry, row0, nrows, nb;
};

// Group e's first row and row count (offsets clamped into [0, M], 0 rows if its entry is
// outside the matrices).
template <class P>
__device__ __forceinline__ int group_rows(const ProductArgs& a, P offsets, P entry_of, int e, int* lo) {
  const int b = min(max(offsets[e], 0), a.M), t = min(max(offsets[e + 1], 0), a.M);
  const int en = entry_of ? entry_of[e] : e;
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

__device__ __forceinline__ constexpr int div_up(int a, int b) { return (a + b - 1) / b; }

// Sum over the lanes up to and including this one.
__device__ __forceinline__ int lane_prefix(int v) {
  // row_shr 1, 2, 4, 8, then the rows' totals to the rows behind them
#define MC_STEP(CTRL, ROWS) v += __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false)
  MC_STEP(0x111, 0xF);
  MC_STEP(0x112, 0xF);
  MC_STEP(0x114, 0xF);
  MC_STEP(0x118, 0xF);
  MC_STEP(0x142, 0xA);
  MC_STEP(0x143, 0xC);
#undef MC_STEP
  return v;
}

// The row tile j (BM rows) of all groups: its group's tiles begin at `first`.
__device__ __forceinline__ void place_in_group(const ProductArgs& a, int e, int p, int bm, int n_nb, Tile* t) {
  // e is the same for the wave: scalar loads, which no vector load's wait holds up (the tables are
  // not written while the kernel runs)
  typedef const __attribute__((address_space(4))) int32_t* scalar_ptr;
  const scalar_ptr offsets = (scalar_ptr)a.offsets, entry_of = (scalar_ptr)a.entry_of;
  int lo;
  const int rows = group_rows(a, offsets, entry_of, e, &lo);
  int mt;
  tile_place(p, div_up(rows, bm), n_nb, &mt, &t->nb);
  t->row0 = lo + mt * bm;
  t->nrows = min(bm, rows - mt * bm);
  t->entry = a.entry_of ? entry_of[e] : e;
}

__device__ __forceinline__ void place_ungrouped(const ProductArgs& a, int p, int bm, int n_nb, Tile* t) {
  int mt;
  tile_place(p, div_up(a.M, bm), n_nb, &mt, &t->nb);
  t->entry = 0;
  t->row0 = mt * bm;
  t->nrows = min(bm, a.M - t->row0);
}

// Row tiles of groups base + 64 c + lane, c < 4: all tables are read before the first is used.
template <int BM>
__device__ __forceinline__ void group_tiles(const ProductArgs& a, int base, int* m) {
  const int lane = threadIdx.x & 63;
  int rows[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int e = base + 64 * c + lane;
    int lo;
    rows[c] = group_rows(a, a.offsets, a.entry_of, min(e, a.E - 1), &lo);
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) m[c] = base + 64 * c + lane < a.E ? div_up(rows[c], BM) : 0;
}

// Tile b of the call, group by group.  Every wave runs the search by itself: lane l looks at group
// 64 c + l, a prefix sum over the lanes gives each group's first tile.
template <int BM>
__device__ __forceinline__ bool find_tile(const ProductArgs& a, int b, int n_nb, Tile* t) {
  if (!a.offsets) {
    if (b >= div_up(a.M, BM) * n_nb) return false;
    place_ungrouped(a, b, BM, n_nb, t);
    return true;
  }
  const int j = b / n_nb;
  int before = 0;
  for (int base = 0; base < a.E; base += 256) {
    int m[4];
    group_tiles<BM>(a, base, m);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int incl = lane_prefix(m[c]);
      const uint64_t past = __ballot(before + incl > j);
      if (past) {
        const int src = __ffsll((unsigned long long)past) - 1;
        const int first = before + __builtin_amdgcn_readlane(incl - m[c], src);
        place_in_group(a, base + 64 * c + src, b - first * n_nb, BM, n_nb, t);
        return true;
      }
      before += __builtin_amdgcn_readlane(incl, 63);
    }
  }
  return false;
}

// The same with the groups' first tiles in LDS, for workgroups that take several tiles: after
// first_tiles (one wave) and a barrier, first[e] is group e's first row tile, first[E] their number.
template <int BM>
__device__ __forceinline__ void first_tiles(const ProductArgs& a, int* first) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int base = 0; base < a.E; base += 256) {
    int m[4];
    group_tiles<BM>(a, base, m);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int e = base + 64 * c + lane, incl = lane_prefix(m[c]);
      if (e < a.E) first[e] = before + incl - m[c];
      before += __builtin_amdgcn_readlane(incl, 63);
    }
  }
  if (lane == 0) first[a.E] = before;
}

// Tile b in the order of the XCDs (total: tiles of the call).
template <int BM>
__device__ __forceinline__ void next_tile(const ProductArgs& a, int b, int total, int n_nb, const int* first, Tile* t) {
  const int L = xcd_order(b, total);
  if (!a.offsets) return place_ungrouped(a, L, BM, n_nb, t);
  const int lane = threadIdx.x & 63;
  const int j = L / n_nb;
  for (int base = 0;; base += 64) {                // first[E] > j, so a group is found
    const uint64_t past = __ballot(first[min(base + lane, a.E - 1) + 1] > j);
    if (past) {
      const int e = base + __ffsll((unsigned long long)past) - 1;
      place_in_group(a, e, L - __builtin_amdgcn_readfirstlane(first[e]) * n_nb, BM, n_nb, t);
      return;
    }
  }
}

// Row of x of sorted row i whose route is r; -1 if it is outside x.
__device__ __forceinline__ int x_row(const ProductArgs& a, int i, int r) {
  if (!a.x_perm) return i < a.x_rows ? i : -1;
  const int xr = a.x_div == 1 ? r : r / a.x_div;
  return r >= 0 && xr < a.x_rows ? xr : -1;
}

// fp32 -> bf16 pairs, round to nearest even (one instruction per pair).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const bf16x2_t r = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, r);
}

// N (4 or 8) results of columns col .. col + N - 1 of a row of y that starts at p.  YF: y's type; VEC:
// rows and columns allow vector stores.  Those of fp32 pass the caches by, the operands' (6144 routes x 4096
// 267 -> 264 us, a layer of bf16 experts 341 -> 335; bf16 ones did not gain: 8192 x 4096 82 -> 90 us).
template <int YF, bool VEC, int N>
__device__ __forceinline__ void store_cols(uint8_t* p, int col, int n_out, const float* v) {
  if (YF == MC_F32) {
    float* q = reinterpret_cast<float*>(p) + col;
    if (VEC && col + N <= n_out) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        __builtin_nontemporal_store(f32x4_t{v[i], v[i + 1], v[i + 2], v[i + 3]}, reinterpret_cast<f32x4_t*>(q + i));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (col + i < n_out) q[i] = v[i];
    }
  } else {
    uint16_t* q = reinterpret_cast<uint16_t*>(p) + col;
    uint32_t c[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) c[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    if (VEC && col + N <= n_out) {
      __builtin_memcpy(__builtin_assume_aligned(q, 2 * N), c, 2 * N);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (col + i < n_out) q[i] = (uint16_t)(c[i / 2] >> (16 * (i & 1)));
    }
  }
}

// Where a sorted row goes: its row of y (-1: nowhere) and its gate.
struct RowOut {
  int64_t y;
  float gate;
};

// The rows i[m] (those with !on[m] go nowhere).  Every route is read before the first gate, and every
// gate before the first result is stored: no chain of round trips row by row.
template <int N>
__device__ __forceinline__ void rows_out(const ProductArgs& a, const int* i, const bool* on, RowOut* o) {
  int r[N];
  if (a.perm) {
#pragma unroll
    for (int m = 0; m < N; ++m) r[m] = a.perm[i[m]];
  } else {
#pragma unroll
    for (int m = 0; m < N; ++m) r[m] = i[m];
  }
  // r / x_div < x_rows without the division
  const int64_t most = a.x_perm ? (int64_t)a.x_rows * a.x_div : INT64_MAX;
#pragma unroll
  for (int m = 0; m < N; ++m) {
    const int yr = a.y_perm ? r[m] : i[m];
    const bool to = on[m] && r[m] >= 0 && r[m] < most && (a.x_perm || i[m] < a.x_rows) && yr < a.y_rows &&
                    (!a.gate || r[m] < a.n_gate);
    o[m] = RowOut{to ? yr : -1, 1.0f};
    if (!to) r[m] = 0;
  }
  if (a.gate && a.n_gate > 0) {
#pragma unroll
    for (int m = 0; m < N; ++m) o[m].gate = a.gate[r[m]];
  }
}

// Two 16-column fragments (32 neighbouring columns from col0) of one 16-row fragment: vf[i] is column
// col0 + 16 f + 4 (lane / 16) + i of the lane's row (lane % 16 of the fragment).
template <int YF, bool VEC>
__device__ __forceinline__ void store_pair(const ProductArgs& a, const RowOut& o, int col0, int n_out,
                                           const f32x4_t& v0, const f32x4_t& v1) {
  const int g = (threadIdx.x & 63) >> 4;
  // lane quarters 1 and 3 of the first fragment change places with 0 and 2 of the second: a lane
  // then holds eight neighbouring columns, 8 (g / 2) of fragment g % 2
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v0[i]), __float_as_uint(v1[i]), false, false);
    v[i] = __uint_as_float(s[0]);
    v[4 + i] = __uint_as_float(s[1]);
  }
  if (a.gate) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= o.gate;
  }
  const int col = col0 + 16 * (g & 1) + 8 * (g >> 1);
  if (YF == MC_MXFP4) {
    // the block's four lanes meet by lane exchanges over lane bits 4 and 5
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    const auto m16 = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = max(m16[0], m16[1]);
    const auto m32 = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    const uint32_t X = block_exponent(max(m32[0], m32[1]));
    const uint32_t c = fp4x8_codes(v, X);
    if (o.y >= 0 && col0 < n_out) {
      *reinterpret_cast<uint32_t*>(a.y + o.y * (int64_t)(n_out / 2) + (col >> 1)) = c;
      if (g == 0) a.ys[o.y * (int64_t)(n_out / 32) + (col0 >> 5)] = (uint8_t)X;
    }
  } else if (o.y >= 0 && col < n_out) {
    store_cols<YF, VEC, 8>(a.y + o.y * a.ldy * (YF == MC_F32 ? 4 : 2), col, n_out, v);
  }
}

// One 16-column fragment (bf16 or fp32 y).
template <int YF, bool VEC>
__device__ __forceinline__ void store_one(const ProductArgs& a, const RowOut& o, int col0, int n_out,
                                          const f32x4_t& f) {
  const int col = col0 + 4 * ((threadIdx.x & 63) >> 4);
  const float v[4] = {o.gate * f[0], o.gate * f[1], o.gate * f[2], o.gate * f[3]};
  if (YF != MC_MXFP4 && o.y >= 0 && col < n_out)
    store_cols<YF, VEC, 4>(a.y + o.y * a.ldy * (YF == MC_F32 ? 4 : 2), col, n_out, v);
}

// f(type of y, rows aligned for vector stores) with both as constants: the branches are taken once.
template <int V>
struct Const {
  static constexpr int value = V;
};
template <class F>
__device__ __forceinline__ void with_format(const ProductArgs& a, F f) {
  // 16-byte stores, from a column divisible by 8
  const bool vec = (a.ldy & (a.y_fmt == MC_F32 ? 3 : 7)) == 0;
  if (a.y_fmt == MC_MXFP4) f(Const<MC_MXFP4>(), Const<1>());
  else if (a.y_fmt == MC_F32 && vec) f(Const<MC_F32>(), Const<1>());
  else if (a.y_fmt == MC_F32) f(Const<MC_F32>(), Const<0>());
  else if (vec) f(Const<MC_BF16>(), Const<1>());
  else f(Const<MC_BF16>(), Const<0>());
}

__device__ __forceinline__ f32x4_t swiglu4(const f32x4_t& g, const f32x4_t& u) {
  // The division is exact: the reciprocal instruction flushes results below 2^-126 to zero, and with
  // them silu(g) of g under -87.3, about -1e-36 and a normal number (layer of 8192 tokens 1.39 ms with
  // the reciprocal, 1.41 so).
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
// Tiles of 16 rows x 16 NT weight rows (SwiGLU: NT / 2 fragments of gate rows and the matching up
// rows), NT x KW waves: a wave multiplies one 16-row weight fragment over every KW-th
// step of K (64 bytes of each weight row per step), operands straight from memory, and the KW
// partial sums meet in LDS in a fixed order.  With few rows the weights are read once and bound
// the product; what counts is that all of a wave's loads are on their way at once (STEPS steps per
// round) and that even a small matrix fills the chip, hence the split of K over waves
// and the narrow tiles.  A launch holds less than 2^32 threads; beyond, workgroups take several tiles.

template <int XF, int WF, int NT, int KW, int STEPS>
__device__ __forceinline__ void few_tile(const ProductArgs& a, const Tile& t, f32x4_t (*part)[NT][64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const int f = wave % NT, kw = wave / NT;
  const int n_out = a.swiglu ? a.N / 2 : a.N;
  const int c0 = t.nb * (a.swiglu ? 8 * NT : 16 * NT);
  const int64_t K = a.K;
  const int64_t wrow_b = WF == MC_BF16 ? 2 * K : K / 2, xrow_b = XF == MC_BF16 ? 2 * a.ldx : K / 2;
  const int nblk = a.K / 32;
  const int steps = WF == MC_BF16 ? nblk : (nblk + 3) / 4;
  constexpr int HT = NT > 1 ? NT / 2 : 1;
  const int wrow = NT > 1 && a.swiglu ? min(c0 + (f % HT) * 16 + l16, n_out - 1) + (f >= HT ? n_out : 0)
                                      : min(c0 + f * 16 + l16, n_out - 1);
  const uint8_t* wp = a.w + ((int64_t)t.entry * a.N + wrow) * wrow_b;
  const uint8_t* wsp = a.ws + ((int64_t)t.entry * a.N + wrow) * (K / 32);
  const int i_row = t.row0 + min(l16, t.nrows - 1);
  const int64_t xr = max(x_row(a, i_row, a.perm ? a.perm[i_row] : i_row), 0);
  const uint8_t* xp = a.x + xr * xrow_b;
  const uint8_t* xsp = a.xs + xr * (K / 32);

  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = kw; s0 < steps; s0 += KW * STEPS) {
    u32x4_t w[STEPS];
    uint32_t sw[STEPS];
    // steps and blocks past the end re-read the last ones and count as zeros
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
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
    for (int u = 0; u < STEPS; ++u) {
      const int s = min(s0 + u * KW, steps - 1);
      const bool in = s0 + u * KW < steps && (WF == MC_BF16 || 4 * s + g < nblk);
      const int b = WF == MC_BF16 ? s : min(4 * s + g, nblk - 1);
      if (!in) w[u] = u32x4_t{0, 0, 0, 0};
      if (WF == MC_BF16) {
        u32x4_t x = *reinterpret_cast<const u32x4_t*>(xp + (int64_t)b * 64 + 16 * g);
        if (!in) x = u32x4_t{0, 0, 0, 0};         // a zero times an infinity is no zero
        acc = mfma_bf16(w[u], x, acc);
      } else if (XF == MC_MXFP4) {
        const u32x4_t x = *reinterpret_cast<const u32x4_t*>(xp + (int64_t)b * 16);
        const uint32_t sx = xsp[b];
        acc = mfma_fp4(w[u], in ? sw[u] : 127u, x, in ? sx : 127u, acc);
      } else {
        // the K order of the four products is permuted: lane group g holds block b of its row
        const float s32 = in ? e8m0_or_nan(sw[u]) : 1.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u32x4_t x = *reinterpret_cast<const u32x4_t*>(xp + (int64_t)b * 64 + 16 * j);
          if (!in) x = u32x4_t{0, 0, 0, 0};
          acc = mfma_bf16(__builtin_bit_cast(u32x4_t, fp4x8_bf16(w[u][j], s32)), x, acc);
        }
      }
    }
  }
  part[kw][f][lane] = acc;
  __syncthreads();
  if (wave > 0) return;
  f32x4_t v[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    v[q] = part[0][q][lane];
#pragma unroll
    for (int k = 1; k < KW; ++k) v[q] += part[k][q][lane];
  }
  const bool on = l16 < t.nrows;
  RowOut o;
  rows_out<1>(a, &i_row, &on, &o);
  with_format(a, [&](auto yf, auto vec) {
    constexpr int YF = decltype(yf)::value;
    constexpr bool VEC = decltype(vec)::value;
    if (a.swiglu) {
      if constexpr (NT == 4) store_pair<YF, VEC>(a, o, c0, n_out, swiglu4(v[0], v[2]), swiglu4(v[1], v[3]));
      else if constexpr (NT == 2) store_one<YF, VEC>(a, o, c0, n_out, swiglu4(v[0], v[1]));
    } else if constexpr (NT == 1) {
      store_one<YF, VEC>(a, o, c0, n_out, v[0]);
    } else {
#pragma unroll
      for (int q = 0; q < NT; q += 2) store_pair<YF, VEC>(a, o, c0 + 16 * q, n_out, v[q], v[q + 1]);
    }
  });
}

template <int XF, int WF, int NT, int KW, int STEPS>
__global__ void __launch_bounds__(64 * NT * KW)
product_few_kernel(ProductArgs a, int n_nb, uint32_t tiles) {
  __shared__ f32x4_t part[KW][NT][64];
  for (uint32_t b = blockIdx.x;;) {
    Tile t;
    if (!find_tile<16>(a, b, n_nb, &t)) return;
    few_tile<XF, WF, NT, KW, STEPS>(a, t, part);
    b += gridDim.x;
    if (b >= tiles) return;
    __syncthreads();                               // the sums have been read
  }
}

// ---------------------------------------------------------------- many rows
//
// BM rows x BN weight rows (SwiGLU: BN / 2 gate and the matching up rows) per workgroup of WM waves
// along the rows x WN along the weight rows: a wave multiplies MF 16-row fragments (rows
// 16 (WM f + wm) of the tile, so that a tile of fewer rows runs fewer fragments in every wave
// alike) with 64 weight rows (32 at 32 wn of each half of the weight tile: with SwiGLU the
// gate rows and their up rows).  K moves in stages of 128 bytes per row, a whole cache line
// (with 64 the requests to L2, not its bytes, bound the product), through two LDS buffers
// (global_load_lds, no registers): stage s + 1 is requested when stage s begins, one barrier
// per stage.  A row's eight 16-byte chunks are stored at chunk c ^ (row % 8), with which the
// operand reads run at the LDS's full rate (218 of 256 B/clk measured, 62 without).
//
// kBf16: bf16 x bf16, 64 elements per stage.  kFp4: MXFP4 x MXFP4, 256 elements per stage.
// kA16W4: bf16 rows, 64 elements per stage; the weights' codes come in every four stages and
// become bf16 when a wave reads its fragment.  Scale bytes come in 16 per row at a time, like
// the operands, where every row's scales are 16-byte aligned and K is a multiple of 512 (SDMA);
// else a stage's 8 (2) per row through a register, loaded two stages ahead and stored behind
// the barrier in between, which has waited for every load anyway.
//
// Where few tiles would leave the chip empty, K is shared out among KG groups of waves, each with
// buffers of its own, whose sums meet in LDS.
//
// What bounds it: in fp4 the 8192 x 4096 x 4096 product's stage (256 x 256 x 256) takes 1.9 us, 1.5
// without its loads and 1.3 without its products, which are 0.9 us of MFMA time at 2.2 GHz: the LDS
// serves 192 KiB of operands, 24 of scales and 72 of arriving data in it.  A wave tile of 128 x 128
// (one wave per SIMD) reads a third less and took 2.3 us a stage; 64-byte stages four deep 1.7
// times as many L2 requests and 106 against 92 us a product.  That is one dense product, all of whose
// tiles run the same code.  Every form of results is compiled into every number of row fragments:
// the 256 x 256 kernels have 470-485 KB of code, those of 128 x 128 130-148 and those of 64 x 64 44-48,
// the first two of more than the instruction cache holds, so groups of uneven sizes, whose
// tiles differ in fragments, fetch each epilogue anew; what that costs has not been measured.  The
// 256 x 256 kernels with MXFP4 weights fill all 256 VGPRs and spill up to 6 of them, and they and
// the 128 x 128 ones without K groups keep 83-113 SGPRs in lanes of VGPRs.

enum { kBf16 = 0, kA16W4 = 1, kFp4 = 2 };

template <int WM_, int WN_, int NF_, int MFX_, int KG_, int PER_CU_>
struct WideShape {
  static constexpr int WM = WM_, WN = WN_, NF = NF_, MFX = MFX_, KG = KG_;
  static constexpr int BM = 16 * WM * MFX, BN = 16 * NF * WN;
  static constexpr int group = 64 * WM * WN, threads = group * KG;   // of a K group, of the workgroup
  static constexpr int resident = 256 * PER_CU_;             // workgroups that the chip holds at once
  static constexpr int waves = PER_CU_ * threads / 256;      // per SIMD
};

// At most VM loads outstanding, every LDS access done, then the workgroup's barrier.
template <int VM>
__device__ __forceinline__ void wait_stage() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((VM & 15) | (7 << 4) | ((VM >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

typedef __attribute__((address_space(3))) void* lds_ptr;

__device__ __forceinline__ uint32_t lds_offset(void* p) { return (uint32_t)(uintptr_t)(lds_ptr)p; }

// 16 bytes per lane from base + off into LDS at offset dst + 16 lane; base and dst are the same for the
// wave.  Written as an instruction with no register result: the compiler's builtin makes every
// later LDS read wait for all such loads, those for the other buffer among them.  The reader's
// wait is wait_stage's; the compiler's own waits for other loads count these as unknown older or
// newer ones, which can only make them longer.
__device__ __forceinline__ void load_lds16(const uint8_t* base, uint32_t off, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(dst), "v"(off), "s"(base)
               : "memory", "m0");
}
// The same from an address of the lane's own; 4 bytes per lane.
__device__ __forceinline__ void load_lds16(const uint8_t* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(dst), "v"(src) : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(const void* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(dst), "v"(src) : "memory", "m0");
}

// N (2 or 8) scale bytes of a row of n blocks from block b on, at any alignment (blocks past the last
// count as 2^0): load() is one load, whose wait comes with value().
template <int N>
struct Scales {
  uint64_t raw;
  __device__ __forceinline__ void load(const uint8_t* row, int b, int n) {   // n >= N
    raw = 0;
    __builtin_memcpy(&raw, row + min(b, n - N), N);
  }
  __device__ __forceinline__ uint64_t value(int b, int n) const {
    const uint64_t none = 0x7F7F7F7F7F7F7F7Full;
    const int d = b - min(b, n - N);              // bytes that were read too early
    return d == 0 ? raw : d >= N ? none : (raw >> (8 * d)) | (none << (8 * (N - d)));
  }
  // the first N bytes of a row of any length
  __device__ __forceinline__ static uint64_t first(const uint8_t* row, int n) {
    uint64_t v = 0x7F7F7F7F7F7F7F7Full;
    if (n >= N) {
      __builtin_memcpy(&v, row, N);
    } else {
      for (int i = 0; i < n; ++i) v = (v & ~(0xFFull << (8 * i))) | ((uint64_t)row[i] << (8 * i));
    }
    return v;
  }
};

template <int MODE, class S>
struct WideRing {
  uint8_t x[2][S::BM * 128];
  uint8_t w[2][S::BN * 128];
  // scales of the weight rows, then (MXFP4) of the rows, 16 bytes each
  uint8_t s[MODE == kBf16 ? 1 : 2][MODE == kBf16 ? 16 : (S::BN + (MODE == kFp4 ? S::BM : 0)) * 16];
};
template <int MODE, class S>
struct WideLds {
  WideRing<MODE, S> ring[S::KG];
  int perm[S::KG == 1 ? S::BM : 1];               // routes of the next tile's rows
  int first[kMaxGroups + 1];
};

// The stages of a row that a K group takes: from `from` on, `n` of them (`most` in the first group,
// which has the most).  Shares are multiples of what the weights or the scales come in for, so they are
// uneven, and groups of a short row get nothing: bf16 x MXFP4 takes K = 2080 in 20 and 13 stages,
// or in 12, 12, 9 and none, and K = 512 whole.
template <int MODE, class S, bool SDMA>
struct WideShare {
  int from, n, most;
  __device__ __forceinline__ WideShare(int stages, int kg) {
    // scales (SDMA) and kA16W4's weights come in for so many stages at a time
    constexpr int align = MODE == kFp4 && SDMA ? 2 : MODE != kA16W4 ? 1 : SDMA ? 8 : 4;
    const int per = S::KG == 1 ? stages : div_up(div_up(stages, S::KG), align) * align;
    from = S::KG == 1 ? 0 : kg * per;
    n = S::KG == 1 ? stages : min(max(stages - from, 0), per);
    most = S::KG == 1 ? stages : min(stages, per);
  }
};

// What a thread loads of a tile: its 16 bytes of every stage, of rows tid / 8 + RQ q, and the scales
// of one row.
template <int MODE, class S>
struct WideSource {
  static constexpr int T = S::group, RQ = T / 8, WQ = S::BN / RQ, XQ = S::BM / RQ;
  static constexpr int SR = MODE == kBf16 ? 0 : S::BN + (MODE == kFp4 ? S::BM : 0);
  static constexpr int SQ = SR == 0 ? 1 : div_up(SR, T);      // rows of scales per thread: tid + T q
  // offsets (32 bits: launch_by_size checks that a matrix and x are that small) from the group's
  // matrix and from x, or, where a tile's rows lie one behind the other, from the first of them; the
  // scales' address
  const uint8_t *wbase, *xbase, *s[SQ];
  uint32_t w[WQ], x[XQ];

  // perm: the routes of the tile's rows (any pointer; unused without a.x_perm).
  template <class P>
  __device__ __forceinline__ void point(const ProductArgs& a, const Tile& t, int ch, int from, P perm) {
    constexpr int HN = S::BN / 2;
    const int tid = threadIdx.x % T;
    // where stage `from` begins: bytes of x and of the weights, scale bytes
    const int x0 = from * 128, w0 = MODE == kA16W4 ? from * 32 : from * 128, s0 = from * (MODE == kFp4 ? 8 : 2);
    // rows outside x are read as its first (last, without x_perm) one
    const int x_first = a.x_perm ? 0 : min(t.row0, a.x_rows - 1);
    auto x_at = [&](int r) {
      const int m = min(r, t.nrows - 1), i = t.row0 + m;
      return a.x_perm ? max(x_row(a, i, perm[m]), 0) : min(i, a.x_rows - 1) - x_first;
    };
    const int n_out = a.swiglu ? a.N / 2 : a.N, c0 = t.nb * (a.swiglu ? HN : S::BN);
    const int64_t K = a.K;
    const uint32_t wrow_b = MODE == kBf16 ? 2 * a.K : a.K / 2, xrow_b = MODE == kFp4 ? a.K / 2 : 2 * (uint32_t)a.ldx;
    auto w_row = [&](int r) {
      return a.swiglu ? min(c0 + r % HN, n_out - 1) + (r >= HN ? n_out : 0) : min(c0 + r, n_out - 1);
    };
    wbase = a.w + (int64_t)t.entry * a.N * wrow_b;
    xbase = a.x + (int64_t)x_first * xrow_b;
#pragma unroll
    for (int q = 0; q < WQ; ++q) w[q] = w_row(q * RQ + (tid >> 3)) * wrow_b + w0 + ch * 16;
#pragma unroll
    for (int q = 0; q < XQ; ++q) x[q] = x_at(q * RQ + (tid >> 3)) * xrow_b + x0 + ch * 16;
    if (MODE != kBf16) {
#pragma unroll
      for (int q = 0; q < SQ; ++q) {
        const int r = q * T + tid;
        if (MODE == kFp4 && r >= S::BN) s[q] = a.xs + ((int64_t)x_first + x_at(r - S::BN)) * (K / 32) + s0;
        else s[q] = a.ws + ((int64_t)t.entry * a.N + w_row(min(r, S::BN - 1))) * (K / 32) + s0;
      }
    }
  }
};

// Buffers that the stages, the weights (kA16W4: every four stages) and the scales of a tile begin in.
struct WideTurn {
  int stage, w, s;
};

template <int MODE, class S, bool SDMA, int MF>
__device__ __forceinline__ void wide_tile(const ProductArgs& a, int n_nb, WideLds<MODE, S>& all, const Tile& t,
                                          WideSource<MODE, S>& src, WideTurn& turn, Scales<MODE == kFp4 ? 8 : 2>* sc,
                                          bool more, int b, int total, Tile& next, uint32_t wdst, uint32_t xdst,
                                          uint32_t sdst) {
  constexpr int WM = S::WM, HN = S::BN / 2, T = S::group, RQ = T / 8, KG = S::KG;
  constexpr int WQ = S::BN / RQ, XQ = (MF * 16 * WM + RQ - 1) / RQ;
  constexpr int SR = WideSource<MODE, S>::SR, SQ = WideSource<MODE, S>::SQ, NF = S::NF;
  constexpr int period = MODE == kFp4 ? 2 : 8;               // stages that one load of scales covers
  const int tid = threadIdx.x % T, lane = tid & 63, wave = tid >> 6, g = lane >> 4, l16 = lane & 15;
  const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / T);
  WideRing<MODE, S>& lds = all.ring[kg];
  const int wm = wave % WM, wn = wave / WM;
  const int n_out = a.swiglu ? a.N / 2 : a.N;
  const int c0 = t.nb * (a.swiglu ? HN : S::BN);
  // bytes of a row, and its stages and blocks, from where the K group begins
  const int row_b = MODE == kFp4 ? a.K / 2 : 2 * a.K;
  const WideShare<MODE, S, SDMA> share((row_b + 127) / 128, kg);
  const int stages = share.n;
  const int xb = row_b - share.from * 128, wb = MODE == kA16W4 ? a.K / 2 - share.from * 32 : xb;
  const int nblk = a.K / 32 - share.from * (MODE == kFp4 ? 8 : 2);
  const int ch = (tid & 7) ^ ((tid >> 3) & 7);
  const uint32_t pdst = __builtin_amdgcn_readfirstlane(lds_offset(&all.perm[0]) + wave * 256);

  // Scales of period p straight into LDS; or of stage s, in two steps through a register.
  auto request_scales = [&](int p, int at) {
#pragma unroll
    for (int q = 0; q < SQ; ++q)
      if (SR % T == 0 || q * T + wave * 64 < SR)
        load_lds16(src.s[q] + p * 16, sdst + ((p + at) & 1) * sizeof(lds.s[0]) + q * T * 16);
  };
  constexpr int SN = MODE == kFp4 ? 8 : 2;
  auto put_scales = [&](int s, int q, uint64_t v) {
    if (SR % T == 0 || q * T + tid < SR) __builtin_memcpy(&lds.s[(s + turn.stage) & 1][(q * T + tid) * 16], &v, SN);
  };
  // Stage s: 128 bytes of every weight row (kA16W4: four stages of x), of every row of x; a chunk past
  // the row's end (only in the last stage) re-reads the row's first bytes.
  auto request_w = [&](int s, int at) {
    const uint32_t dst = wdst + ((s + at) & 1) * S::BN * 128;
    if ((s + 1) * 128 <= wb) {
#pragma unroll
      for (int q = 0; q < WQ; ++q) load_lds16(src.wbase + s * 128, src.w[q], dst + q * RQ * 128);
    } else {
      const uint32_t off = s * 128 + ch * 16 < wb ? s * 128 : -(uint32_t)(ch * 16);
#pragma unroll
      for (int q = 0; q < WQ; ++q) load_lds16(src.wbase, src.w[q] + off, dst + q * RQ * 128);
    }
  };
  auto request_x = [&](int s, int at, int q) {
    const uint32_t dst = xdst + (((s + at) & 1) * S::BM + q * RQ) * 128;
    if ((s + 1) * 128 <= xb)
      load_lds16(src.xbase + s * 128, src.x[q], dst);
    else
      load_lds16(src.xbase, src.x[q] + (s * 128 + ch * 16 < xb ? s * 128 : -(uint32_t)(ch * 16)), dst);
  };

  f32x4_t acc[NF][MF];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int m = 0; m < MF; ++m) acc[f][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const int swz = l16 & 7;
  // The products of stage s: two halves of 64 bytes (the second missing where the row ends), of each
  // NF weight fragments x MF row fragments.  The next row fragment is read from LDS, and a weight
  // fragment of the second half, ahead of each row fragment's products; left free, the scheduler
  // sinks every read to its use, with its latency in between.
  auto compute = [&](int s, bool two) {
    // buffer and place of the stage's scales
    const int sb = (SDMA ? s / period + turn.s : s + turn.stage) & 1, so = SDMA ? s % period * SN : 0;
    const int b = (s + turn.stage) & 1;
    const int at[2] = {l16 * 128 + ((g ^ swz) << 4), l16 * 128 + (((4 + g) ^ swz) << 4)};
    u32x4_t w[2][NF], x[2];
    uint32_t sw[2][NF], sx[2];
    auto read_w = [&](int kk, int f) {
      const int row = f / (NF / 2) * HN + f % (NF / 2) * 16 + wn * (8 * NF);
      if constexpr (MODE == kA16W4) {
        // elements 8 g .. 8 g + 7 of a block: one dword of its chunk
        const int c = ((s >> 2) + turn.w) & 1, j = (s & 3) * 2 + kk;
        w[kk][f][0] = *reinterpret_cast<const uint32_t*>(&lds.w[c][(row + l16) * 128 + ((j ^ swz) << 4) + g * 4]);
        sw[kk][f] = lds.s[sb][(row + l16) * 16 + so + kk];
      } else {
        w[kk][f] = *reinterpret_cast<const u32x4_t*>(&lds.w[b][row * 128 + at[kk]]);
        // both halves' scales in one read (8192 x 4096 x 4096 83.0 -> 82.2 us; the row fragments' too, 99: the
        // registers that they stay in until the second half are not there)
        if (MODE == kFp4 && kk == 0) {
          const uint2 v = *reinterpret_cast<const uint2*>(&lds.s[sb][(row + l16) * 16 + so]);
          sw[0][f] = v.x;
          sw[1][f] = v.y;
        }
      }
    };
    auto read_x = [&](int kk, int m) {
      const int row = (m * WM + wm) * 16;
      x[m & 1] = *reinterpret_cast<const u32x4_t*>(&lds.x[b][row * 128 + at[kk]]);
      if constexpr (MODE == kFp4)
        sx[m & 1] = *reinterpret_cast<const uint32_t*>(&lds.s[sb][(S::BN + row + l16) * 16 + so + kk * 4]);
    };
    auto half = [&](auto k) {
      constexpr int kk = decltype(k)::value;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        if constexpr (MODE == kA16W4)
          w[kk][f] = __builtin_bit_cast(u32x4_t, fp4x8_bf16(w[kk][f][0], e8m0_or_nan(sw[kk][f])));
        else if constexpr (MODE == kFp4)
          sw[kk][f] >>= 8 * g;
      }
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        if (m + 1 < MF) read_x(kk, m + 1);
        if (kk == 0) {
#pragma unroll
          for (int f = m * NF / MF; f < (m + 1) * NF / MF; ++f) read_w(1, f);
        }
        __builtin_amdgcn_sched_barrier(0);
        const uint32_t sxm = MODE == kFp4 ? sx[m & 1] >> (8 * g) : 0;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          if constexpr (MODE == kFp4) acc[f][m] = mfma_fp4(w[kk][f], sw[kk][f], x[m & 1], sxm, acc[f][m]);
          else acc[f][m] = mfma_bf16(w[kk][f], x[m & 1], acc[f][m]);
        }
      }
    };
#pragma unroll
    for (int f = 0; f < NF; ++f) read_w(0, f);
    read_x(0, 0);
    half(Const<0>());
    if (two) {
      read_x(1, 0);
      half(Const<1>());
    }
  };

  for (int s = 0; s < share.most; ++s) {
    const bool last = s + 1 == stages;
    if (MODE == kFp4 && last && xb < stages * 128) {
      // chunks past the row's end count as zeros: of one operand, since every e2m1 code is finite
      __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));
      asm volatile("" ::: "memory");
      if (s * 128 + ch * 16 >= wb) {
#pragma unroll
        for (int q = 0; q < WQ; ++q)
          *reinterpret_cast<u32x4_t*>(&lds.w[(s + turn.stage) & 1][q * RQ * 128 + tid * 16]) = u32x4_t{0, 0, 0, 0};
      }
    }
    // stage s is in; of a tile's first stage every wave has made sure before it stored the last
    // tile's results, which may still be on their way
    if (s == 0) wait_stage<63>();
    else wait_stage<0>();
    if (s + 1 < stages) {
      if (MODE != kBf16 && !SDMA) {
#pragma unroll
        for (int q = 0; q < SQ; ++q) {
          put_scales(s + 1, q, sc[q].value((s + 1) * SN, nblk));
          sc[q].load(src.s[q], (s + 2) * SN, nblk);
        }
      }
      if (MODE == kFp4 && SDMA && (s + 1) % period == 0) request_scales((s + 1) / period, turn.s);
      if (MODE == kA16W4 && (s & 3) == 0 && s + 4 < stages) {
        if (SDMA && (s & 7) == 4) request_scales((s >> 3) + 1, turn.s);
        request_w((s >> 2) + 1, turn.w);
      }
      if (MODE != kA16W4) request_w(s + 1, turn.stage);
#pragma unroll
      for (int q = 0; q < XQ; ++q) request_x(s + 1, turn.stage, q);
    }
    // The workgroup's next tile: looked up while the first stage is computed, its first stage
    // requested while the last one is.  No vector load into registers here: the compiler would
    // wait for it, and so for the stage on its way, before this stage's products.
    if (KG == 1 && s == 0 && more) {
      next_tile<S::BM>(a, b, total, n_nb, all.first, &next);
      if (a.x_perm && wave * 64 < S::BM)
        load_lds4(a.perm + next.row0 + min(tid, next.nrows - 1), pdst);
    }
    if (KG == 1 && last && more) {
      if (stages == 1) wait_stage<0>();
      src.point(a, next, ch, 0, all.perm);
      const int sn = turn.stage + stages;
      if (MODE != kBf16 && SDMA) request_scales(0, turn.s + (stages + period - 1) / period);
      request_w(0, MODE == kA16W4 ? turn.w + (stages + 3) / 4 : sn);
#pragma unroll
      for (int q = 0; q < S::BM / RQ; ++q)
        if (q * RQ < next.nrows) request_x(0, sn, q);
    }
    if (KG == 1 || s < stages) compute(s, MODE == kFp4 || s * 128 + 64 < xb);
  }
  turn.stage += stages;
  turn.s += (stages + period - 1) / period;
  turn.w += (stages + 3) / 4;
  if (MODE != kBf16 && !SDMA && KG == 1 && more) {
#pragma unroll
    for (int q = 0; q < SQ; ++q) {
      put_scales(0, q, Scales<SN>::first(src.s[q], nblk));
      if (stages > 1) sc[q].load(src.s[q], SN, nblk);
    }
  }

  if constexpr (KG > 1) {
    // the groups' sums meet in LDS, added in the order of K
    static_assert(sizeof(all.ring) >= (size_t)(KG - 1) * T * NF * S::MFX * 16, "room for the partial sums");
    f32x4_t(*part)[NF * MF][T] = reinterpret_cast<f32x4_t(*)[NF * MF][T]>(&all.ring[0]);
    wait_stage<0>();
    if (kg > 0) {
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int m = 0; m < MF; ++m) part[kg - 1][f * MF + m][tid] = acc[f][m];
    }
    wait_stage<0>();
    if (kg > 0) return;
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int k = 1; k < KG; ++k) acc[f][m] += part[k - 1][f * MF + m][tid];
  }

  int row[MF];
  bool on[MF];
  RowOut o[MF];
#pragma unroll
  for (int m = 0; m < MF; ++m) {
    const int r = (m * WM + wm) * 16 + l16;
    row[m] = t.row0 + min(r, t.nrows - 1);
    on[m] = r < t.nrows;
  }
  rows_out<MF>(a, row, on, o);
  __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));          // the next tile's first stage
  asm volatile("" ::: "memory");
  with_format(a, [&](auto yf, auto vec) {
    constexpr int YF = decltype(yf)::value;
    constexpr bool VEC = decltype(vec)::value;
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      const int col = c0 + wn * (8 * NF);
#pragma unroll
      for (int f = 0; f < NF / 2; f += 2) {
        if (a.swiglu) {
          store_pair<YF, VEC>(a, o[m], col + f * 16, n_out, swiglu4(acc[f][m], acc[NF / 2 + f][m]),
                              swiglu4(acc[f + 1][m], acc[NF / 2 + f + 1][m]));
        } else {
          store_pair<YF, VEC>(a, o[m], col + f * 16, n_out, acc[f][m], acc[f + 1][m]);
          store_pair<YF, VEC>(a, o[m], col + HN + f * 16, n_out, acc[NF / 2 + f][m], acc[NF / 2 + f + 1][m]);
        }
      }
    }
  });
}

// A workgroup takes tiles blockIdx.x, blockIdx.x + gridDim.x, ... (the grid is as large as the chip
// holds at once): the first stage of its next tile arrives while it finishes the last one.
template <int MODE, class S, bool SDMA>
__global__ void __launch_bounds__(S::threads, S::waves)
product_wide_kernel(ProductArgs a, int n_nb) {
  __shared__ __attribute__((aligned(16))) WideLds<MODE, S> lds;
  int total;
  if (a.offsets) {
    if (threadIdx.x < 64) first_tiles<S::BM>(a, lds.first);
    __syncthreads();
    total = __builtin_amdgcn_readfirstlane(lds.first[a.E]) * n_nb;
  } else {
    total = div_up(a.M, S::BM) * n_nb;
  }
  int b = blockIdx.x;
  if (b >= total) return;
  Tile t;
  next_tile<S::BM>(a, b, total, n_nb, lds.first, &t);
  constexpr int T = S::group, RQ = T / 8, SR = WideSource<MODE, S>::SR, SQ = WideSource<MODE, S>::SQ;
  constexpr int SN = MODE == kFp4 ? 8 : 2;
  const int tid = threadIdx.x % T, wave = tid >> 6;
  const int kg = S::KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / T);
  WideRing<MODE, S>& ring = lds.ring[kg];
  const int ch = (tid & 7) ^ ((tid >> 3) & 7);
  const uint32_t wdst = __builtin_amdgcn_readfirstlane(lds_offset(&ring.w[0][wave * 1024]));
  const uint32_t xdst = __builtin_amdgcn_readfirstlane(lds_offset(&ring.x[0][wave * 1024]));
  const uint32_t sdst = __builtin_amdgcn_readfirstlane(lds_offset(&ring.s[0][0]) + wave * 1024);
  const int row_b = MODE == kFp4 ? a.K / 2 : 2 * a.K;
  const WideShare<MODE, S, SDMA> share((row_b + 127) / 128, kg);
  const int xb = row_b - share.from * 128, wb = MODE == kA16W4 ? a.K / 2 - share.from * 32 : xb;
  const int nblk = a.K / 32 - share.from * (MODE == kFp4 ? 8 : 2);
  WideSource<MODE, S> src;
  Scales<SN> sc[SQ] = {};
  if (S::KG == 1 || share.n > 0) {
    // the first tile's first stage
    src.point(a, t, ch, share.from, a.perm + t.row0);
    if (MODE != kBf16) {
#pragma unroll
      for (int q = 0; q < SQ; ++q) {
        if (SDMA) {
          if (SR % T == 0 || q * T + wave * 64 < SR) load_lds16(src.s[q], sdst + q * T * 16);
        } else {
          const uint64_t v = Scales<SN>::first(src.s[q], nblk);
          if (SR % T == 0 || q * T + tid < SR) __builtin_memcpy(&ring.s[0][(q * T + tid) * 16], &v, SN);
          if (share.n > 1) sc[q].load(src.s[q], SN, nblk);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < S::BN / RQ; ++q)
      load_lds16(src.wbase, src.w[q] - (ch * 16 < wb ? 0 : ch * 16), wdst + q * RQ * 128);
#pragma unroll
    for (int q = 0; q < S::BM / RQ; ++q)
      if (q * RQ < t.nrows) load_lds16(src.xbase, src.x[q] - (ch * 16 < xb ? 0 : ch * 16), xdst + q * RQ * 128);
  }
  __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));
  asm volatile("" ::: "memory");

  WideTurn turn{0, 0, 0};
  for (;;) {
    b += gridDim.x;
    const bool more = S::KG == 1 && b < total;     // with K groups every tile has its own workgroup
    Tile next = t;
    // fragments that the tile's rows need of every wave, the same for the whole workgroup
    const int steps = div_up(t.nrows, 16 * S::WM);
    auto run = [&](auto mf) {
      wide_tile<MODE, S, SDMA, decltype(mf)::value>(a, n_nb, lds, t, src, turn, sc, more, b, total, next, wdst, xdst, sdst);
    };
    // without direct scales two forms only, which keep the 256 x 256 kernel at 161 instead of 485 KB
    // of code: a tile of 150 rows then computes 256
    if constexpr (!SDMA || S::MFX == 2) {
      if (2 * steps <= S::MFX) run(Const<S::MFX / 2>());
      else run(Const<S::MFX>());
    } else if (S::MFX > 4 && steps > 4) {
      if (steps == 8) run(Const<S::MFX>());
      else if (steps == 7) run(Const<S::MFX - S::MFX / 8>());
      else if (steps == 6) run(Const<S::MFX - S::MFX / 4>());
      else run(Const<S::MFX / 2 + S::MFX / 8>());
    } else {
      if (steps == 4) run(Const<4>());
      else if (steps == 3) run(Const<3>());
      else if (steps == 2) run(Const<2>());
      else run(Const<1>());
    }
    if (!more) return;
    t = next;
  }
}

// ---------------------------------------------------------------- launch

// Row tiles of all groups together, at most: sum over groups of ceil(rows / bm).
inline int64_t most_row_tiles(const ProductArgs& a, int64_t bm) {
  return a.offsets ? a.M / bm + (a.E < a.M ? a.E : a.M) : (a.M + bm - 1) / bm;
}

template <int XF, int WF>
int launch_few(const ProductArgs& a, hipStream_t s) {
  const int64_t n_out = a.swiglu ? a.N / 2 : a.N, rt = most_row_tiles(a, 16);
  // as narrow as the epilogue allows (a block of quantised results is 32 columns) where 32 columns
  // would not fill the chip (8 x 4096 x 4096: 7 against 11 us)
  const int nt = a.swiglu ? (a.y_fmt == MC_MXFP4 ? 4 : 2) : a.y_fmt != MC_MXFP4 && rt * ((n_out + 31) / 32) <= 256 ? 1 : 2;
  const int64_t cols = a.swiglu ? 8 * nt : 16 * nt;
  const int64_t n_nb = (n_out + cols - 1) / cols, tiles = rt * n_nb;
  MC_REQUIRE(tiles <= 0x7FFF0000, "product of %d rows with %d columns is too large", a.M, a.N);
  const int steps = WF == MC_BF16 ? a.K / 32 : (a.K + 127) / 128;
  auto run = [&](auto kernel, int kw) {
    const int64_t most = UINT32_MAX / (64 * nt * kw);
    hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles < most ? tiles : most)), dim3(64 * nt * kw), 0, s, a, (int)n_nb,
                       (uint32_t)tiles);
  };
  // Waves along K x steps in flight per wave: loads of steps past the end cost what others do, so both
  // follow K (one token 4096 x 2048 4.5 us in 8 x 2, 5.8 in 8 x 4, 4.6 in 16 x 1; 8 x 8192 x 2048 7.1 /
  // 11.8 / 8.3; one token's eight experts 1024 x 2048 7.3 in 4 x 4, 7.6 in 8 x 2; 2048 x 512 8.8 / 8.3
  // and 6.6 in 4 x 2).
  if (nt == 4) run(product_few_kernel<XF, WF, 4, 4, 4>, 4);
  else if (nt == 1 && steps <= 16) run(product_few_kernel<XF, WF, 1, 8, 2>, 8);
  else if (nt == 1) run(product_few_kernel<XF, WF, 1, 8, 4>, 8);
  else if (steps <= 8) run(product_few_kernel<XF, WF, 2, 4, 2>, 4);
  else if (steps <= 16) run(product_few_kernel<XF, WF, 2, 4, 4>, 4);
  else run(product_few_kernel<XF, WF, 2, 8, 4>, 8);
  MC_LAUNCH_CHECK();
  return MC_OK;
}

template <int MODE, class S>
int launch_wide(const ProductArgs& a, hipStream_t s) {
  const int64_t n_out = a.swiglu ? a.N / 2 : a.N, cols = a.swiglu ? S::BN / 2 : S::BN;
  const int64_t n_nb = (n_out + cols - 1) / cols, tiles = most_row_tiles(a, S::BM) * n_nb;
  MC_REQUIRE(tiles <= 0x7FFF0000, "product of %d rows with %d columns is too large", a.M, a.N);
  const int64_t grid = S::KG > 1 || tiles < S::resident ? tiles : S::resident;
  const bool sdma = a.K % 512 == 0 && ((uintptr_t)a.xs | (uintptr_t)a.ws) % 16 == 0;
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(S::threads), 0, s, a, (int)n_nb);
  };
  if constexpr (MODE == kBf16) {
    run(product_wide_kernel<MODE, S, true>);
  } else {
    if (sdma) run(product_wide_kernel<MODE, S, true>);
    else run(product_wide_kernel<MODE, S, false>);
  }
  MC_LAUNCH_CHECK();
  return MC_OK;
}

// Tiles of a shape, at most.
template <class S>
int64_t most_tiles(const ProductArgs& a) {
  const int64_t n_out = a.swiglu ? a.N / 2 : a.N, cols = a.swiglu ? S::BN / 2 : S::BN;
  return most_row_tiles(a, S::BM) * ((n_out + cols - 1) / cols);
}

typedef WideShape<2, 4, 4, 8, 1, 1> Big;          // 256 x 256, one workgroup per CU
typedef WideShape<2, 2, 4, 4, 1, 2> Medium;       // 128 x 128, two per CU
typedef WideShape<2, 2, 4, 4, 2, 1> Medium2;      // 128 x 128, K in two parts
typedef WideShape<2, 1, 4, 2, 2, 2> Small2;       // 64 x 64, K in two parts, two per CU
typedef WideShape<2, 1, 4, 2, 4, 1> Small4;       // 64 x 64, K in four parts

// f(a value of the shape's type) for a product's sizes; f(nullptr): tiles of 16 rows (launch_few).
template <class F>
int with_shape(const ProductArgs& a, F f) {
  // bytes of a matrix and of x (of a tile's rows of it, if they lie one behind the other), which the
  // wide kernels reach with 32-bit offsets (beyond, the tiles of 16 rows read with 64-bit ones)
  const int64_t w_bytes = (int64_t)a.N * (a.w_fmt == MC_BF16 ? 2 * (int64_t)a.K : a.K / 2);
  const int64_t x_bytes = (a.x_perm ? a.x_rows : Big::BM) * (a.x_fmt == MC_BF16 ? 2 * a.ldx : a.K / 2);
  // Up to 16 rows: one token's experts 8 us (12 in Small4), 8 x 4096 x 4096 7 us (16); from 17 rows on
  // Small4 is level or ahead (17 x 4096 x 2048 bf16: 8 against 12 us, 64 x 4096 x 4096: 19 against
  // 35 us; products of one group.  Of grouped ones both sides have not been compared: with eight
  // routes a token, bf16 x MXFP4 1024 x 2048, 2 tokens take 11 us in tiles of 16 rows, 3 take 18, 4 18
  // and 8 32 in the others).
  if (a.M > 16 && w_bytes <= UINT32_MAX && x_bytes <= UINT32_MAX) {
    // The large tiles read each operand half as often, and win where they fill the chip with full
    // tiles: 8192 x 4096 x 4096 in fp4 86 against 101 us, 256 experts of 192 rows 1.40 against
    // 1.68 ms a layer.  Where groups are small or uneven the 128 x 128 ones win: 24 rows a group
    // 268 against 276 us, 64 groups of 250 rows on average, skewed, 207 against 231 us.
    const int64_t groups = a.offsets ? (a.E < a.M ? a.E : a.M) : 1;
    const int64_t n_nb = most_tiles<Big>(a) / most_row_tiles(a, Big::BM);
    const int64_t big = (a.offsets ? a.M / Big::BM + groups / 2 : (a.M + Big::BM - 1) / Big::BM) * n_nb;
    if (a.M / groups >= 128 && big >= (a.offsets ? 1024 : 192)) return f(Big());
    // Too few tiles for the chip: smaller ones, or K shared out among the waves (bf16 rows x MXFP4, us
    // in Small4 / Small2 / Medium: 128 x 4096 x 2048, 128 tiles of 64 x 64, 12 / 16 / 37; 333 x 4100 x
    // 2080, 390 tiles, 34 / 25 / 41; 1000 x 4096 x 2080, 1024 tiles, 61 / 50 / 37 and in Medium2 30).  At
    // K = 2080 one of Small4's four groups is without work, and the halves of the others are 20 and
    // 13 stages.
    const int64_t small = most_tiles<Small4>(a);
    if (small <= 256) return f(Small4());
    if (small <= 768) return f(Small2());
    if (most_tiles<Medium2>(a) <= 256) return f(Medium2());
    return f(Medium());
  }
  return f(nullptr);
}

// The kernel for a product's sizes.
template <int XF, int WF>
int launch_by_size(const ProductArgs& a, hipStream_t s) {
  constexpr int MODE = WF == MC_BF16 ? kBf16 : XF == MC_BF16 ? kA16W4 : kFp4;
  return with_shape(a, [&](auto shape) {
    typedef decltype(shape) S;
    if constexpr (std::is_null_pointer_v<S>) return launch_few<XF, WF>(a, s);
    else return launch_wide<MODE, S>(a, s);
  });
}

}  // namespace mc
