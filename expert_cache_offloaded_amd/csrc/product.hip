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

// Tile L of the call: row tiles of BM rows group by group, a group's tiles column block by
// column block (consecutive tiles share the weights).  Every wave runs the search by itself:
// lane l looks at group 64 c + l, a prefix sum over the lanes gives each group's first tile.
template <int BM>
__device__ __forceinline__ bool find_tile(const ProductArgs& a, int L, int n_nb, Tile* t) {
  if (!a.offsets) {
    const int m = (a.M + BM - 1) / BM;
    if (L >= m * n_nb) return false;
    t->entry = 0;
    t->nb = L / m;
    t->row0 = (L - t->nb * m) * BM;
    t->nrows = min(BM, a.M - t->row0);
    return true;
  }
  const int lane = threadIdx.x & 63;
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
      const int first = before + __shfl(incl - m, src, 64);
      const int me = __shfl(m, src, 64), lo_e = __shfl(lo, src, 64), rows_e = __shfl(rows, src, 64);
      const int Lp = L - first * n_nb;
      t->nb = Lp / me;
      const int mt = Lp - t->nb * me;
      t->row0 = lo_e + mt * BM;
      t->nrows = min(BM, rows_e - mt * BM);
      t->entry = a.entry_of ? a.entry_of[base + src] : base + src;
      return true;
    }
    before += __shfl(incl, 63, 64);
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

// Output of NF 16-column fragments of one 16-row fragment: fragment f holds columns
// col0 + 16 f + 4 (lane / 16) + i of row i_row (the lane's: lane % 16 of the fragment).
// `on` is false for lanes past the tile's rows (they stay for the lane exchanges).
template <int NF>
__device__ __forceinline__ void store_row(const ProductArgs& a, int i_row, bool on, int col0, int n_out,
                                          const f32x4_t* v) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int r = a.perm ? a.perm[i_row] : i_row;
  const int64_t yr = a.y_perm ? r : i_row;
  on = on && r >= 0 && x_row(a, i_row, r) >= 0 && yr < a.y_rows && (!a.gate || r < a.n_gate);
  const float s = a.gate && on ? a.gate[r] : 1.0f;
  if (a.y_fmt == MC_MXFP4) {
    // two neighbouring fragments are one block of 32 columns: its 8 lane quarters of four
    // columns meet by lane exchanges over lane bits 4 and 5
#pragma unroll
    for (int f = 0; f + 1 < NF; f += 2) {
      float o[8];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i] = s * v[f + i / 4][i % 4];
        m = max(m, abs_bits(o[i]));
      }
      m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
      const uint32_t X = block_exponent(m);
      const uint32_t c = fp4x8_codes(o, X);
      const int col = col0 + 16 * f;
      if (on && col < n_out) {
        uint8_t* p = a.y + yr * (int64_t)(n_out / 2) + (col >> 1) + 2 * g;
        *reinterpret_cast<uint16_t*>(p) = (uint16_t)c;
        *reinterpret_cast<uint16_t*>(p + 8) = (uint16_t)(c >> 16);
        if (g == 0) a.ys[yr * (int64_t)(n_out / 32) + (col >> 5)] = (uint8_t)X;
      }
    }
  } else if (on) {
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int col = col0 + 16 * f + 4 * g;
      if (col < n_out) store4(a, yr, col, n_out, a.gate ? s * v[f] : v[f]);
    }
  }
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

// ---------------------------------------------------------------- the kernel
//
// 64 rows x 64 weight rows (SwiGLU: 32 gate and the matching 32 up rows) per workgroup of 4
// waves; a wave multiplies 16 rows with all 64 weight rows, operands straight from memory.

constexpr int kBM = 64, kBN = 64;

template <int XF, int WF>
__global__ void __launch_bounds__(256)
product_kernel(ProductArgs a, int n_nb) {
  Tile t;
  if (!find_tile<kBM>(a, blockIdx.x, n_nb, &t)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  if (wave * 16 >= t.nrows) return;
  const int n_out = a.swiglu ? a.N / 2 : a.N;
  const int cols = a.swiglu ? kBN / 2 : kBN;        // output columns of a tile
  const int c0 = t.nb * cols;
  const int64_t K = a.K;
  const int64_t wrow_b = WF == MC_BF16 ? 2 * K : K / 2, xrow_b = XF == MC_BF16 ? 2 * a.ldx : K / 2;
  const uint8_t* wp[4];
  const uint8_t* wsp[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    int row = a.swiglu ? c0 + (f & 1) * 16 + l16 : c0 + f * 16 + l16;
    row = min(row, n_out - 1) + (a.swiglu && f >= 2 ? n_out : 0);
    const int64_t wr = (int64_t)t.entry * a.N + row;
    wp[f] = a.w + wr * wrow_b;
    wsp[f] = a.ws + wr * (K / 32);
  }
  const int m = wave * 16 + l16;
  const int i_row = t.row0 + min(m, t.nrows - 1);
  const int64_t xr = max(x_row(a, i_row, a.perm ? a.perm[i_row] : i_row), 0);
  const uint8_t* xp = a.x + xr * xrow_b;
  const uint8_t* xsp = a.xs + xr * (K / 32);

  f32x4_t acc[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (WF == MC_BF16) {
    for (int64_t k = 0; k < 2 * K; k += 64) {
      const u32x4_t x = *reinterpret_cast<const u32x4_t*>(xp + k + 16 * g);
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[f] = mfma_bf16(*reinterpret_cast<const u32x4_t*>(wp[f] + k + 16 * g), x, acc[f]);
    }
  } else {
    const int nblk = a.K / 32;
    for (int b0 = 0; b0 < nblk; b0 += 4) {
      const int b = b0 + g;
      const bool in = b < nblk;                     // blocks past K count as zeros
      u32x4_t w[4];
      uint32_t sw[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        w[f] = in ? *reinterpret_cast<const u32x4_t*>(wp[f] + (int64_t)b * 16) : u32x4_t{0, 0, 0, 0};
        sw[f] = in ? wsp[f][b] : 127u;
      }
      if (XF == MC_MXFP4) {
        const u32x4_t x = in ? *reinterpret_cast<const u32x4_t*>(xp + (int64_t)b * 16) : u32x4_t{0, 0, 0, 0};
        const uint32_t sx = in ? xsp[b] : 127u;
#pragma unroll
        for (int f = 0; f < 4; ++f) acc[f] = mfma_fp4(w[f], sw[f], x, sx, acc[f]);
      } else {
        // the K order of the four products is permuted: lane group g holds block b0 + g
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4_t x = in ? *reinterpret_cast<const u32x4_t*>(xp + (int64_t)b * 64 + 16 * j) : u32x4_t{0, 0, 0, 0};
#pragma unroll
          for (int f = 0; f < 4; ++f)
            acc[f] = mfma_bf16(__builtin_bit_cast(u32x4_t, fp4x8_bf16(w[f][j], e8m0_or_nan(sw[f]))), x, acc[f]);
        }
      }
    }
  }
  if (a.swiglu) {
    f32x4_t h[2];
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) h[f][i] = silu(acc[f][i]) * acc[f + 2][i];
    store_row<2>(a, i_row, m < t.nrows, c0, n_out, h);
  } else {
    store_row<4>(a, i_row, m < t.nrows, c0, n_out, acc);
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

int launch_product(const ProductArgs& a, hipStream_t s) {
  if (a.M == 0 || a.N == 0 || a.x_rows == 0 || a.y_rows == 0 || a.n == 0) return MC_OK;
  const int64_t n_out = a.swiglu ? a.N / 2 : a.N, cols = a.swiglu ? kBN / 2 : kBN;
  const int64_t n_nb = (n_out + cols - 1) / cols;
  // sum over groups of ceil(rows / BM)
  const int64_t mt = a.M / kBM + (a.offsets ? (a.E < a.M ? a.E : a.M) : 1);
  MC_REQUIRE(mt * n_nb <= 0x7FFFFFFF, "product of %d rows with %d columns is too large", a.M, a.N);
  const dim3 grid((unsigned)(mt * n_nb)), block(256);
  if (a.x_fmt == MC_MXFP4) hipLaunchKernelGGL((product_kernel<MC_MXFP4, MC_MXFP4>), grid, block, 0, s, a, (int)n_nb);
  else if (a.w_fmt == MC_MXFP4) hipLaunchKernelGGL((product_kernel<MC_BF16, MC_MXFP4>), grid, block, 0, s, a, (int)n_nb);
  else hipLaunchKernelGGL((product_kernel<MC_BF16, MC_BF16>), grid, block, 0, s, a, (int)n_nb);
  MC_LAUNCH_CHECK();
  return MC_OK;
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
