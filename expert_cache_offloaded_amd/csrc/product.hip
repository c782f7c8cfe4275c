// mc_mxfp4_matmul and mc_grouped_matmul: argument checks and the choice of the operands' formats.
// The kernels are in product_dev.h, compiled for each pair of formats in a file of its own.
#include "product_dev.h"

namespace mc {

int check_product(const char* fn, const ProductArgs& a) {
  MC_REQUIRE((a.x_fmt == MC_BF16 && (a.w_fmt == MC_BF16 || a.w_fmt == MC_MXFP4)) ||
                 (a.x_fmt == MC_MXFP4 && a.w_fmt == MC_MXFP4),
             "%s: no product of x format %d with w format %d", fn, a.x_fmt, a.w_fmt);
  MC_REQUIRE(a.y_fmt == MC_BF16 || a.y_fmt == MC_F32 || a.y_fmt == MC_MXFP4, "%s: unknown y format %d", fn, a.y_fmt);
  MC_REQUIRE(a.M >= 0 && a.N >= 0 && a.K >= 32 && a.K % 32 == 0, "%s: M=%d N=%d K=%d (K must be a positive multiple of 32)",
             fn, a.M, a.N, a.K);
  // tile and byte counts stay within 32 bits
  MC_REQUIRE(a.M <= 0x7FFF0000 && a.N <= 0x7FFF0000 && a.K <= 1 << 28, "%s: M=%d N=%d K=%d too large", fn, a.M, a.N, a.K);
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
  if (a.x_fmt == MC_MXFP4) return launch_product_fp4(a, s);
  if (a.w_fmt == MC_MXFP4) return launch_product_a16w4(a, s);
  return launch_product_bf16(a, s);
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

static ProductArgs grouped_args(const mc_grouped* g) {
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
  return a;
}

extern "C" int mc_grouped_matmul(const mc_grouped* g, hipStream_t s) {
  clear_error();
  MC_REQUIRE(g != nullptr, "mc_grouped_matmul: descriptor is NULL");
  const ProductArgs a = grouped_args(g);
  int rc;
  if ((rc = check_product("mc_grouped_matmul", a)) != MC_OK) return rc;
  MC_REQUIRE(a.offsets || a.M == 0, "mc_grouped_matmul: offsets is NULL");
  // the kernels' sums over groups stay within 32 bits whatever offsets holds: descending ones let groups
  // overlap, each with up to M rows
  MC_REQUIRE((((int64_t)a.M + 15) / 16) * a.E <= 0x7FFFFFFF, "mc_grouped_matmul: M=%d rows of E=%d groups are too many", a.M,
             a.E);
  return launch_product(a, s);
}

extern "C" int mc_grouped_tile(const mc_grouped* g, int32_t* tile) {
  clear_error();
  MC_REQUIRE(g && tile, "mc_grouped_tile: NULL pointer");
  const ProductArgs a = grouped_args(g);
  int rc;
  if ((rc = check_product("mc_grouped_tile", a)) != MC_OK) return rc;
  return with_shape(a, [&](auto shape) {
    typedef decltype(shape) S;
    if constexpr (std::is_null_pointer_v<S>) tile[0] = 16, tile[1] = 0, tile[2] = 1;
    else tile[0] = S::BM, tile[1] = S::BN, tile[2] = S::KG;
    return MC_OK;
  });
}
