// moe_experts_prefill_act: the prefill MoE layer as grouped products on MXFP4 or bf16
// activations ([jjl357] "4.1"-"4.3", "6.8").
//
// Steps on the compute stream, fixed grids, no host synchronisation: the token sort; for MXFP4
// activations x quantised once per token; gate_up product of each expert's routes with the
// SwiGLU (and the quantisation of h) in its epilogue, rows in sorted order; down product whose
// epilogue multiplies by the gate and scatters each route to its own row of a [T*k][H] buffer
// (no atomics); the sum of each token's routes in route order, in fp32, rounded once.
//
// The route outputs are fp32, but for act MC_MXFP4, whose caller asked for the shorter buffer: its
// write and read, 805 MB each way at 8192 tokens x 6 routes x 4096 in fp32, are a quarter of the
// layer's traffic (layer 1.40 ms with fp32 outputs, 1.24 with bf16).  Each route is then off by up to
// 2^-8 of itself, which makes the rounding error of y about 1.4 times as large (rms, six routes).
#include "prefill.h"
#include "product.h"

namespace mc {

static size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

struct ActWs {
  SortBuffers sort;
  uint8_t *xq, *xqs;          // MXFP4 x: [T][H/2], [T][H/32]
  uint8_t *h, *hs;            // sorted rows of h: bf16 [T*k][I], or MXFP4 codes and scales
  void* yr;                   // gated route outputs [T*k][H]: fp32, or bf16 (bf16_routes)
};

// The format of an act's activations, and whether its route outputs are bf16.
static int act_fmt(int act) { return act == MC_MXFP4_F32 ? MC_MXFP4 : act; }
static bool bf16_routes(int act) { return act == MC_MXFP4; }

static size_t ws_layout(int T, int k, int E, int H, int I, int act, ActWs* w, uint8_t* base) {
  size_t o = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = base + o;
    o = align256(o + bytes);
    return p;
  };
  const size_t nr = (size_t)T * k;
  ActWs v{};
  v.sort.counts = (int32_t*)take((size_t)E * 4);
  v.sort.counts4 = (int32_t*)take((size_t)E * 16);
  v.sort.offsets = (int32_t*)take((size_t)(E + 1) * 4);
  v.sort.mtile_off = (int32_t*)take((size_t)(E + 1) * 4);
  v.sort.perm = (int32_t*)take(nr * 4);
  if (act_fmt(act) == MC_MXFP4) {
    v.xq = take((size_t)T * H / 2);
    v.xqs = take((size_t)T * H / 32);
    v.h = take(nr * I / 2);
    v.hs = take(nr * I / 32);
  } else {
    v.h = take(nr * I * 2);
  }
  v.yr = take(nr * H * (bf16_routes(act) ? 2 : 4));
  if (w) *w = v;
  return o;
}

// y[t] = bf16 of the sum of token t's valid routes' bf16 rows of yr, in route order; 8 columns per
// thread, up to 8 routes' rows on their way at once.  Bound by yr's bytes.
__global__ void __launch_bounds__(256)
act_combine_kernel(const int32_t* __restrict__ ids, int T, int k, int E, int H, const int32_t* __restrict__ n_tok,
                   const uint16_t* __restrict__ yr, uint16_t* __restrict__ y) {
  const int nt = n_tok ? min(max(*n_tok, 0), T) : T;
  const int h8 = H / 8;
  const int64_t n = (int64_t)T * h8;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int t = (int)(i / h8), c = (int)(i - (int64_t)t * h8) * 8;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (t < nt) {
      for (int j0 = 0; j0 < k; j0 += 8) {
        u32x4_t v[8];
        int id[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // rows of invalid routes lie inside yr too, and are skipped below
          const int64_t r = (int64_t)t * k + min(j0 + j, k - 1);
          id[j] = j0 + j < k ? ids[r] : -1;
          v[j] = *reinterpret_cast<const u32x4_t*>(yr + r * H + c);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (id[j] < 0 || id[j] >= E) continue;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            s[2 * q] += bf16_lo(v[j][q]);
            s[2 * q + 1] += bf16_hi(v[j][q]);
          }
        }
      }
    }
    u32x4_t o;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      o[q] = (uint32_t)f32_to_bf16_rne(s[2 * q]) | ((uint32_t)f32_to_bf16_rne(s[2 * q + 1]) << 16);
    *reinterpret_cast<u32x4_t*>(y + (int64_t)t * H + c) = o;
  }
}

}  // namespace mc

using namespace mc;

extern "C" size_t moe_experts_prefill_act_ws_bytes(int32_t T, int32_t k, int32_t E, int32_t H, int32_t I, int32_t act) {
  if (T < 0 || k < 0 || E < 0 || H < 0 || I < 0 || (act != MC_BF16 && act != MC_MXFP4 && act != MC_MXFP4_F32)) return 0;
  return ws_layout(T, k, E, H, I, act, nullptr, nullptr);
}

static int check_args(const char* fn, const void* x, const int32_t* ids, const float* w, int32_t T, int32_t k, int32_t E,
                      const mc_banks* buf, int32_t act, const void* ws, size_t ws_bytes, const void* y, bool need_n,
                      bool need_y) {
  int rc;
  if ((rc = check_banks(buf, fn)) != MC_OK) return rc;
  MC_REQUIRE(act == MC_BF16 || act == MC_MXFP4 || act == MC_MXFP4_F32, "%s: activations of format %d", fn, act);
  MC_REQUIRE(act == MC_BF16 || buf->fmt == MC_MXFP4, "%s: MXFP4 activations need MXFP4 experts", fn);
  MC_REQUIRE(T >= 0 && k >= 1 && E >= 1 && E <= kP_MaxE && k <= E, "%s: T=%d k=%d E=%d", fn, T, k, E);
  // the products' limits (check_product)
  MC_REQUIRE((int64_t)T * k <= 0x7FFF0000, "%s: T=%d x k=%d routes are too many", fn, T, k);
  MC_REQUIRE(buf->H <= 1 << 28 && buf->I <= 1 << 28, "%s: H=%d I=%d too large", fn, buf->H, buf->I);
  MC_REQUIRE(!need_n || buf->n >= E, "%s: layer buffer holds %lld < E=%d experts", fn, (long long)buf->n, E);
  const size_t need = moe_experts_prefill_act_ws_bytes(T, k, E, buf->H, buf->I, act);
  MC_REQUIRE(T == 0 || ws_bytes >= need, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
  MC_REQUIRE(((uintptr_t)x | (uintptr_t)ws | (uintptr_t)y) % 16 == 0, "%s: x, ws and y must be 16-byte aligned", fn);
  MC_REQUIRE(T == 0 || (x && ids && w && ws && (y || !need_y)), "%s: NULL pointer", fn);
  return MC_OK;
}

// The steps of a layer (MC_PF_*) on one workspace.
static int act_steps(const void* x_bf16, const int32_t* ids, const float* w, int32_t T, int32_t k, const int32_t* n_tok,
                     int32_t E, const mc_banks* buf, const int32_t* entry_of, int32_t act, int32_t steps, void* ws,
                     int32_t* counts, void* y_bf16, hipStream_t s) {
  int rc;
  const int H = buf->H, I = buf->I, fmt = act_fmt(act);
  ActWs v{};
  ws_layout(T, k, E, H, I, act, &v, static_cast<uint8_t*>(ws));
  if (steps & MC_PF_SORT) {
    // the counts go straight to the caller's array, if there is one
    if (counts) v.sort.counts = counts;
    if ((rc = sort_routes_launch(ids, T, k, n_tok, E, v.sort, s)) != MC_OK) return rc;
    if (fmt == MC_MXFP4 && (rc = mc_mxfp4_quantize(x_bf16, MC_BF16, T, H, H, v.xq, v.xqs, s)) != MC_OK) return rc;
  }
  if (steps & MC_PF_EXPERTS) {
    ProductArgs p{};
    p.E = E;
    p.n = buf->n;
    p.M = T * k;
    p.offsets = v.sort.offsets;
    p.perm = v.sort.perm;
    p.entry_of = entry_of;
    p.x_fmt = fmt;
    p.w_fmt = buf->fmt;
    // h = silu(x W_gate^T) * (x W_up^T), rows in sorted order
    p.x = fmt == MC_MXFP4 ? v.xq : static_cast<const uint8_t*>(x_bf16);
    p.xs = v.xqs;
    p.ldx = H;
    p.x_rows = T;
    p.x_div = k;
    p.x_perm = 1;
    p.w = static_cast<const uint8_t*>(buf->gate_up);
    p.ws = static_cast<const uint8_t*>(buf->gate_up_scale);
    p.N = 2 * I;
    p.K = H;
    p.swiglu = 1;
    p.y = v.h;
    p.ys = v.hs;
    p.y_fmt = fmt;
    p.ldy = I;
    p.y_rows = T * k;
    if ((rc = launch_product(p, s)) != MC_OK) return rc;
    // the gated route outputs
    p.x = v.h;
    p.xs = v.hs;
    p.ldx = I;
    p.x_rows = T * k;
    p.x_perm = 0;
    p.w = static_cast<const uint8_t*>(buf->down);
    p.ws = static_cast<const uint8_t*>(buf->down_scale);
    p.N = H;
    p.K = I;
    p.swiglu = 0;
    p.y = static_cast<uint8_t*>(v.yr);
    p.ys = nullptr;
    p.y_fmt = bf16_routes(act) ? MC_BF16 : MC_F32;
    p.ldy = H;
    p.y_perm = 1;
    p.gate = w;
    p.n_gate = T * k;
    if ((rc = launch_product(p, s)) != MC_OK) return rc;
  }
  if (steps & MC_PF_COMBINE) {
    if (!bf16_routes(act))
      return combine_launch(ids, T, k, E, H, n_tok, static_cast<const float*>(v.yr), static_cast<uint16_t*>(y_bf16), s);
    const int64_t blocks = ((int64_t)T * (H / 8) + 255) / 256;
    hipLaunchKernelGGL(act_combine_kernel, dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), 0, s, ids, T, k, E,
                       H, n_tok, static_cast<const uint16_t*>(v.yr), static_cast<uint16_t*>(y_bf16));
    MC_LAUNCH_CHECK();
  }
  return MC_OK;
}

extern "C" int moe_experts_prefill_act(const void* x_bf16, const int32_t* ids, const float* w, int32_t T, int32_t k,
                                       const int32_t* n_tok, int32_t E, const mc_banks* buf, int32_t act, void* ws,
                                       size_t ws_bytes, void* y_bf16, hipStream_t s, const mc_prefetch* next) {
  clear_error();
  const char* fn = "moe_experts_prefill_act";
  int rc;
  if ((rc = check_args(fn, x_bf16, ids, w, T, k, E, buf, act, ws, ws_bytes, y_bf16, true, true)) != MC_OK) return rc;
  if (next && (rc = prefetch_launch(fn, next, E)) != MC_OK) return rc;
  if (T == 0) return MC_OK;
  return act_steps(x_bf16, ids, w, T, k, n_tok, E, buf, nullptr, act, MC_PF_ALL, ws, nullptr, y_bf16, s);
}

extern "C" int moe_experts_prefill_act_part(const void* x_bf16, const int32_t* ids, const float* w, int32_t T, int32_t k,
                                            const int32_t* n_tok, int32_t E, const mc_banks* part_buf,
                                            const int32_t* entry_of, int32_t act, int32_t steps, void* ws,
                                            size_t ws_bytes, int32_t* counts, void* y_bf16, hipStream_t s) {
  clear_error();
  const char* fn = "moe_experts_prefill_act_part";
  int rc;
  MC_REQUIRE(steps != 0 && (steps & ~MC_PF_ALL) == 0, "%s: steps=0x%x", fn, steps);
  if ((rc = check_args(fn, x_bf16, ids, w, T, k, E, part_buf, act, ws, ws_bytes, y_bf16, false,
                       (steps & MC_PF_COMBINE) != 0)) != MC_OK)
    return rc;
  MC_REQUIRE(!(steps & MC_PF_EXPERTS) || entry_of, "%s: the experts step needs entry_of", fn);
  if (T == 0) return MC_OK;
  return act_steps(x_bf16, ids, w, T, k, n_tok, E, part_buf, entry_of, act, steps, ws, counts, y_bf16, s);
}
