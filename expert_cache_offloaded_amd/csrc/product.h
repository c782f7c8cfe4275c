// Products of rows with expert matrices: the arguments the kernels take, and the launch that
// mc_mxfp4_matmul, mc_grouped_matmul and the prefill layer share.
#pragma once

#include "mc_common.h"

namespace mc {

constexpr int kMaxGroups = 1024;

struct ProductArgs {
  const uint8_t* x;           // rows of x: bf16, or MXFP4 codes
  const uint8_t* xs;          // their scales (MXFP4)
  const uint8_t* w;           // n matrices [N][K]
  const uint8_t* ws;
  uint8_t* y;                 // bf16, fp32 or MXFP4 codes
  uint8_t* ys;
  const int32_t* offsets;     // [E + 1], or null: one group of M rows
  const int32_t* perm;
  const int32_t* entry_of;
  const float* gate;
  int64_t ldx, ldy;           // elements
  int64_t n;
  int32_t x_fmt, w_fmt, y_fmt;
  int32_t swiglu;
  int32_t E, M, N, K;
  int32_t x_rows, x_div, x_perm;
  int32_t y_rows, y_perm;
  int32_t n_gate;
};

// Enqueues the product; the arguments have been checked (check_product).
int launch_product(const ProductArgs& a, hipStream_t s);
// ... of bf16 x bf16, bf16 x MXFP4 and MXFP4 x MXFP4, something to do
int launch_product_bf16(const ProductArgs& a, hipStream_t s);
int launch_product_a16w4(const ProductArgs& a, hipStream_t s);
int launch_product_fp4(const ProductArgs& a, hipStream_t s);
int check_product(const char* fn, const ProductArgs& a);

}  // namespace mc
