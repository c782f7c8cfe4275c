// MXFP4 encoding on the device: the block exponent and the e2m1 codes, shared by the
// quantiser and by the products that write quantised rows.
#pragma once

#include "mc_common.h"

namespace mc {

// Largest |v| of a block, kept as the bits of |v|: for finite values these order like the
// values, an infinity is above every finite value and a NaN above both.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Block exponent byte from the bits of the block's largest |v|: X - 127 = floor(log2 max) - 2
// (2 = the exponent of e2m1's largest binade), not below -127.  The biased exponent field is
// floor(log2 max) + 127, so X = field - 2; a subnormal or zero maximum has field 0 and takes
// X = 0.  A block that holds an infinity or a NaN takes X = 255, e8m0's NaN.
__device__ __forceinline__ uint32_t block_exponent(uint32_t amax) {
  const uint32_t f = amax >> 23;
  return f == 255u ? 255u : (f > 2u ? f - 2u : 0u);
}

// Codes of 8 values v / 2^(X-127), round to nearest even, magnitudes over 6 to 6, packed with
// the first value in the lowest nibble.  A NaN block's codes are 0.
__device__ __forceinline__ uint32_t fp4x8_codes(const float* v, uint32_t X) {
  const float s = e8m0_to_f32(X == 255u ? 127u : X);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  return X == 255u ? 0u : c;
}

// e8m0 byte -> fp32 scale, 255 -> NaN.
__device__ __forceinline__ float e8m0_or_nan(uint32_t X) {
  return X == 255u ? __uint_as_float(0x7FC00000u) : e8m0_to_f32(X);
}

}  // namespace mc
