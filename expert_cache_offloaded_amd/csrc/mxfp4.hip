// mc_mxfp4_quantize / mc_mxfp4_dequantize: rows to MXFP4 blocks and back.
#include "mxfp4_dev.h"

namespace mc {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

// 8 consecutive elements -> fp32
template <int TYPE>
__device__ __forceinline__ void load8(const uint8_t* p, float* v) {
  if (TYPE == MC_F32) {
    const f32x4_t a = reinterpret_cast<const f32x4_t*>(p)[0], b = reinterpret_cast<const f32x4_t*>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else if (TYPE == MC_BF16) {
    const u32x4_t a = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(a[i]);
      v[2 * i + 1] = bf16_hi(a[i]);
    }
  } else {
    const f16x8_t a = *reinterpret_cast<const f16x8_t*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)a[i];
  }
}

// The values of N codes, N = 8 or, fp32, 4: 16 bytes either way.
template <int TYPE>
__device__ __forceinline__ void store_values(uint8_t* p, uint32_t codes, float s) {
  float v[8];
  const f32x2_t p0 = fp4x2_to_f32x2<0>(codes, s), p1 = fp4x2_to_f32x2<1>(codes, s);
  if (TYPE == MC_F32) {
    *reinterpret_cast<f32x4_t*>(p) = f32x4_t{p0[0], p0[1], p1[0], p1[1]};
    return;
  }
  const f32x2_t p2 = fp4x2_to_f32x2<2>(codes, s), p3 = fp4x2_to_f32x2<3>(codes, s);
  v[0] = p0[0]; v[1] = p0[1]; v[2] = p1[0]; v[3] = p1[1];
  v[4] = p2[0]; v[5] = p2[1]; v[6] = p3[0]; v[7] = p3[1];
  if (TYPE == MC_BF16) {
    u32x4_t o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = (uint32_t)f32_to_bf16_rne(v[2 * i]) | ((uint32_t)f32_to_bf16_rne(v[2 * i + 1]) << 16);
    *reinterpret_cast<u32x4_t*>(p) = o;
  } else {
    f16x8_t o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (_Float16)v[i];
    *reinterpret_cast<f16x8_t*>(p) = o;
  }
}

constexpr int type_bytes(int type) { return type == MC_F32 ? 4 : 2; }

// Rows of c8 chunks that start ld elements apart: the first element of chunk q, for
// q < 2^31 (N elements per chunk).  q / c8 = q m >> s with m = ceil(2^s / c8), 2^s >= 2^31 c8: two
// instructions for the dozens of a 64-bit division.
struct Rows {
  int64_t ld;
  uint64_t m;
  uint32_t c8, s;
  template <int N>
  __device__ __forceinline__ int64_t at(uint32_t q) const {
    const uint32_t r = (uint32_t)((q * m) >> s);
    return r * ld + (int64_t)(q - r * c8) * N;
  }
};

// A lane holds 8 elements, four neighbouring lanes a block of 32 (cols % 32 == 0, so a quad
// never crosses a row).  q counts the 8-element chunks of all rows.
template <int TYPE>
__global__ void __launch_bounds__(256)
quantize_kernel(const uint8_t* __restrict__ src, uint32_t n8, Rows rows, uint8_t* __restrict__ codes,
                uint8_t* __restrict__ scales) {
  for (uint32_t q = blockIdx.x * 256 + threadIdx.x; q < n8; q += gridDim.x * 256) {
    float v[8];
    load8<TYPE>(src + rows.at<8>(q) * type_bytes(TYPE), v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
    const uint32_t X = block_exponent(m);
    reinterpret_cast<uint32_t*>(codes)[q] = fp4x8_codes(v, X);
    if ((threadIdx.x & 3) == 0) scales[q >> 2] = (uint8_t)X;
  }
}

// A lane writes 16 bytes, a wave 1 KiB without gaps (with 8 fp32 values per lane, in two stores 32
// bytes apart, 65536 x 4096 took 340 us, 3.6 TB/s).
constexpr int chunk_values(int type) { return type == MC_F32 ? 4 : 8; }

template <int TYPE>
__global__ void __launch_bounds__(256)
dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, uint32_t n, Rows rows,
                  uint8_t* __restrict__ dst) {
  constexpr int N = chunk_values(TYPE);
  for (uint32_t q = blockIdx.x * 256 + threadIdx.x; q < n; q += gridDim.x * 256) {
    const uint32_t c = N == 8 ? reinterpret_cast<const uint32_t*>(codes)[q] : reinterpret_cast<const uint16_t*>(codes)[q];
    store_values<TYPE>(dst + rows.at<N>(q) * type_bytes(TYPE), c, e8m0_or_nan(scales[q / (32 / N)]));
  }
}

static int check_rows(const char* fn, const void* wide, const char* what, int32_t type, int64_t rows, int64_t cols,
                      int64_t ld, const void* codes, const void* scales) {
  MC_REQUIRE(type == MC_BF16 || type == MC_F16 || type == MC_F32, "%s: %s type %d is not bf16, fp16 or fp32", fn, what,
             type);
  MC_REQUIRE(rows >= 0 && cols >= 0 && cols % 32 == 0, "%s: rows=%lld, cols=%lld (must be a multiple of 32)", fn,
             (long long)rows, (long long)cols);
  MC_REQUIRE(cols <= (int64_t)1 << 32, "%s: cols=%lld is too large", fn, (long long)cols);
  MC_REQUIRE(ld >= cols && ld % 8 == 0, "%s: ld=%lld must be at least cols=%lld and a multiple of 8", fn, (long long)ld,
             (long long)cols);
  MC_REQUIRE(rows == 0 || ld <= ((int64_t)1 << 60) / rows, "%s: rows=%lld x ld=%lld is too large", fn, (long long)rows,
             (long long)ld);
  if (rows == 0 || cols == 0) return MC_OK;
  MC_REQUIRE(wide && codes && scales, "%s: NULL pointer", fn);
  MC_REQUIRE(((uintptr_t)wide | (uintptr_t)codes) % 16 == 0, "%s: %s and codes must be 16-byte aligned", fn, what);
  return MC_OK;
}

// f(first row, chunks, their layout) for parts of whole rows of less than 2^31 chunks of `values`.
template <class F>
static void by_parts(int64_t rows, int64_t cols, int64_t ld, int values, F f) {
  const uint32_t c8 = (uint32_t)(cols / values);
  uint32_t s = 31;
  while (((uint64_t)1 << (s - 31)) < c8) ++s;
  const Rows layout{ld, (((uint64_t)1 << s) + c8 - 1) / c8, c8, s};
  const int64_t most = 0x7FFFFFFF / c8;           // rows of a part (c8 <= 2^30)
  for (int64_t r = 0; r < rows; r += most) f(r, (uint32_t)((rows - r < most ? rows - r : most) * c8), layout);
}

static unsigned chunk_grid(uint32_t n8) {
  const uint32_t g = n8 / 256 + (n8 % 256 != 0);
  return g > 16384 ? 16384 : g;
}

}  // namespace mc

using namespace mc;

extern "C" int mc_mxfp4_quantize(const void* src, int32_t type, int64_t rows, int64_t cols, int64_t ld, void* codes,
                                 void* scales, hipStream_t s) {
  clear_error();
  int rc;
  if ((rc = check_rows("mc_mxfp4_quantize", src, "src", type, rows, cols, ld, codes, scales)) != MC_OK) return rc;
  if (rows == 0 || cols == 0) return MC_OK;
  by_parts(rows, cols, ld, 8, [&](int64_t r, uint32_t n8, const Rows& layout) {
    auto run = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(chunk_grid(n8)), dim3(256), 0, s,
                         static_cast<const uint8_t*>(src) + r * ld * type_bytes(type), n8, layout,
                         static_cast<uint8_t*>(codes) + r * (cols / 2), static_cast<uint8_t*>(scales) + r * (cols / 32));
    };
    if (type == MC_BF16) run(quantize_kernel<MC_BF16>);
    else if (type == MC_F16) run(quantize_kernel<MC_F16>);
    else run(quantize_kernel<MC_F32>);
  });
  MC_LAUNCH_CHECK();
  return MC_OK;
}

extern "C" int mc_mxfp4_dequantize(const void* codes, const void* scales, int64_t rows, int64_t cols, void* dst,
                                   int32_t type, int64_t ld, hipStream_t s) {
  clear_error();
  int rc;
  if ((rc = check_rows("mc_mxfp4_dequantize", dst, "dst", type, rows, cols, ld, codes, scales)) != MC_OK) return rc;
  if (rows == 0 || cols == 0) return MC_OK;
  by_parts(rows, cols, ld, chunk_values(type), [&](int64_t r, uint32_t n8, const Rows& layout) {
    auto run = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(chunk_grid(n8)), dim3(256), 0, s,
                         static_cast<const uint8_t*>(codes) + r * (cols / 2),
                         static_cast<const uint8_t*>(scales) + r * (cols / 32), n8, layout,
                         static_cast<uint8_t*>(dst) + r * ld * type_bytes(type));
    };
    if (type == MC_BF16) run(dequantize_kernel<MC_BF16>);
    else if (type == MC_F16) run(dequantize_kernel<MC_F16>);
    else run(dequantize_kernel<MC_F32>);
  });
  MC_LAUNCH_CHECK();
  return MC_OK;
}
