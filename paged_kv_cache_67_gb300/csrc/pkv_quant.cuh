// pkv_quant.cuh -- the formats of a quantised cache, on the device (see
// pkv.h for their definition).
#pragma once

#include <cuda_fp8.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kInt8 = PKV_QUANT_INT8, kE4m3 = PKV_QUANT_E4M3, kInt4 = PKV_QUANT_INT4;

// Bytes of a row of codes, floats of its parameters.
template <int FMT>
__host__ __device__ constexpr int quant_row_bytes(int D) { return FMT == kInt4 ? D / 2 : D; }
template <int FMT>
__host__ __device__ constexpr int quant_params() { return FMT == kInt4 ? 2 : 1; }
inline size_t quant_codes_bytes(pkv_quant_format fmt, int64_t rows, int D) {
  return (size_t)rows * (fmt == PKV_QUANT_INT4 ? D / 2 : D);
}
inline size_t quant_params_bytes(pkv_quant_format fmt, int64_t rows) {
  return (size_t)rows * (fmt == PKV_QUANT_INT4 ? 8 : 4);
}

// Adding 1.5 * 2^23 in one fused multiply-add rounds the exact product to the
// nearest whole number (halves to even); it is then the sum's low bits.  Good
// for |x * inv| < 2^22.
constexpr float kRintMagic = 12582912.f;
__device__ __forceinline__ int rint_product(float x, float inv) {
  return __float_as_int(fmaf(x, inv, kRintMagic)) - __float_as_int(kRintMagic);
}

// Two e4m3 codes (low, high byte) as halves, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return h;
}
// Two floats as e4m3 codes: `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2_from(float lo, float hi) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}
// (Values in e4m3 that are not numbers, 0x7f and 0xff, come out as NaN.)
__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

}  // namespace pkv
