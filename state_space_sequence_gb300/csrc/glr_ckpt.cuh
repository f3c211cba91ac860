// glr_ckpt.cuh -- the 8-bit checkpoint format of include/glr.h: groups of 32 channels with a
// power-of-two scale, values in e4m3. A power-of-two scale makes both the division by it and the
// product with it exact, so the only rounding is that to e4m3's 3 mantissa bits.
#pragma once

#include <cuda_fp8.h>

#include "glr_common.cuh"

namespace dlr {
namespace glr {

// |t| where t is finite, else 0
__device__ __forceinline__ float finite_abs(float t) {
  const float a = fabsf(t);
  return a <= 3.40282347e38f ? a : 0.0f;
}

// s + 127 for the least s with amax <= 448 * 2^s. amax = m 2^E with 1 <= m < 2 and 448 = 1.75 * 2^8,
// so s = E - 8, or E - 7 where m > 1.75; below -127 it is held there.
__device__ __forceinline__ int scale_byte(float amax) {
  const int bits = __float_as_int(amax);
  const int b = (bits >> 23) - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  return b < 0 ? 0 : b;
}
__device__ __forceinline__ float scale_of(int byte) {  // 2^(byte - 127)
  return __int_as_float(byte ? byte << 23 : 0x400000);
}
__device__ __forceinline__ float inverse_scale_of(int byte) {  // 2^(127 - byte), byte <= 253
  return __int_as_float((254 - byte) << 23);
}

// the code of a value already divided by its scale; infinities become NaN
__device__ __forceinline__ uint32_t encode(float q) {
  const uint32_t c = __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
  return isinf(q) ? 0x7fu : c;
}
__device__ __forceinline__ float decode(uint32_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
}

// Two at a time: the first in the low byte.
__device__ __forceinline__ uint32_t encode2(float2 q) {
  const uint32_t c = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
  return (isinf(q.x) ? 0x7fu : c & 0xffu) | (isinf(q.y) ? 0x7f00u : c & 0xff00u);
}
__device__ __forceinline__ float2 decode2(uint32_t codes) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3)));
}

}  // namespace glr
}  // namespace dlr
