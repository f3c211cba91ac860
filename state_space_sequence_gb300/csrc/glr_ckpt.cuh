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

// s + 127 for the least s with amax <= 448 * 2^s. amax = m 2^E with 1 <= m < 2 and 448 = 1.75 *
// 2^8, so s = E - 8, or E - 7 where m > 1.75; below -127 it is held there.
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
  return __half22float2(
      __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3)));
}

// The largest bit pattern of |t| in an item; patterns of floats of one sign are in their order.
template <typename T, int VEC>
__device__ __forceinline__ uint32_t top_bits(const words<T, VEC>& t) {
  if constexpr (sizeof(T) == 4) {
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < VEC; ++v) m = max(m, t.w[v] & 0x7fffffffu);
    return m;
  } else {
    uint32_t m = t.w[0] & 0x7fff7fffu;
#pragma unroll
    for (int v = 1; v < VEC / 2; ++v) m = __vmaxu2(m, t.w[v] & 0x7fff7fffu);
    return max(m & 0xffffu, m >> 16);
  }
}
template <typename T>
__device__ __forceinline__ float from_bits(uint32_t bits) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(bits);
  const uint16_t h = (uint16_t)bits;
  return to_f(*reinterpret_cast<const T*>(&h));
}

// VEC codes and their group's scale. A group is 32 / VEC neighbouring lanes; whole warps call it.
template <typename T, int VEC>
__device__ __forceinline__ void keep(const words<T, VEC>& t, bool on, uint8_t* codes,
                                     uint8_t* scale) {
  uint32_t top = top_bits<T, VEC>(t);
#pragma unroll
  for (int o = 16 / VEC; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  float f[VEC];
  t.to(f);
  float amax = from_bits<T>(top);
  const bool finite = amax <= 3.40282347e38f;
  if (__any_sync(0xffffffffu, !finite)) {  // once more, over what is finite
    amax = 0.0f;
#pragma unroll
    for (int v = 0; v < VEC; ++v) amax = fmaxf(amax, finite_abs(f[v]));
#pragma unroll
    for (int o = 16 / VEC; o >= 1; o >>= 1)
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  }
  if (!on) return;
  const int b = scale_byte(amax);
  const float inv = inverse_scale_of(b);
  if constexpr (VEC == 1) {
    *codes = (uint8_t)encode(f[0] * inv);
  } else {
    uint32_t w[VEC / 4];
#pragma unroll
    for (int v = 0; v < VEC; v += 4) {
      const float2 p = mul2(make_float2(f[v], f[v + 1]), two(inv));
      const float2 q = mul2(make_float2(f[v + 2], f[v + 3]), two(inv));
      if (finite)
        w[v / 4] = (uint32_t)__nv_cvt_float2_to_fp8x2(p, __NV_SATFINITE, __NV_E4M3) |
                   (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3) << 16;
      else
        w[v / 4] = encode2(p) | encode2(q) << 16;
    }
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(codes) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(codes) = w[0];
  }
  if ((threadIdx.x & (32 / VEC - 1)) == 0) *scale = (uint8_t)b;
}
template <int VEC>
__device__ __forceinline__ void kept(const words<uint8_t, VEC>& k, int scale, float* out) {
  const float s = scale_of(scale);
  if constexpr (VEC == 1) {
    out[0] = decode(k.w[0]) * s;
  } else {
#pragma unroll
    for (int v = 0; v < VEC; v += 4) {
      const float2 p = mul2(decode2(k.w[v / 4] & 0xffffu), two(s));
      const float2 q = mul2(decode2(k.w[v / 4] >> 16), two(s));
      out[v] = p.x, out[v + 1] = p.y, out[v + 2] = q.x, out[v + 3] = q.y;
    }
  }
}

}  // namespace glr
}  // namespace dlr
