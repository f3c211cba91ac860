// glr_common.cuh -- device helpers shared by the kernels behind include/glr.h: element types,
// the gates of the gated linear recurrence, and the sums of a block.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dlr_common.cuh"
#include "glr.h"

namespace dlr {
namespace glr {

template <typename T>
constexpr bool is_half = false;
template <>
inline constexpr bool is_half<__half> = true;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// Two 16-bit values of a word as floats and back, the first in the low half.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (sizeof(T) == 2 && !is_half<T>)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float2 v) {
  if constexpr (is_half<T>) {
    const __half2 p = __float22half2_rn(v);
    return *reinterpret_cast<const uint32_t*>(&p);
  } else {
    const __nv_bfloat162 p = __float22bfloat162_rn(v);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
}
// An item of memory by one access of its size, in words.
template <typename T, int VEC>
struct words {
  static constexpr int kBytes = VEC * (int)sizeof(T), kWords = (kBytes + 3) / 4;
  uint32_t w[kWords] = {};
  __device__ __forceinline__ void get(const void* p) {
    if constexpr (kBytes == 16) {
      const uint4 t = *static_cast<const uint4*>(p);
      w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
    } else if constexpr (kBytes == 8) {
      const uint2 t = *static_cast<const uint2*>(p);
      w[0] = t.x, w[1] = t.y;
    } else if constexpr (kBytes == 4) {
      w[0] = *static_cast<const uint32_t*>(p);
    } else if constexpr (kBytes == 2) {
      w[0] = *static_cast<const uint16_t*>(p);
    } else {
      w[0] = *static_cast<const uint8_t*>(p);
    }
  }
  __device__ __forceinline__ void put(void* p) const {
    if constexpr (kBytes == 16)
      *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (kBytes == 8)
      *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (kBytes == 4)
      *static_cast<uint32_t*>(p) = w[0];
    else if constexpr (kBytes == 2)
      *static_cast<uint16_t*>(p) = (uint16_t)w[0];
    else
      *static_cast<uint8_t*>(p) = (uint8_t)w[0];
  }
  __device__ __forceinline__ void to(float* out) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) out[v] = __uint_as_float(w[v]);
    } else if constexpr (VEC == 1) {
      out[0] = unpack2<T>(w[0]).x;
    } else {
#pragma unroll
      for (int v = 0; v < VEC; v += 2) {
        const float2 t = unpack2<T>(w[v / 2]);
        out[v] = t.x, out[v + 1] = t.y;
      }
    }
  }
  __device__ __forceinline__ void from(const float* in) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) w[v] = __float_as_uint(in[v]);
    } else if constexpr (VEC == 1) {
      w[0] = pack2<T>(make_float2(in[0], 0.0f));
    } else {
#pragma unroll
      for (int v = 0; v < VEC; v += 2) w[v / 2] = pack2<T>(make_float2(in[v], in[v + 1]));
    }
  }
};

// An array [B, L, H] with contiguous channels (strides in elements).
template <typename T>
struct view {
  T* p;
  int64_t sb, st;
  __device__ __forceinline__ T* row(int64_t b, int64_t t) const { return p + b * sb + t * st; }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN stays a NaN
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

constexpr float kLog2e = 1.44269504f;

// 1 / (1 + e^-v): 1 at +inf, 0 at -inf (the reciprocal of an overflowed sum)
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.0f + ex2(-kLog2e * v)); }

// softplus(v) = log(1 + e^v); above 20 it is v to float precision
__device__ __forceinline__ float softplus(float v) { return v > 20.0f ? v : log1pf(expf(v)); }

// Two elements at a time: one instruction works on both halves.
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

__device__ __forceinline__ float2 sigmoid2(float2 v) {
  const float2 t = mul2(v, two(-kLog2e));
  const float2 d = add2(make_float2(ex2(t.x), ex2(t.y)), two(1.0f));
  return make_float2(rcp(d.x), rcp(d.y));
}

// 1 - a and a for a = 2^z, z <= 0. With n = rint(z), f = z - n and q = 1 - 2^f (a polynomial with
// q(0) = 0, so its relative error of 2e-8 holds down to z = 0), 1 - a = 2^n q + (1 - 2^n). 1 - a
// therefore keeps its digits where a is next to 1, and so does 1 - a^2 = (1 - a)(1 + a): from a
// alone its rounding to 2^-24 would be 6e-5 of 1 - a^2 at a memory of 1000 steps. The coefficients
// are a least-maximum fit of (1 - 2^f) / f on |f| <= 1/2. Below z = -126 a is held at 2^-126.
__device__ __forceinline__ void decay2(float2 z, float2& rest, float2& a) {
  z = make_float2(max_nan(z.x, -126.0f), max_nan(z.y, -126.0f));
  const float2 t = add2(z, two(12582912.0f));  // 1.5 * 2^23: n in the low bits
  const float2 f = fma2(add2(t, two(-12582912.0f)), two(-1.0f), z);
  const float2 s = make_float2(__int_as_float((__float_as_int(t.x) << 23) + 0x3f800000),
                               __int_as_float((__float_as_int(t.y) << 23) + 0x3f800000));  // 2^n
  float2 q = two(-0.000154035120f);
  q = fma2(q, f, two(-0.00133907355f));
  q = fma2(q, f, two(-0.00961823750f));
  q = fma2(q, f, two(-0.0555035743f));
  q = fma2(q, f, two(-0.240226498f));
  q = fma2(q, f, two(-0.693147188f));
  q = mul2(q, f);
  rest = fma2(s, q, fma2(s, two(-1.0f), two(1.0f)));
  a = mul2(s, fma2(q, two(-1.0f), two(1.0f)));
}

// 1 / sqrt(u), a finite number where u is 0
__device__ __forceinline__ float2 rsqrt2(float2 u) {
  return make_float2(rsqrt_approx(max_nan(u.x, 1e-36f)), rsqrt_approx(max_nan(u.y, 1e-36f)));
}
__device__ __forceinline__ float min_nan(float a, float b) {  // a NaN stays a NaN
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Two elements' decays and inputs: a, and b = sqrt(1 - a^2) sigmoid(i) x. kz = -c softplus(p)
// log2(e). With u = 1 - a^2 and E = e^i, b = x E u / sqrt(u (1 + E)^2), which takes one special
// function less than sqrt(u) and 1 / (1 + E) by themselves. E is held at 2^40, where the gate is 1
// to float precision, so that the square stays finite; a gate that shuts keeps its value while
// sqrt(u) E is a normal float, and is 0 at i = -inf.
__device__ __forceinline__ void gates2(float2 r, float2 i, float2 x, float2 kz, float2& a,
                                       float2& b) {
  float2 rest;
  decay2(mul2(kz, sigmoid2(r)), rest, a);
  const float2 u = mul2(rest, add2(a, two(1.0f)));
  const float2 t = mul2(i, two(kLog2e));
  const float2 e = make_float2(min_nan(ex2(t.x), 0x1p40f), min_nan(ex2(t.y), 0x1p40f));
  const float2 d = add2(e, two(1.0f));
  b = mul2(mul2(mul2(u, rsqrt2(mul2(mul2(u, d), d))), e), x);
}

}  // namespace glr
}  // namespace dlr
