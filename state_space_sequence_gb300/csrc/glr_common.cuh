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

// VEC neighbouring elements, read or written at once.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) pack {
  T v[VEC];
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

// a - 1 and a for a = 2^z, z <= 0. With n = rint(z), f = z - n and q = 2^f - 1 (a polynomial with
// q(0) = 0, so its relative error of 2e-8 holds down to z = 0), a - 1 = 2^n q + (2^n - 1). a - 1
// therefore keeps its digits where a is next to 1, and so does 1 - a^2 = -(a - 1)(2 + (a - 1)): with
// a alone its rounding to 2^-24 would be 6e-5 of 1 - a^2 at a memory of 1000 steps. The
// coefficients are a least-maximum fit of (2^f - 1) / f on |f| <= 1/2. Below z = -126 a is held
// at 2^-126.
__device__ __forceinline__ void decay(float z, float& w, float& a) {
  z = max_nan(z, -126.0f);
  const float t = z + 12582912.0f;  // 1.5 * 2^23: n in the low bits
  const float f = z - (t - 12582912.0f);
  const float s = __int_as_float((__float_as_int(t) << 23) + 0x3f800000);  // 2^n
  float q = 0.000154035120f;
  q = fmaf(q, f, 0.00133907355f);
  q = fmaf(q, f, 0.00961823750f);
  q = fmaf(q, f, 0.0555035743f);
  q = fmaf(q, f, 0.240226498f);
  q = fmaf(q, f, 0.693147188f);
  q *= f;
  w = -fmaf(-s, q, 1.0f - s);  // -0 where a = 1
  a = fmaf(s, q, s);
}

// One step's gates. kz = -c softplus(p) log2(e).
struct gate {
  float sr, si;  // sigmoid(r), sigmoid(i)
  float w, a;    // the decay less 1, and the decay
  float m, rm;   // sqrt(1 - a^2) and its reciprocal (a finite number where m is 0)
};
__device__ __forceinline__ gate make_gate(float r, float i, float kz) {
  gate g;
  g.sr = sigmoid(r);
  g.si = sigmoid(i);
  decay(kz * g.sr, g.w, g.a);
  const float v = -g.w * (2.0f + g.w);
  g.rm = rsqrt_approx(max_nan(v, 1e-36f));
  g.m = v * g.rm;
  return g;
}

}  // namespace glr
}  // namespace dlr
