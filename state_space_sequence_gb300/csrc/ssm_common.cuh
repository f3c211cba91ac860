// ssm_common.cuh -- device helpers shared by the kernels behind include/ssm.h: the token's step, the
// decays of a pair of states, pieces of activation rows, and sums over the lanes of a warp.
//
// The scan's layout, the same in all its kernels. A warp has 128 / LN channels of one batch entry,
// LN lanes to a channel: a lane has kStates = 4 states of each of kChannels = 4 neighbouring
// channels, sixteen numbers in registers. N <= 4 LN; missing states and channels are zeros. So a
// word of Bm or Cm that a lane reads from shared memory serves four channels, and one of the step
// four states: with one channel and sixteen states to a lane the scan would read twice as much of
// shared memory, whose bandwidth it is near. Steps go in tiles of kT, staged by the warp for itself:
// no warp waits for another.
#pragma once

#include "glr_common.cuh"
#include "ssm.h"

namespace dlr {
namespace ssm {

using glr::add2;
using glr::ex2;
using glr::from_f;
using glr::fma2;
using glr::kLog2e;
using glr::max_nan;
using glr::min_nan;
using glr::mul2;
using glr::rcp;
using glr::to_f;
using glr::two;
using glr::view;
using glr::words;

constexpr int kT = SSM_STATE_STEPS;  // steps of a tile
constexpr int kStates = 4, kChannels = 4;

// softplus(v) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1], and sigmoid(v). log1p(e) =
// 2 atanh(r), r = e / (2 + e) <= 1/3, by its odd series to r^15: the next term is 2e-9 of the
// first. The logarithm of the rounded 1 + e would lose 6e-5 of a step of 0.001. 0 at -inf, inf at
// +inf, a NaN stays one.
__device__ __forceinline__ float softplus(float v, float& sig) {
  const float e = ex2(-kLog2e * fabsf(v));
  const float r = e * rcp(2.0f + e), s = r * r;
  float q = 1.0f / 15.0f;
  q = fmaf(q, s, 1.0f / 13.0f);
  q = fmaf(q, s, 1.0f / 11.0f);
  q = fmaf(q, s, 1.0f / 9.0f);
  q = fmaf(q, s, 1.0f / 7.0f);
  q = fmaf(q, s, 1.0f / 5.0f);
  q = fmaf(q, s, 1.0f / 3.0f);
  q = fmaf(q, s, 1.0f);
  const float w = rcp(1.0f + e);
  sig = v >= 0.0f ? w : e * w;
  return fmaf(2.0f * r, q, max_nan(v, 0.0f));
}

// What a pair of states keeps of `v` over a step whose exponents (in powers of two) are z: v 2^z.
// For 16-bit activations 2^z comes from the special-function unit. For float32 1 - 2^z comes first
// (glr::decay2: its digits hold next to a decay of 1) and v - (1 - 2^z) v keeps them, so that a
// memory of thousands of steps does not add up the rounding of its decay. z is held at +-126.
template <bool PRECISE>
struct decay {
  float2 a;  // the decay, or (PRECISE) one less it, negative
  __device__ __forceinline__ explicit decay(float2 z) {
    if constexpr (PRECISE) {
      z = make_float2(min_nan(z.x, 126.0f), min_nan(z.y, 126.0f));
      float2 rest, unused;
      glr::decay2(z, rest, unused);
      a = mul2(rest, two(-1.0f));
    } else {
      a = make_float2(ex2(min_nan(z.x, 126.0f)), ex2(min_nan(z.y, 126.0f)));
    }
  }
  __device__ __forceinline__ float2 of(float2 v) const {
    if constexpr (PRECISE)
      return fma2(a, v, v);
    else
      return mul2(a, v);
  }
  __device__ __forceinline__ float2 of_plus(float2 v, float2 b) const {
    if constexpr (PRECISE)
      return add2(fma2(a, v, v), b);
    else
      return fma2(a, v, b);
  }
};

// n <= VE neighbouring elements of a row, by one access where `whole` says that there are VE and
// that they stand on a multiple of their size; missing ones are zero.
template <typename T, int VE>
__device__ __forceinline__ void get_piece(words<T, VE>& w, const T* p, int n, bool whole) {
  if (whole) {
    w.get(p);
    return;
  }
  float v[VE];
#pragma unroll
  for (int i = 0; i < VE; ++i) v[i] = i < n ? to_f(p[i]) : 0.0f;
  w.from(v);
}
template <typename T, int VE>
__device__ __forceinline__ void put_piece(T* p, const float* v, int n, bool whole) {
  if (whole) {
    words<T, VE> w;
    w.from(v);
    w.put(p);
    return;
  }
#pragma unroll
  for (int i = 0; i < VE; ++i)
    if (i < n) p[i] = from_f<T>(v[i]);
}

template <int VE>
__device__ __forceinline__ void store_floats(float* p, const float* v) {
  static_assert(VE % 4 == 0, "");
#pragma unroll
  for (int i = 0; i < VE; i += 4)
    *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int VE>
__device__ __forceinline__ void load_floats(float* v, const float* p) {
#pragma unroll
  for (int i = 0; i < VE; i += 4) {
    const float4 t = *reinterpret_cast<const float4*>(p + i);
    v[i] = t.x, v[i + 1] = t.y, v[i + 2] = t.z, v[i + 3] = t.w;
  }
}

// Sums of four values over LANES lanes that stand STRIDE apart; `at` is a lane's place among them.
// Each exchange halves what a lane still has to add, so that four sums over four lanes take three
// exchanges. Afterwards a lane has value at & 3 (LANES >= 4; the same in every fourth lane), values
// 2 at and 2 at + 1 (2 lanes) or all four (1 lane). The order of the additions is fixed.
template <int STRIDE, int LANES>
__device__ __forceinline__ void sum4(float (&v)[4], int at) {
  constexpr uint32_t kAll = 0xffffffffu;
  if constexpr (LANES >= 4) {
    const bool hi = at & 2, odd = at & 1;
    const float s0 = hi ? v[0] : v[2], s1 = hi ? v[1] : v[3];
    const float k0 = hi ? v[2] : v[0], k1 = hi ? v[3] : v[1];
    const float t0 = k0 + __shfl_xor_sync(kAll, s0, 2 * STRIDE);
    const float t1 = k1 + __shfl_xor_sync(kAll, s1, 2 * STRIDE);
    v[0] = (odd ? t1 : t0) + __shfl_xor_sync(kAll, odd ? t0 : t1, STRIDE);
#pragma unroll
    for (int d = 4; d < LANES; d *= 2) v[0] += __shfl_xor_sync(kAll, v[0], d * STRIDE);
  } else if constexpr (LANES == 2) {
    const bool odd = at & 1;
    const float s0 = odd ? v[0] : v[2], s1 = odd ? v[1] : v[3];
    const float k0 = odd ? v[2] : v[0], k1 = odd ? v[3] : v[1];
    v[0] = k0 + __shfl_xor_sync(kAll, s0, STRIDE);
    v[1] = k1 + __shfl_xor_sync(kAll, s1, STRIDE);
  }
}
// Writes them: p is the place of the first of the four, 16-byte aligned.
template <int LANES>
__device__ __forceinline__ void put4(float* p, const float (&v)[4], int at) {
  if constexpr (LANES >= 4) {
    if (at < 4) p[at] = v[0];
  } else if constexpr (LANES == 2) {
    *reinterpret_cast<float2*>(p + 2 * at) = make_float2(v[0], v[1]);
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// How a warp's tile is cut into pieces of VE channels (and VB states) for its lanes.
template <typename T, int LN>
struct shape {
  static constexpr int kCW = 32 / LN * kChannels;  // channels of a warp
  static constexpr int kNP = LN * kStates;         // states of a channel, with the missing ones
  static constexpr int VE = 16 / (int)sizeof(T) < kCW ? 16 / (int)sizeof(T) : kCW;
  static constexpr int VB = 16 / (int)sizeof(T) < kNP ? 16 / (int)sizeof(T) : kNP;
  static constexpr int kRow = kCW / VE, kRowB = kNP / VB;  // pieces of a step
  static constexpr int NV = (kT * kRow + 31) / 32, NB = (kT * kRowB + 31) / 32;
  static_assert(kRow <= 32 && kRowB <= 32 && 32 % kRow == 0 && 32 % kRowB == 0, "");
};

// Where a warp works.
struct place {
  int64_t b;
  int split, group, c0, n_ch;  // c0: first channel; n_ch: channels of the warp that exist (<= kCW)
};

inline int lanes_for(int64_t N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

}  // namespace ssm
}  // namespace dlr
