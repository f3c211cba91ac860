// ssm_common.cuh -- device helpers shared by the kernels behind include/ssm.h: the token's step, the
// decays of a pair of states, pieces of activation rows, and sums over the lanes of a warp.
//
// The scan's layout, the same in all its kernels. A unit is 64 / LN channels of one batch entry with
// their N <= 8 LN states (missing states and channels are zeros): 512 numbers. Two warps run it, each
// with one half of the states: LN lanes to a channel, a lane has kStates = 4 states of each of
// kChannels = 2 neighbouring channels, eight numbers in registers, in pairs of neighbouring states. A
// lane reads per step one 16-byte word of Bm and of Cm, which the lanes beside it share, and 8-byte
// words of its channels' steps and inputs. One warp with sixteen numbers a lane reads a third less but
// waits for itself: forwards B4 L4096 H4096 N16 bfloat16 takes 406 to 422 us with it and 423 with two,
// B1 L65536 H256 N64 float32 8% longer, and the gradients have no registers for it.
//
// Helpers stage what a unit reads, a tile of kT steps ahead, and finish what it leaves, a tile behind,
// so that neither the latency of memory nor the elementwise work stands in the recurrence's way.
// A unit's warps meet once a tile.
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
using glr::mul2;
using glr::rcp;
using glr::to_f;
using glr::two;
using glr::view;
using glr::words;

constexpr int kT = SSM_STATE_STEPS;  // steps of a tile
constexpr int kStates = 4, kChannels = 2, kPairs = kStates / 2;  // of a lane
constexpr int kHalves = 2;  // warps that share a unit's states

// log1p(e) for e in [0, 1]: e P(e), P of degree 8 by a fit of the relative error (at most 6.4e-8, 6e-8 low
// where e is small, for P(0) = 1 - 2^-24; 1.7e-7 with its roundings). The logarithm of the rounded 1 + e
// would lose 6e-5 of a step of 0.001, and this needs neither a logarithm nor a reciprocal.
__device__ __forceinline__ float2 log1p2(float2 e) {
  float2 q = two(0.0052326940931379795f);
  q = fma2(q, e, two(-0.029505237936973572f));
  q = fma2(q, e, two(0.07822595536708832f));
  q = fma2(q, e, two(-0.13663245737552643f));
  q = fma2(q, e, two(0.19106006622314453f));
  q = fma2(q, e, two(-0.2484298199415207f));
  q = fma2(q, e, two(0.3331909775733948f));
  q = fma2(q, e, two(-0.4999949336051941f));
  q = fma2(q, e, two(0.9999999403953552f));
  return mul2(q, e);
}
// softplus(v) = max(v, 0) + log1p(e), e = exp(-|v|): 0 at -inf, inf at +inf, a NaN stays one.
__device__ __forceinline__ float2 softplus2(float2 v) {
  const float2 z = mul2(make_float2(fabsf(v.x), fabsf(v.y)), two(-kLog2e));
  return add2(log1p2(make_float2(ex2(z.x), ex2(z.y))),
              make_float2(max_nan(v.x, 0.0f), max_nan(v.y, 0.0f)));
}
// What a pair of states keeps of `v` over a step whose exponents (in powers of two) are rate * s.
// For 16-bit activations the decay comes from the special-function unit, whose results lie 1.9e-8 of
// themselves low on average next to 1 (measured; as cutting off would make them): over a memory of a
// thousand steps that adds up, so the exponent gets kNudge, which is still no step where s is 0.
// For float32 a decay next to 1 goes by the decay less 1: v + (a - 1) v keeps its digits, so that a memory
// of thousands of steps does not add up the rounding of its decay. Below |z| = 1/4 that is z P(z), a
// least-maximum fit of (2^z - 1) / z (2.0e-8); from there on v is multiplied by 2^z itself, which has its
// digits however small it is (a - 1 would round it to a multiple of 2^-24). The choice is made on z + v
// 2^-126, which is z for all but enormous states: those, and infinite ones, of which v + (a - 1) v would
// make a NaN, are multiplied.
constexpr float kNudge = 2.7e-8f;
template <bool PRECISE>
struct decay {
  float2 z, a, less;  // (PRECISE: the exponents,) the decay (and the decay less 1)
  __device__ __forceinline__ decay(float2 rate, float2 s) {
    if constexpr (PRECISE) {
      z = mul2(rate, s);
      float2 p = two(0.0013333556708f);
      p = fma2(p, z, two(0.0096301622689f));
      p = fma2(p, z, two(0.0555041655898f));
      p = fma2(p, z, two(0.2402263134718f));
      p = fma2(p, z, two(0.6931471824646f));
      less = mul2(p, z);
      a = make_float2(ex2(z.x), ex2(z.y));
    } else {
      z = fma2(rate, s, two(kNudge));
      a = make_float2(ex2(z.x), ex2(z.y));
    }
  }
  __device__ __forceinline__ float2 of(float2 v) const {
    if constexpr (PRECISE) {
      const float2 near = fma2(less, v, v), far = mul2(a, v), t = fma2(v, two(0x1p-126f), z);
      return make_float2(fabsf(t.x) < 0.25f ? near.x : far.x, fabsf(t.y) < 0.25f ? near.y : far.y);
    } else {
      return mul2(a, v);
    }
  }
  __device__ __forceinline__ float2 of_plus(float2 v, float2 b, float2 x) const {  // and b x
    if constexpr (PRECISE)
      return fma2(b, x, of(v));
    else
      return fma2(a, v, mul2(b, x));
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
__device__ __forceinline__ void put_piece(T* p, const float (&v)[VE], int n, bool whole) {
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

__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void load4(float (&v)[4], const float* p) {
  const float4 t = *reinterpret_cast<const float4*>(p);
  v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
}

// Sums of COUNT values over LANES lanes that stand STRIDE apart; `at` is a lane's place among them.
// Each exchange halves what a lane still has to add, so that eight sums over eight lanes take seven
// exchanges, and what is left of the lanes is added up whole. The order of the additions is fixed.
template <int STRIDE, int COUNT, int LANES>
__device__ __forceinline__ void sum_lanes(float* v, int at) {
  constexpr uint32_t kAll = 0xffffffffu;
  if constexpr (LANES > 1) {
    if constexpr (COUNT > 1) {
      const bool upper = at & (LANES / 2);
#pragma unroll
      for (int i = 0; i < COUNT / 2; ++i) {
        const float send = upper ? v[i] : v[i + COUNT / 2];
        const float keep = upper ? v[i + COUNT / 2] : v[i];
        v[i] = keep + __shfl_xor_sync(kAll, send, STRIDE * (LANES / 2));
      }
    } else {
      v[0] += __shfl_xor_sync(kAll, v[0], STRIDE * (LANES / 2));
    }
    sum_lanes<STRIDE, (COUNT > 1 ? COUNT / 2 : 1), LANES / 2>(v, at);
  }
}
// Writes them to p[0 .. COUNT), by the lanes that have them.
template <int COUNT, int LANES>
__device__ __forceinline__ void put_lanes(float* p, const float* v, int at) {
  if constexpr (COUNT <= LANES) {
    if (at % (LANES / COUNT) == 0) p[at / (LANES / COUNT)] = v[0];
  } else if constexpr (COUNT == 2 * LANES) {
    *reinterpret_cast<float2*>(p + 2 * at) = make_float2(v[0], v[1]);
  } else {
    static_assert(COUNT % (4 * LANES) == 0, "");
#pragma unroll
    for (int i = 0; i < COUNT / LANES; i += 4)
      *reinterpret_cast<float4*>(p + COUNT / LANES * at + i) =
          make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
}

// The WARPS warps of a unit meet (barriers 1 .. units), and the UNITS finishing warps of a block.
template <int WARPS>
__device__ __forceinline__ void meet_unit(int k) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + k), "n"(32 * WARPS) : "memory");
}
template <int UNITS>
__device__ __forceinline__ void meet_finishing() {
  asm volatile("bar.sync %0, %1;" ::"n"(1 + UNITS), "n"(32 * UNITS) : "memory");
}

// How a unit's tile is cut into pieces of 4 channels (or 4 states) for a warp's lanes: a lane has the
// same channels in all its pieces, and words that lie beside those of its neighbours in shared memory.
constexpr int kPiece = 4;
template <int LN>
struct shape {
  static constexpr int kCW = 32 / LN * kChannels;     // channels of a unit
  static constexpr int kNP = kHalves * LN * kStates;  // states of a channel, with the missing ones
  static constexpr int kRow = kCW / kPiece, kRowB = kNP / kPiece;  // pieces of a step
  static constexpr int NV = kT * kRow / 32, NB = kT * kRowB / 32;  // and of a lane
  static_assert(kT * kRow % 32 == 0 && kT * kRowB % 32 == 0 && 32 % kRow == 0 && 32 % kRowB == 0, "");
};

// Lanes of a channel.
inline int lanes_for(int64_t N) { return N <= 8 ? 1 : N <= 16 ? 2 : N <= 32 ? 4 : 8; }

}  // namespace ssm
}  // namespace dlr
