// ssm_scan.cuh -- what the selective scan's two directions share: their parameters, the cut of a
// sequence into splits, and the joining of the splits' maps.
#pragma once

#include <algorithm>

#include "ssm_common.cuh"

namespace dlr {
namespace ssm {

constexpr int kSiteFileScan = 27;  // bounds-checked build: this header's site number

template <typename T>
struct inputs {
  int64_t B, L;
  int H, Hg, N, G;  // Hg = H / G channels of a group
  int softplus;
  int blocks;       // blocks of channels of a group
  int tiles, per_split, splits;
  view<const T> x, dt, z, Bm, Cm;
  const float *A, *D, *bias, *h0;
  const uint8_t* reset;
  // the splits' maps: what a split adds to the state that enters it, [B, splits, H, N], and the sum
  // of its steps, [B, splits, H], a NaN where a mark stops all
  float *ends, *sums;
};

// The bits of a tile's marked steps (bit t: step t0 + t), the same in all lanes.
__device__ __forceinline__ uint32_t marks(const uint8_t* reset, int64_t row, int64_t t0, int64_t L,
                                          int lane) {
  if (!reset) return 0;
  const bool hit = lane < kT && t0 + lane < L && reset[row * L + t0 + lane] != 0;
  return __ballot_sync(0xffffffffu, hit);
}

// The rates of a lane's states times log2(e), in pairs of neighbouring states; zero for states and
// channels that do not exist.
__device__ __forceinline__ void load_rates(float2 (&a)[kChannels][kPairs], const float* A, int N,
                                           int64_t c, int n_ch, int n0) {
#pragma unroll
  for (int i = 0; i < kChannels; ++i)
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      const int n = n0 + 2 * p;
      const float* q = A + (c + i) * N + n;
      a[i][p] = make_float2(i < n_ch && n < N ? q[0] * kLog2e : 0.0f,
                            i < n_ch && n + 1 < N ? q[1] * kLog2e : 0.0f);
    }
}
__device__ __forceinline__ void clear(float2 (&h)[kChannels][kPairs]) {
#pragma unroll
  for (int i = 0; i < kChannels; ++i)
#pragma unroll
    for (int p = 0; p < kPairs; ++p) h[i][p] = two(0.0f);
}
// A lane's states from an array [.., H, N] whose row of the lane's first channel begins at p, and
// back.
__device__ __forceinline__ float4 get_quad(const float* p, int n, int N, bool whole) {
  float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (n >= N) return t;
  if (whole && DLR_IN_FILE(n + 3, N, kSiteFileScan)) return *reinterpret_cast<const float4*>(p + n);
  t.x = p[n];
  if (n + 1 < N) t.y = p[n + 1];
  if (n + 2 < N) t.z = p[n + 2];
  if (n + 3 < N) t.w = p[n + 3];
  return t;
}
__device__ __forceinline__ bool quads(const float* p, int N) {
  return (N & 3) == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}
__device__ __forceinline__ void load_states(float2 (&h)[kChannels][kPairs], const float* p, int N,
                                            int n_ch, int n0) {
  const bool whole = quads(p, N);
#pragma unroll
  for (int i = 0; i < kChannels; ++i) {
    const float4 t = i < n_ch ? get_quad(p + (int64_t)i * N, n0, N, whole)
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    h[i][0] = make_float2(t.x, t.y);
    h[i][1] = make_float2(t.z, t.w);
  }
}
__device__ __forceinline__ void store_states(float* p, const float2 (&h)[kChannels][kPairs], int N,
                                             int n_ch, int n0) {
  const bool whole = quads(p, N);
#pragma unroll
  for (int i = 0; i < kChannels; ++i) {
    if (i >= n_ch || n0 >= N) continue;
    float* q = p + (int64_t)i * N + n0;
    if (whole && DLR_IN_FILE(n0 + 3, N, kSiteFileScan)) {
      *reinterpret_cast<float4*>(q) = make_float4(h[i][0].x, h[i][0].y, h[i][1].x, h[i][1].y);
    } else {
      q[0] = h[i][0].x;
      if (n0 + 1 < N) q[1] = h[i][0].y;
      if (n0 + 2 < N) q[2] = h[i][1].x;
      if (n0 + 3 < N) q[3] = h[i][1].y;
    }
  }
}
// A lane's words of a step: its states' (of Bm or Cm), and its channels'.
__device__ __forceinline__ void get_map(float2 (&v)[kPairs], const float* p) {
  const float4 t = *reinterpret_cast<const float4*>(p);
  v[0] = make_float2(t.x, t.y);
  v[1] = make_float2(t.z, t.w);
}
__device__ __forceinline__ void get_channels(float (&v)[kChannels], const float* p) {
  const float2 t = *reinterpret_cast<const float2*>(p);
  v[0] = t.x, v[1] = t.y;
}

// 2^z v + e, over a split. Over many steps 2^z may underflow or overflow where no step's does: an infinite v
// then still passes, and zero stays zero.
__device__ __forceinline__ float pass(float z, float v, float e) {
  const float a = ex2(z), r = fmaf(a, v, e);
  if (r == r) return r;
  const bool all = (a == 0.0f && fabsf(v) == INFINITY && z > -INFINITY) || (a == INFINITY && v == 0.0f);
  return all ? v + e : r;
}

// A split of a sequence takes the state that enters it to P h + e: e is its end from zero, and P =
// exp(A sum of its steps). What enters a split, from what enters the sequence (`h`): forwards through
// the splits before it, backwards (the gradients) through those behind it, the same for every split in
// the same order. One split, the common case, has no maps.
template <bool BACK, typename T>
__device__ __forceinline__ void enter(float2 (&h)[kChannels][kPairs], const inputs<T>& in, int64_t b,
                                      int split, int64_t c, int n_ch, int n0,
                                      const float2 (&rate)[kChannels][kPairs]) {
  const int64_t HN = (int64_t)in.H * in.N;
  const int count = BACK ? in.splits - 1 - split : split;
#pragma unroll 4
  for (int j = 0; j < count; ++j) {
    const int64_t row = b * in.splits + (BACK ? in.splits - 1 - j : j);
    float2 e[kChannels][kPairs];
    load_states(e, in.ends + row * HN + c * in.N, in.N, n_ch, n0);
#pragma unroll
    for (int i = 0; i < kChannels; ++i) {
      if (i >= n_ch) continue;
      const float s = DLR_IN_FILE(row, in.B * in.splits, kSiteFileScan) &&
                              DLR_IN_FILE(c + i, in.H, kSiteFileScan)
                          ? in.sums[row * in.H + c + i]
                          : 0.0f;
#pragma unroll
      for (int p = 0; p < kPairs; ++p) {
        const float2 z = mul2(rate[i][p], two(s));
        h[i][p] = s != s ? e[i][p]
                         : make_float2(pass(z.x, h[i][p].x, e[i][p].x), pass(z.y, h[i][p].y, e[i][p].y));
      }
    }
  }
}

// Where a unit works, and how its rows lie.
template <typename T, int LN>
struct unit {
  using S = shape<LN>;
  using piece = words<T, kPiece>;
  int64_t b;
  int split, group, c0, n_ch;  // c0: first channel; n_ch: how many of the unit's exist
  bool whole, whole_b;         // pieces of rows go by whole accesses

  // units of a batch entry and split: `blocks` of each group
  __device__ __forceinline__ bool find(const inputs<T>& in, int64_t id, int n_split) {
    const int per_row = in.blocks * in.G;
    if (id >= (int64_t)per_row * n_split * in.B) return false;
    const int cb = (int)(id % per_row);
    split = (int)(id / per_row % n_split);
    b = id / per_row / n_split;
    place(in, cb / in.blocks, cb % in.blocks * S::kCW);
    return true;
  }
  __device__ __forceinline__ void place(const inputs<T>& in, int g, int first) {
    group = g;
    c0 = g * in.Hg + first;
    n_ch = max(0, min(S::kCW, in.Hg - first));
    whole = n_ch == S::kCW && pieces(in.x) && pieces(in.dt);
    whole_b = in.N % kPiece == 0 && maps(in.Bm, in.N) && maps(in.Cm, in.N);
  }
  template <typename V>
  __device__ __forceinline__ bool pieces(const view<V>& v) const {
    return !v.p || ((reinterpret_cast<uintptr_t>(v.p + c0) | (uintptr_t)(v.sb * (int64_t)sizeof(T)) |
                     (uintptr_t)(v.st * (int64_t)sizeof(T))) &
                    (uintptr_t)(kPiece * sizeof(T) - 1)) == 0;
  }
  __device__ __forceinline__ bool maps(const view<const T>& v, int N) const {
    return ((reinterpret_cast<uintptr_t>(v.p + (int64_t)group * N) |
             (uintptr_t)(v.sb * (int64_t)sizeof(T)) | (uintptr_t)(v.st * (int64_t)sizeof(T))) &
            (uintptr_t)(kPiece * sizeof(T) - 1)) == 0;
  }
  // a lane's channels of the unit, and the step of its piece k
  static __device__ __forceinline__ int channel(int lane) { return lane % S::kRow * kPiece; }
  static __device__ __forceinline__ int step(int k, int lane) {
    return lane / S::kRow + k * (32 / S::kRow);
  }
  static __device__ __forceinline__ int state(int lane) { return lane % S::kRowB * kPiece; }
  static __device__ __forceinline__ int step_b(int k, int lane) {
    return lane / S::kRowB + k * (32 / S::kRowB);
  }
  // A tile's pieces of a row, zeros where the row or the sequence ends: COUNT of them, every STRIDE
  // one from `from` on.
  template <int COUNT, int STRIDE, typename V>
  __device__ __forceinline__ void fetch(piece (&w)[COUNT], const view<V>& v, int64_t t0, int64_t L,
                                        int lane, bool ok, int from = 0) const {
    const int c = channel(lane);
    const V* p = v.p + (b * v.sb + (t0 + step(from, lane)) * v.st + c0 + c);
    if (ok && t0 + kT <= L) {
#pragma unroll
      for (int k = 0; k < COUNT; ++k)
        if (DLR_IN_FILE(t0 + step(from + k * STRIDE, lane), L, kSiteFileScan) &&
            DLR_IN_FILE(c + kPiece - 1, n_ch, kSiteFileScan))
          w[k].get(p + k * STRIDE * (32 / S::kRow) * v.st);
    } else {
#pragma unroll
      for (int k = 0; k < COUNT; ++k) {
        w[k] = piece();
        if (t0 + step(from + k * STRIDE, lane) < L && c < n_ch)
          get_piece<T, kPiece>(w[k], p + k * STRIDE * (32 / S::kRow) * v.st, n_ch - c, ok);
      }
    }
  }
  template <typename V>
  __device__ __forceinline__ void fetch(piece (&w)[S::NV], const view<V>& v, int64_t t0, int64_t L,
                                        int lane, bool ok) const {
    fetch<S::NV, 1>(w, v, t0, L, lane, ok);
  }
  __device__ __forceinline__ void fetch_b(piece (&w)[S::NB], const view<const T>& v, int64_t t0,
                                          int64_t L, int N, int lane) const {
    const int n = state(lane);
    const T* p = v.p + (b * v.sb + (t0 + step_b(0, lane)) * v.st + (int64_t)group * N + n);
    if (whole_b && N == S::kNP && t0 + kT <= L) {
#pragma unroll
      for (int k = 0; k < S::NB; ++k)
        if (DLR_IN_FILE(t0 + step_b(k, lane), L, kSiteFileScan) &&
            DLR_IN_FILE(n + kPiece - 1, N, kSiteFileScan))
          w[k].get(p + k * (32 / S::kRowB) * v.st);
    } else {
#pragma unroll
      for (int k = 0; k < S::NB; ++k) {
        w[k] = piece();
        if (t0 + step_b(k, lane) < L && n < N)
          get_piece<T, kPiece>(w[k], p + k * (32 / S::kRowB) * v.st, N - n, whole_b);
      }
    }
  }
  static __device__ __forceinline__ void put_b(float (*m)[S::kNP], const piece (&w)[S::NB],
                                               int lane) {
#pragma unroll
    for (int k = 0; k < S::NB; ++k) {
      float v[kPiece];
      w[k].to(v);
      store4(&m[step_b(k, lane)][state(lane)], v);
    }
  }
};

// The steps s and the inputs s x of a tile's pieces (`bias`: of this lane's channels): softplus, and
// zeros where there is no channel or step (which leave the state as it is).
template <int COUNT, int STRIDE, typename T, int LN>
__device__ __forceinline__ void stage_steps(const unit<T, LN>& u, int softplus, int64_t t0, int64_t L,
                                            int lane, const float (&bias)[kPiece],
                                            const words<T, kPiece> (&wx)[COUNT],
                                            const words<T, kPiece> (&wd)[COUNT],
                                            float (*s)[shape<LN>::kCW], float (*in)[shape<LN>::kCW],
                                            int from = 0) {
  using S = shape<LN>;
  const int c = u.channel(lane);
  const bool all = u.n_ch == S::kCW && t0 + kT <= L;
#pragma unroll
  for (int k = 0; k < COUNT; ++k) {
    const int t = u.step(from + k * STRIDE, lane);
    float xv[kPiece], dv[kPiece];
    wx[k].to(xv);
    wd[k].to(dv);
#pragma unroll
    for (int i = 0; i < kPiece; i += 2) {
      float2 d = add2(make_float2(dv[i], dv[i + 1]), make_float2(bias[i], bias[i + 1]));
      if (softplus) d = softplus2(d);
      dv[i] = d.x, dv[i + 1] = d.y;
    }
    if (!all) {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const bool there = t0 + t < L && c + i < u.n_ch;
        dv[i] = there ? dv[i] : 0.0f;
        xv[i] = there ? xv[i] : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < kPiece; i += 2) {
      const float2 p = mul2(make_float2(xv[i], xv[i + 1]), make_float2(dv[i], dv[i + 1]));
      xv[i] = p.x, xv[i + 1] = p.y;
    }
    store4(&s[t][c], dv);
    store4(&in[t][c], xv);
  }
}
// A lane's channels of a parameter (zeros for none).
template <typename T, int LN>
__device__ __forceinline__ void load_channels(float (&v)[kPiece], const float* p,
                                              const unit<T, LN>& u, int lane) {
  const int c = u.channel(lane);
#pragma unroll
  for (int i = 0; i < kPiece; ++i) v[i] = p && c + i < u.n_ch ? p[u.c0 + c + i] : 0.0f;
}

// How many splits a sequence is cut into. A unit goes through its rows step by step, so few channels
// leave the GPU idle; rows are then cut, and the states at the cuts come from a pass over the steps
// alone, which takes `maps` of the time of the pass itself and, to be launched, that of two tiles. A
// split takes two tiles more, to fill and to drain. Blocks have `per_block` units, an SM has four:
// with one, two and three of them a tile takes 0.58, 0.64 and 0.84 of its time with four (measured forwards
// at N = 16 in 16 bits, and taken for all types, numbers of states and directions).
inline int splits_for(int64_t B, int64_t L, int64_t H, int64_t G, int lanes, int per_block,
                      double maps) {
  constexpr int64_t kSMs = 152, kUnits = 4;
  constexpr double kTime[kUnits + 1] = {0.0, 0.58, 0.64, 0.84, 1.0};
  const int64_t cw = 64 / lanes, units = (H / G + cw - 1) / cw, tiles = (L + kT - 1) / kT;
  const int64_t blocks = B * G * ((units + per_block - 1) / per_block);
  int best = 1;
  double least = 0.0;
  for (int s = 1; s <= std::min<int64_t>(64, tiles); ++s) {
    const int64_t all = (blocks * s + kSMs - 1) / kSMs * per_block;  // units that an SM goes through
    const double cost = (double(all / kUnits) + kTime[all % kUnits]) * ((tiles + s - 1) / s + 2) *
                            (s == 1 ? 1.0 : 1.0 + maps) + (s == 1 ? 0.0 : 2.0);
    if (s == 1 || cost < least) best = s, least = cost;
  }
  return best;
}

template <typename T, typename ARGS>
inputs<T> make_inputs(const ARGS& a, int want) {
  inputs<T> q{};
  q.B = a.B, q.L = a.L, q.H = (int)a.H, q.N = (int)a.N, q.G = (int)a.G;
  q.Hg = q.H / q.G;
  q.softplus = (int)a.softplus;
  auto in = [](const glr_view& v) {
    return view<const T>{static_cast<const T*>(v.data), v.stride_b, v.stride_t};
  };
  q.x = in(a.x), q.dt = in(a.dt), q.z = in(a.z), q.Bm = in(a.Bm), q.Cm = in(a.Cm);
  q.A = a.A, q.D = a.D, q.bias = a.dt_bias, q.h0 = a.h0, q.reset = a.reset;
  q.tiles = (int)((a.L + kT - 1) / kT);
  q.per_split = (q.tiles + want - 1) / want;
  q.splits = (q.tiles + q.per_split - 1) / q.per_split;  // each has at least one tile
  return q;
}
template <typename T>
view<T> out_view(const glr_out& v) {
  return view<T>{static_cast<T*>(v.data), v.stride_b, v.stride_t};
}
// Floats of the maps of `splits` splits.
inline int64_t map_floats(int64_t B, int64_t H, int64_t N, int64_t splits) {
  return splits > 1 ? B * splits * H * (N + 1) : 0;
}

}  // namespace ssm
}  // namespace dlr
