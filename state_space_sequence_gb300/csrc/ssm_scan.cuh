// ssm_scan.cuh -- what the selective scan's two directions share: their parameters, the cut of a
// sequence into splits, and the joining of the splits' maps.
#pragma once

#include <algorithm>

#include "ssm_common.cuh"

namespace dlr {
namespace ssm {

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
  // the splits' maps: what a split adds to the state that enters it, later what enters the next
  // one, [B, splits, H, N]; and the sum of its steps, [B, splits, H], a NaN where a mark stops all
  float *ends, *sums;
};

// A split of a sequence takes the state that enters it to P h + e: e is its end from zero, and P =
// exp(A sum of its steps). One split (the common case) has no maps. Forwards the states are joined
// from the first split on, backwards the gradients from the last one on; `ends` then holds what
// enters: the split behind (forwards), the one before (backwards).
template <bool BACK>
__global__ void join_splits(const float* A, const float* first, float* ends, const float* sums,
                            int64_t B, int splits, int64_t HN, int N) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= B * HN) return;
  const int64_t b = i / HN, k = i - b * HN, c = k / N;
  const float rate = A[k] * kLog2e;
  float h = first ? first[i] : 0.0f;
  const int64_t H = HN / N;
  // forwards splits 0 .. splits-2 pass something on, backwards splits-1 .. 1
  constexpr int kAhead = 8;
  for (int j0 = 0; j0 < splits - 1; j0 += kAhead) {
    float e[kAhead], s[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = min(j0 + u, splits - 2);
      const int64_t row = b * splits + (BACK ? splits - 1 - j : j);
      e[u] = ends[row * HN + k];
      s[u] = sums[row * H + c];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (j0 + u >= splits - 1) break;
      const int j = j0 + u;
      const int64_t row = b * splits + (BACK ? splits - 1 - j : j);
      h = s[u] != s[u] ? e[u] : fmaf(ex2(min_nan(rate * s[u], 126.0f)), h, e[u]);
      ends[row * HN + k] = h;
    }
  }
}

// The bits of a tile's marked steps (bit t: step t0 + t), the same in all lanes.
__device__ __forceinline__ uint32_t marks(const uint8_t* reset, int64_t row, int64_t t0, int64_t L,
                                          int lane) {
  if (!reset) return 0;
  const bool hit = lane < kT && t0 + lane < L && reset[row * L + t0 + lane] != 0;
  return __ballot_sync(0xffffffffu, hit);
}

// The rates of a lane's states times log2(e), in pairs of neighbouring states; zero for states and
// channels that do not exist.
__device__ __forceinline__ void load_rates(float2 (&a)[kChannels][2], const float* A, int N,
                                           int64_t c, int n_ch, int n0) {
#pragma unroll
  for (int i = 0; i < kChannels; ++i) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = i < n_ch && n0 + j < N ? A[(c + i) * N + n0 + j] * kLog2e : 0.0f;
    a[i][0] = make_float2(v[0], v[1]);
    a[i][1] = make_float2(v[2], v[3]);
  }
}
// A lane's states from an array [.., H, N] whose row of channel c begins at p (or zeros), and back.
__device__ __forceinline__ void load_states(float2 (&h)[kChannels][2], const float* p, int N,
                                            int n_ch, int n0) {
#pragma unroll
  for (int i = 0; i < kChannels; ++i) {
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (p && i < n_ch) {
      const float* q = p + (int64_t)i * N + n0;
      if ((N & 3) == 0 && n0 < N && (reinterpret_cast<uintptr_t>(q) & 15) == 0) {
        const float4 t = *reinterpret_cast<const float4*>(q);
        v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n0 + j < N) v[j] = q[j];
      }
    }
    h[i][0] = make_float2(v[0], v[1]);
    h[i][1] = make_float2(v[2], v[3]);
  }
}
__device__ __forceinline__ void store_states(float* p, const float2 (&h)[kChannels][2], int N,
                                             int n_ch, int n0) {
#pragma unroll
  for (int i = 0; i < kChannels; ++i) {
    if (i >= n_ch) break;
    float* q = p + (int64_t)i * N + n0;
    const float v[4] = {h[i][0].x, h[i][0].y, h[i][1].x, h[i][1].y};
    if ((N & 3) == 0 && n0 < N && (reinterpret_cast<uintptr_t>(q) & 15) == 0) {
      *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n0 + j < N) q[j] = v[j];
    }
  }
}

// Whether a view's pieces of `bytes` from element `first` of each row on stand on multiples of them.
template <typename T>
__host__ __device__ inline bool pieces(const view<T>& v, int64_t first, int64_t bytes) {
  return ((reinterpret_cast<uintptr_t>(v.p + first) | (uintptr_t)(v.sb * (int64_t)sizeof(T)) |
           (uintptr_t)(v.st * (int64_t)sizeof(T))) & (uintptr_t)(bytes - 1)) == 0;
}

// How many splits a sequence is cut into. The warps of a call, B * H / (128 / LN), each go through
// their rows step by step; with fewer warps than the GPU has room for the rows are cut, and the
// states at the cuts come from a pass over the steps alone.
inline int splits_for(int64_t B, int64_t L, int64_t H, int64_t N, int64_t G) {
  const int64_t cw = 128 / lanes_for(N);
  const int64_t warps = B * G * ((H / G + cw - 1) / cw), tiles = (L + kT - 1) / kT;
  if (warps >= 608 || tiles < 4) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>(tiles / 2, (1824 + warps - 1) / warps));
}

template <typename T, typename ARGS>
inputs<T> make_inputs(const ARGS& a) {
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
  const int want = splits_for(a.B, a.L, a.H, a.N, a.G);
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
