// glr_join.cuh -- what the kernels over rows share (glr_join and its gradients): a row of H
// channels belongs to a block of R threads (a multiple of 32) and stays in their registers. Item
// (j, v) of thread t is channel (j R + t) VEC + v. VEC elements make a 16-byte access when H, the
// strides and the pointers allow it, else VEC = 1. Every sum over a row is taken from registers, in
// two passes where a mean has to come off first, and each activation is read once and written once.
// Blocks stay on the GPU and go from row to row; while a row's sums go around its warps, the next
// row's inputs come into shared memory by asynchronous copies, each thread its own items, so that
// no barrier waits for them. One row to a block keeps every row's address in uniform registers.
#pragma once

#include <algorithm>

#include "glr_ckpt.cuh"

namespace dlr {
namespace glr {

constexpr int kStages = 2;  // rows in shared memory: the one at work and the next

template <typename T, int VEC>
__device__ __forceinline__ void load(const T* p, float* out) {
  words<T, VEC> k;
  k.get(p);
  k.to(out);
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T* p, const float* in) {
  words<T, VEC> k;
  k.from(in);
  k.put(p);
}
__device__ __forceinline__ float sum2(float2 v) { return v.x + v.y; }

struct JoinArgs {
  int64_t M;
  int H, norm, act;
  float eps;
  const float* w;
  const float* alpha;
  const float* v;
};
template <typename T>
struct Rows {
  T* p;
  int64_t st;
  __device__ __forceinline__ T* at(int64_t row, int c) const { return p + row * st + c; }
};
struct Ckpt {
  uint8_t *hc, *hs, *gc, *gs;
};

// The sums of K values over the threads of a block. buf holds two sets of kSums floats for each of
// 32 warps, used in turn (`turn`), so that one barrier a call is enough.
constexpr int kSums = 3;
template <int K>
__device__ __forceinline__ void row_sum(float (&s)[K], float* buf, int& turn) {
  static_assert(K <= kSums, "the sets do not meet");
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  float* set = buf + (turn & 1) * 32 * kSums;
  ++turn;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) set[(threadIdx.x >> 5) * kSums + k] = s[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = 0.0f;
  for (int j = 0; j < warps; ++j)
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] += set[j * kSums + k];
}

// A thread's items of a row as pairs of floats, and where they are.
template <int VEC, int NV>
struct Items {
  static constexpr int P = VEC * NV / 2;
  static_assert(VEC % 2 == 0 || NV % 2 == 0, "whole pairs");
  int H, R;
  __device__ __forceinline__ int channel(int j) const { return (j * R + (int)threadIdx.x) * VEC; }
  __device__ __forceinline__ bool on(int j) const { return channel(j) < H; }
  __device__ __forceinline__ bool all() const { return on(NV - 1); }  // no item past the end
  // the items of pair p's halves
  static __device__ __forceinline__ constexpr int first(int p) {
    return VEC > 1 ? p * 2 / VEC : 2 * p;
  }
  static __device__ __forceinline__ constexpr int second(int p) {
    return VEC > 1 ? p * 2 / VEC : 2 * p + 1;
  }
  // float32 parameters of the channels; 0 past the end
  __device__ __forceinline__ void params(const float* w, float2 (&out)[P]) const {
    if (all()) {
#pragma unroll
      for (int j = 0; j < NV; ++j) param<true>(w, j, out);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) param<false>(w, j, out);
    }
  }
  template <bool kAll>
  __device__ __forceinline__ void param(const float* w, int j, float2 (&out)[P]) const {
    float t[VEC] = {};
    if (kAll || on(j)) {
      if constexpr (VEC == 8) {
        load<float, 4>(w + channel(j), t);
        load<float, 4>(w + channel(j) + 4, t + 4);
      } else {
        load<float, VEC>(w + channel(j), t);
      }
    }
    place(j, t, out);
  }
  static __device__ __forceinline__ void place(int j, const float* t, float2 (&out)[P]) {
    if constexpr (VEC > 1) {
#pragma unroll
      for (int v = 0; v < VEC; v += 2) out[(j * VEC + v) / 2] = make_float2(t[v], t[v + 1]);
    } else {
      (j & 1 ? out[j / 2].y : out[j / 2].x) = t[0];
    }
  }
  static __device__ __forceinline__ void pick(int j, const float2 (&in)[P], float* t) {
    if constexpr (VEC > 1) {
#pragma unroll
      for (int v = 0; v < VEC; v += 2) {
        t[v] = in[(j * VEC + v) / 2].x;
        t[v + 1] = in[(j * VEC + v) / 2].y;
      }
    } else {
      t[0] = j & 1 ? in[j / 2].y : in[j / 2].x;
    }
  }
  // zeros past the end
  __device__ __forceinline__ void clear(float2 (&z)[P]) const {
    if (all()) return;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (!on(first(p))) z[p].x = 0.0f;
      if (!on(second(p))) z[p].y = 0.0f;
    }
  }
  template <typename T>
  __device__ __forceinline__ void put(const Rows<T>& r, int64_t row, const float2 (&in)[P]) const {
    T* p = r.at(row, 0);
    if (all()) {
#pragma unroll
      for (int j = 0; j < NV; ++j) put_one<true>(p, j, in);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) put_one<false>(p, j, in);
    }
  }
  template <bool kAll, typename T>
  __device__ __forceinline__ void put_one(T* p, int j, const float2 (&in)[P]) const {
    if (!(kAll || on(j)) || !DLR_IN_FILE(channel(j) + VEC - 1, H, 17)) return;
    float t[VEC];
    pick(j, in, t);
    store<T, VEC>(p + channel(j), t);
  }
};

// The shared memory of one array of a block's rows: item j of thread t. Copies of one stage go to
// it asynchronously (16, 8 or 4 bytes an item; single 16-bit elements and bytes by a load and a
// store). kDirect: rows too long for that; nothing is staged and the items are read from memory
// (again by the L2).
template <typename T, int VEC, int NV, bool kDirect>
struct Staged {
  static constexpr int kBytes = VEC * (int)sizeof(T);
  static constexpr bool kAsync = kBytes == 16 || kBytes == 8 || kBytes == 4;
  struct alignas(kBytes) item {
    uint8_t bytes[kBytes];
  };
  static __device__ __forceinline__ int slot(int j) {
    return j * (int)blockDim.x + (int)threadIdx.x;
  }
  static __device__ __forceinline__ int items() { return NV * (int)blockDim.x; }
  // zeros for an item that is not there
  static __device__ __forceinline__ void fetch(item* s, int j, const T* src, const T* any,
                                               bool on) {
    if constexpr (kDirect) return;
    if constexpr (kAsync) {
      const uint32_t d = (uint32_t)__cvta_generic_to_shared(s + slot(j));
      const T* p = on ? src : any;
      const int n = on ? kBytes : 0;
      if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(p), "r"(n)
                     : "memory");
      else if constexpr (kBytes == 8)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(p), "r"(n)
                     : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(p), "r"(n)
                     : "memory");
    } else {
      words<T, VEC> z;
      if (on) z.get(src);
      z.put(s + slot(j));
    }
  }
  // the items of a row that begins at p
  static __device__ __forceinline__ void fetch_row(item* s, const Items<VEC, NV>& it, const T* p) {
    if (it.all()) {
#pragma unroll
      for (int j = 0; j < NV; ++j) fetch(s, j, p + it.channel(j), p, true);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) fetch(s, j, p + it.channel(j), p, it.on(j));
    }
  }
  static __device__ __forceinline__ words<T, VEC> one(const item* s, int j, const T* src, bool on) {
    words<T, VEC> k;
    if constexpr (!kDirect)
      k.get(s + slot(j));
    else if (on)
      k.get(src);
    return k;
  }
  static __device__ __forceinline__ void get(const item* s, const Items<VEC, NV>& it,
                                             const Rows<const T>& r, int64_t row,
                                             float2 (&out)[Items<VEC, NV>::P]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float t[VEC];
      one(s, j, r.at(row, it.channel(j)), it.on(j)).to(t);
      Items<VEC, NV>::place(j, t, out);
    }
  }
};
__device__ __forceinline__ void stage_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void stage_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int P>
__device__ __forceinline__ float dot(const float2 (&a)[P], const float2 (&b)[P]) {
  float2 t = two(0.0f);
#pragma unroll
  for (int p = 0; p < P; ++p) t = fma2(a[p], b[p], t);
  return sum2(t);
}
template <int P>
__device__ __forceinline__ float total(const float2 (&a)[P]) {
  float2 t = two(0.0f);
#pragma unroll
  for (int p = 0; p < P; ++p) t = add2(t, a[p]);
  return sum2(t);
}
// z -> z less its mean. Channels past H hold 0 and are left at 0.
template <int VEC, int NV>
__device__ __forceinline__ void less_mean(const Items<VEC, NV>& it, float2 (&z)[VEC * NV / 2],
                                          float inv_h, float* buf, int& turn) {
  constexpr int P = VEC * NV / 2;
  float m[1] = {total(z)};
  row_sum<1>(m, buf, turn);
#pragma unroll
  for (int p = 0; p < P; ++p) z[p] = add2(z[p], two(-m[0] * inv_h));
  it.clear(z);
}
__device__ __forceinline__ float inverse_deviation(float squares, float inv_h, float eps) {
  return 1.0f / sqrtf(squares * inv_h + eps);
}
// z -> z less its mean (layer) and 1 / its deviation
template <int VEC, int NV>
__device__ __forceinline__ float centre(const Items<VEC, NV>& it, float2 (&z)[VEC * NV / 2],
                                        bool layer, float inv_h, float eps, float* buf, int& turn) {
  if (layer) less_mean<VEC, NV>(it, z, inv_h, buf, turn);
  float q[1] = {dot(z, z)};
  row_sum<1>(q, buf, turn);
  return inverse_deviation(q[0], inv_h, eps);
}

// act(g) = g s or s, s = sigmoid(g); g sigmoid(g) is 0 at -inf (where g is taken as a finite
// number)
__device__ __forceinline__ float2 silu(float2 g, float2 s) {
  return mul2(make_float2(max_nan(g.x, -1e30f), max_nan(g.y, -1e30f)), s);
}
// u -> u act(g)
template <int P>
__device__ __forceinline__ void apply_gate(int act, float2 (&u)[P], const float2 (&g)[P]) {
  if (act == GLR_ACT_SILU) {
#pragma unroll
    for (int p = 0; p < P; ++p) u[p] = mul2(u[p], silu(g[p], sigmoid2(g[p])));
  } else {
#pragma unroll
    for (int p = 0; p < P; ++p) u[p] = mul2(u[p], sigmoid2(g[p]));
  }
}

// 16-byte accesses of `size`-byte elements: every row begins on a 16-byte boundary and H is a
// whole number of them
inline bool wide(const void* p, int64_t st, int64_t size) {
  return !p || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(st * size)) & 15u) == 0;
}
template <typename T, typename P>
Rows<T> rows(P* p, int64_t st) {
  return {static_cast<T*>(p), st};
}

// Threads of a row, for `each` channels of a thread.
inline int row_threads(int64_t H, int each) {
  return (int)(((H + each - 1) / each + 31) / 32 * 32);
}

constexpr size_t kMostSmem = 220 * 1024;  // of an SM for the staged rows

// Blocks that go over M rows: as many as the GPU holds, by threads and shared memory.
inline cudaError_t row_blocks(int64_t M, int R, int threads, size_t smem, unsigned* blocks) {
  int dev = 0, sms = 0;
  const int most = std::min(32, std::max(1, threads / R));
  const int per_sm = smem ? std::max(1, std::min(most, (int)(kMostSmem / smem))) : most;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  *blocks = (unsigned)std::min<int64_t>(M, (int64_t)sms * per_sm);
  return e;
}

}  // namespace glr
}  // namespace dlr
