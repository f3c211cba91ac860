// glr_join.cu -- the end of a recurrent block fused with the norm that begins the next one
// (include/glr.h, glr_join), its gradients, and the 8-bit checkpoints of activations.
//
// A row of H channels belongs to R threads (a multiple of 32) and stays in their registers: item
// (j, v) of thread t is channel (j R + t) VEC + v. VEC elements make a 16-byte access when H, the
// strides and the pointers allow it, else VEC = 1. Every sum over a row is therefore taken from
// registers, in two passes where a mean has to come off first, and each activation is read once
// and written once. Both kernels are bound by memory: blocks stay on the GPU and go from row to
// row, and while a row's sums go around its warps, the next row's inputs come into shared memory by
// asynchronous copies, each thread its own items, so that no barrier waits for them.
#include <algorithm>

#include "glr_ckpt.cuh"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 17;

namespace glr {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kParts = 1024;  // most partial sums of a channel in the gradients
constexpr int kStages = 2;    // rows in shared memory: the one at work and the next

template <typename T, int VEC>
__device__ __forceinline__ void load(const T* p, float* out) {
  const pack<T, VEC> k = *reinterpret_cast<const pack<T, VEC>*>(p);
#pragma unroll
  for (int v = 0; v < VEC; ++v) out[v] = to_f(k.v[v]);
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T* p, const float* in) {
  pack<T, VEC> k;
#pragma unroll
  for (int v = 0; v < VEC; ++v) k.v[v] = from_f<T>(in[v]);
  *reinterpret_cast<pack<T, VEC>*>(p) = k;
}

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

// The sums of K values over the R = blockDim.x threads of a row. buf holds two sets of kSums floats
// for each of 32 warps, used in turn (`turn`), so that one barrier a call is enough. All threads of the
// block call it.
constexpr int kSums = 2;
template <int K>
__device__ __forceinline__ void row_sum(float (&s)[K], float* buf, int& turn) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  static_assert(K <= kSums, "the sets do not meet");
  float* mine = buf + ((turn & 1) * 32 + threadIdx.y * warps) * kSums;
  ++turn;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) mine[(threadIdx.x >> 5) * kSums + k] = s[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = 0.0f;
  for (int j = 0; j < warps; ++j)
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] += mine[j * kSums + k];
}

// A thread's items of a row as pairs of floats, and where they are.
template <int VEC, int NV>
struct Items {
  static constexpr int P = VEC * NV / 2;
  static_assert(VEC % 2 == 0 || NV % 2 == 0, "whole pairs");
  int H, R;
  __device__ __forceinline__ int channel(int j) const { return (j * R + (int)threadIdx.x) * VEC; }
  __device__ __forceinline__ bool on(int j) const { return channel(j) < H; }
  // the items of pair p's halves
  static __device__ __forceinline__ constexpr int first(int p) { return VEC > 1 ? p * 2 / VEC : 2 * p; }
  static __device__ __forceinline__ constexpr int second(int p) { return VEC > 1 ? p * 2 / VEC : 2 * p + 1; }
  // float32 parameters of the channels; 0 past the end
  __device__ __forceinline__ void params(const float* w, float2 (&out)[P]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float t[VEC] = {};
      if (on(j)) {
        if constexpr (VEC == 8) {
          load<float, 4>(w + channel(j), t);
          load<float, 4>(w + channel(j) + 4, t + 4);
        } else {
          load<float, VEC>(w + channel(j), t);
        }
      }
      place(j, t, out);
    }
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
      for (int v = 0; v < VEC; v += 2) t[v] = in[(j * VEC + v) / 2].x, t[v + 1] = in[(j * VEC + v) / 2].y;
    } else {
      t[0] = j & 1 ? in[j / 2].y : in[j / 2].x;
    }
  }
  template <typename T>
  __device__ __forceinline__ void put(const Rows<T>& r, int64_t row, const float2 (&in)[P]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!on(j) || !DLR_IN(channel(j) + VEC - 1, H)) continue;
      float t[VEC];
      pick(j, in, t);
      store<T, VEC>(r.at(row, channel(j)), t);
    }
  }
};

// The shared memory of one array of a block's rows: item j of thread t. Copies of one stage go to it
// asynchronously (16, 8 or 4 bytes an item; single 16-bit elements and bytes by a load and a store).
// kDirect: rows too long for that; nothing is staged and the items are read from memory (again by the L2).
template <typename T, int VEC, int NV, bool kDirect>
struct Staged {
  static constexpr int kBytes = VEC * (int)sizeof(T);
  static constexpr bool kAsync = kBytes == 16 || kBytes == 8 || kBytes == 4;
  using item = pack<T, VEC>;
  static __device__ __forceinline__ int slot(int j) {
    return (j * (int)blockDim.y + (int)threadIdx.y) * (int)blockDim.x + (int)threadIdx.x;
  }
  static __device__ __forceinline__ int items() { return NV * (int)(blockDim.x * blockDim.y); }
  // zeros for an item that is not there
  static __device__ __forceinline__ void fetch(item* s, int j, const T* src, const T* any, bool on) {
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
      item z{};
      if (on) z = *reinterpret_cast<const item*>(src);
      s[slot(j)] = z;
    }
  }
  static __device__ __forceinline__ item one(const item* s, int j, const T* src, bool on) {
    if constexpr (kDirect) return on ? *reinterpret_cast<const item*>(src) : item{};
    else return s[slot(j)];
  }
  static __device__ __forceinline__ void get(const item* s, const Items<VEC, NV>& it, const Rows<const T>& r,
                                             int64_t row, bool here,
                                             float2 (&out)[Items<VEC, NV>::P]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const item k = one(s, j, r.at(row, it.channel(j)), here && it.on(j));
      float t[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) t[v] = to_f(k.v[v]);
      Items<VEC, NV>::place(j, t, out);
    }
  }
};
__device__ __forceinline__ void stage_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void stage_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float sum2(float2 v) { return v.x + v.y; }

// z -> z less its mean (layer) and 1 / its deviation. Channels past H hold 0 and are left at 0.
template <int VEC, int NV>
__device__ __forceinline__ float centre(const Items<VEC, NV>& it, float2 (&z)[VEC * NV / 2], bool layer,
                                        float inv_h, float eps, float* buf, int& turn) {
  constexpr int P = VEC * NV / 2;
  if (layer) {
    float2 t = two(0.0f);
#pragma unroll
    for (int p = 0; p < P; ++p) t = add2(t, z[p]);
    float m[1] = {sum2(t)};
    row_sum<1>(m, buf, turn);
    const float mean = m[0] * inv_h;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (it.on(it.first(p))) z[p].x -= mean;
      if (it.on(it.second(p))) z[p].y -= mean;
    }
  }
  float2 t = two(0.0f);
#pragma unroll
  for (int p = 0; p < P; ++p) t = fma2(z[p], z[p], t);
  float q[1] = {sum2(t)};
  row_sum<1>(q, buf, turn);
  return 1.0f / sqrtf(q[0] * inv_h + eps);
}

// act(g); g sigmoid(g) is 0 at -inf
__device__ __forceinline__ float2 gate_act(int act, float2 g, float2 s) {
  if (act != GLR_ACT_SILU) return s;
  const float2 t = mul2(g, s);
  return make_float2(s.x == 0.0f ? 0.0f : t.x, s.y == 0.0f ? 0.0f : t.y);
}

// VEC codes and their group's scale. A group is 32 / VEC neighbouring lanes.
template <int VEC>
__device__ __forceinline__ void keep(const float* t, bool on, uint8_t* codes, uint8_t* scale) {
  float amax = 0.0f;
#pragma unroll
  for (int v = 0; v < VEC; ++v) amax = fmaxf(amax, finite_abs(t[v]));
#pragma unroll
  for (int o = 16 / VEC; o >= 1; o >>= 1)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (!on) return;
  const int b = scale_byte(amax);
  const float inv = inverse_scale_of(b);
  pack<uint8_t, VEC> k;
  if constexpr (VEC == 1) {
    k.v[0] = (uint8_t)encode(t[0] * inv);
  } else {
#pragma unroll
    for (int v = 0; v < VEC; v += 2) {
      const uint32_t two = encode2(mul2(make_float2(t[v], t[v + 1]), glr::two(inv)));
      k.v[v] = (uint8_t)two, k.v[v + 1] = (uint8_t)(two >> 8);
    }
  }
  *reinterpret_cast<pack<uint8_t, VEC>*>(codes) = k;
  if ((threadIdx.x & (32 / VEC - 1)) == 0) *scale = (uint8_t)b;
}
template <int VEC>
__device__ __forceinline__ void kept(const pack<uint8_t, VEC>& k, int scale, float* out) {
  const float s = scale_of(scale);
  if constexpr (VEC == 1) {
    out[0] = decode(k.v[0]) * s;
  } else {
#pragma unroll
    for (int v = 0; v < VEC; v += 2) {
      const float2 t = mul2(decode2((uint32_t)k.v[v] | (uint32_t)k.v[v + 1] << 8), two(s));
      out[v] = t.x, out[v + 1] = t.y;
    }
  }
}

template <typename T, int VEC, int NV, bool kDirect, int kThreads, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks)
join_kernel(JoinArgs a, Rows<const T> x, Rows<const T> h, Rows<const T> g, Rows<T> y, Rows<T> n,
            Ckpt ck) {
  constexpr int P = VEC * NV / 2;
  using St = Staged<T, VEC, NV, kDirect>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float buf[64 * kSums];
  typename St::item* const sm = reinterpret_cast<typename St::item*>(smem);  // [kStages][x h g][items]
  const Items<VEC, NV> it{a.H, (int)blockDim.x};
  const int per = St::items();
  const bool layer = a.norm == GLR_NORM_LAYER;
  const int groups = (a.H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP;
  const float alpha = h.p ? *a.alpha : 0.0f, inv_h = 1.0f / (float)a.H;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  auto fetch = [&](int64_t r, int k) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool on = r < a.M && it.on(j);
      const int c = it.channel(j);
      St::fetch(sm + (k * 3) * per, j, x.at(r, c), x.p, on);
      if (h.p) St::fetch(sm + (k * 3 + 1) * per, j, h.at(r, c), h.p, on);
      if (g.p) St::fetch(sm + (k * 3 + 2) * per, j, g.at(r, c), g.p, on);
    }
    stage_end();
  };
  fetch(row, 0);
  int turn = 0;
  for (int k = 0; row - threadIdx.y < a.M; row += step, k ^= 1) {
    const bool here = row < a.M;
    fetch(row + step, k ^ 1);
    stage_wait<1>();
    float2 z[P], u[P];
    St::get(sm + (k * 3) * per, it, x, row, here, z);
    if (h.p) {
      St::get(sm + (k * 3 + 1) * per, it, h, row, here, u);
      auto code = [&](const float2 (&v)[P], uint8_t* codes, uint8_t* scales) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float t[VEC];
          it.pick(j, v, t);
          const int c = it.channel(j);
          keep<VEC>(t, here && it.on(j), codes + row * a.H + c,
                    scales + row * groups + c / GLR_CKPT_GROUP);
        }
      };
      if (ck.hc) code(u, ck.hc, ck.hs);
      if (g.p) {
        float2 gv[P];
        St::get(sm + (k * 3 + 2) * per, it, g, row, here, gv);
        if (ck.gc) code(gv, ck.gc, ck.gs);
#pragma unroll
        for (int p = 0; p < P; ++p) u[p] = mul2(u[p], gate_act(a.act, gv[p], sigmoid2(gv[p])));
      }
      const float ru = centre<VEC, NV>(it, u, layer, inv_h, a.eps, buf, turn);
      float2 w[P];
      it.params(a.w, w);
      const float2 c = two(alpha * ru);
#pragma unroll
      for (int p = 0; p < P; ++p) z[p] = fma2(mul2(w[p], u[p]), c, z[p]);
      if (here) it.put(y, row, z);
    }
    if (n.p) {
      const float2 ry = two(centre<VEC, NV>(it, z, layer, inv_h, a.eps, buf, turn));
      float2 v[P];
      it.params(a.v, v);
#pragma unroll
      for (int p = 0; p < P; ++p) v[p] = mul2(v[p], mul2(z[p], ry));
      if (here) it.put(n, row, v);
    }
  }
  stage_wait<0>();
}

// part: [parts, 2, H] sums of D uhat and of dn yhat, then [parts] sums of w D uhat
template <typename T, int VEC, int NV, bool kKept, bool kDirect, int kThreads, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks)
join_back(JoinArgs a, Rows<const T> dy, Rows<const T> dn, Rows<const T> x, Rows<const T> h,
          Rows<const T> g, Ckpt ck, Rows<T> dx, Rows<T> dh, Rows<T> dg, float* __restrict__ part) {
  constexpr int P = VEC * NV / 2;
  using St = Staged<T, VEC, NV, kDirect>;
  using Sc = Staged<uint8_t, VEC, NV, kDirect>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float buf[64 * kSums];
  const Items<VEC, NV> it{a.H, (int)blockDim.x};
  const int per = St::items();
  const bool layer = a.norm == GLR_NORM_LAYER, block = a.w != nullptr;
  const bool gated = block && a.act != GLR_ACT_NONE;
  const int groups = (a.H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP;
  const float alpha = block ? *a.alpha : 0.0f, inv_h = 1.0f / (float)a.H;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  // [kStages][x dy dn h g][items]; codes take the places of h and g
  auto at = [&](int k, int array) {
    return reinterpret_cast<typename St::item*>(smem) + (k * 5 + array) * per;
  };
  auto codes_at = [&](int k, int array) { return reinterpret_cast<typename Sc::item*>(at(k, array)); };
  int scale_h[NV] = {}, scale_g[NV] = {};  // of the next row
  auto fetch = [&](int64_t r, int k) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool on = r < a.M && it.on(j);
      const int c = it.channel(j);
      St::fetch(at(k, 0), j, x.at(r, c), x.p, on);
      if (dy.p) St::fetch(at(k, 1), j, dy.at(r, c), dy.p, on);
      if (dn.p) St::fetch(at(k, 2), j, dn.at(r, c), dn.p, on);
      if constexpr (kKept) {
        Sc::fetch(codes_at(k, 3), j, ck.hc + r * a.H + c, ck.hc, on);
        if (gated) Sc::fetch(codes_at(k, 4), j, ck.gc + r * a.H + c, ck.gc, on);
        const int64_t s = r * groups + c / GLR_CKPT_GROUP;
        scale_h[j] = on ? ck.hs[s] : 0;
        if (gated) scale_g[j] = on ? ck.gs[s] : 0;
      } else {
        if (block) St::fetch(at(k, 3), j, h.at(r, c), h.p, on);
        if (gated) St::fetch(at(k, 4), j, g.at(r, c), g.p, on);
      }
    }
    stage_end();
  };
  float2 sw[P] = {}, sv[P] = {};
  double sa = 0.0;  // one term a row, of either sign: its sum may cancel
  int turn = 0;
  fetch(row, 0);
  for (int k = 0; row - threadIdx.y < a.M; row += step, k ^= 1) {
    const bool here = row < a.M;
    int sch[NV], scg[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) sch[j] = scale_h[j], scg[j] = scale_g[j];
    fetch(row + step, k ^ 1);
    stage_wait<1>();
    auto read = [&](int array, const int (&scale)[NV], float2 (&out)[P]) {  // 3: h, 4: g
      if constexpr (kKept) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float t[VEC];
          const uint8_t* src = (array == 3 ? ck.hc : ck.gc) + row * a.H + it.channel(j);
          kept<VEC>(Sc::one(codes_at(k, array), j, src, here && it.on(j)), scale[j], t);
          it.place(j, t, out);
        }
      } else {
        St::get(at(k, array), it, array == 3 ? h : g, row, here, out);
      }
    };
    float2 z[P], u[P], w[P];
    St::get(at(k, 0), it, x, row, here, z);
    float ru = 0.0f;
    if (block) {
      read(3, sch, u);
      if (gated) {
        float2 gv[P];
        read(4, scg, gv);
#pragma unroll
        for (int p = 0; p < P; ++p) u[p] = mul2(u[p], gate_act(a.act, gv[p], sigmoid2(gv[p])));
      }
      ru = centre<VEC, NV>(it, u, layer, inv_h, a.eps, buf, turn);
      it.params(a.w, w);
      const float2 c = two(alpha * ru);
#pragma unroll
      for (int p = 0; p < P; ++p) z[p] = fma2(mul2(w[p], u[p]), c, z[p]);
    }
    float2 d[P];
    if (dn.p) {
      const float ry = centre<VEC, NV>(it, z, layer, inv_h, a.eps, buf, turn);
      float2 q[P], v[P], s0 = two(0.0f), s1 = two(0.0f);
      St::get(at(k, 2), it, dn, row, here, q);
      it.params(a.v, v);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        z[p] = mul2(z[p], two(ry));  // yhat
        sv[p] = fma2(q[p], z[p], sv[p]);
        q[p] = mul2(q[p], v[p]);
        s0 = fma2(q[p], z[p], s0);
        s1 = add2(s1, q[p]);
      }
      float s[2] = {sum2(s0), sum2(s1)};
      row_sum<2>(s, buf, turn);
      // what cancels does so before it is scaled
      const float2 m = two(-s[0] * inv_h), mean = two(layer ? -s[1] * inv_h : 0.0f);
#pragma unroll
      for (int p = 0; p < P; ++p) z[p] = mul2(fma2(z[p], m, add2(q[p], mean)), two(ry));
    }
    if (dy.p) {
      St::get(at(k, 1), it, dy, row, here, d);
#pragma unroll
      for (int p = 0; p < P; ++p) d[p] = dn.p ? add2(d[p], z[p]) : d[p];
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) d[p] = dn.p ? z[p] : two(0.0f);
    }
    if (here) it.put(dx, row, d);
    if (!block) continue;
    it.params(a.w, w);
    float2 s0 = two(0.0f), s1 = two(0.0f);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      u[p] = mul2(u[p], two(ru));  // uhat
      if (!here || !it.on(it.first(p))) d[p].x = 0.0f;
      if (!here || !it.on(it.second(p))) d[p].y = 0.0f;
      sw[p] = fma2(d[p], u[p], sw[p]);
      d[p] = mul2(d[p], w[p]);
      s0 = fma2(d[p], u[p], s0);
      s1 = add2(s1, d[p]);
    }
    float s[2] = {sum2(s0), sum2(s1)};
    row_sum<2>(s, buf, turn);
    if (threadIdx.x == 0) sa += (double)s[0];
    // alpha stands outside, so that dalpha's sum needs no division
    const float ar = alpha * ru;
    const float2 m = two(-s[0] * inv_h), mean = two(layer ? -s[1] * inv_h : 0.0f);
#pragma unroll
    for (int p = 0; p < P; ++p) d[p] = mul2(fma2(u[p], m, add2(d[p], mean)), two(ar));
    if (gated) {
      float2 hv[P], gv[P];
      read(3, sch, hv);
      read(4, scg, gv);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const float2 sg = sigmoid2(gv[p]), act = gate_act(a.act, gv[p], sg);
        // s + g s (1 - s), or s (1 - s)
        const float2 rest = fma2(sg, two(-1.0f), two(1.0f));
        const float2 slope = a.act == GLR_ACT_SILU ? fma2(act, rest, sg) : mul2(sg, rest);
        gv[p] = mul2(mul2(d[p], hv[p]), slope);
        d[p] = mul2(d[p], act);
      }
      if (here) it.put(dg, row, gv);
    }
    if (here) it.put(dh, row, d);
  }
  stage_wait<0>();
  const int64_t parts = (int64_t)gridDim.x * blockDim.y;
  const int64_t me = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (!DLR_IN(me, kParts)) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (!it.on(j)) continue;
    float t[VEC];
    it.pick(j, sw, t);
    store<float, VEC == 8 ? 4 : VEC>(part + (me * 2) * a.H + it.channel(j), t);
    if constexpr (VEC == 8) store<float, 4>(part + (me * 2) * a.H + it.channel(j) + 4, t + 4);
    it.pick(j, sv, t);
    store<float, VEC == 8 ? 4 : VEC>(part + (me * 2 + 1) * a.H + it.channel(j), t);
    if constexpr (VEC == 8) store<float, 4>(part + (me * 2 + 1) * a.H + it.channel(j) + 4, t + 4);
  }
  if (threadIdx.x == 0) part[parts * 2 * a.H + me] = (float)sa;
}

// dw, dv and dalpha from the partial sums, in a fixed order: 32 channels of one of the two sums to
// a block, its 32 warps taking every 32nd part; the last block takes dalpha
__global__ void __launch_bounds__(1024)
join_sums(const float* __restrict__ part, int parts, int H, const float* __restrict__ alpha,
          float* __restrict__ dw, float* __restrict__ dv, float* __restrict__ dalpha) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int per = (H + 31) / 32;
  if ((int)blockIdx.x == 2 * per) {
    if (!dalpha || row) return;
    double s = 0.0;
    for (int k = lane; k < parts; k += 32) s += (double)part[(int64_t)parts * 2 * H + k];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) *dalpha = (float)s;
    return;
  }
  const int which = (int)blockIdx.x >= per ? 1 : 0;
  const int c = ((int)blockIdx.x - which * per) * 32 + lane;
  float* out = which ? dv : dw;
  if (!out) return;
  float s = 0.0f;
  if (c < H)
#pragma unroll 8
    for (int k = row; k < parts; k += 32) s += part[((int64_t)k * 2 + which) * H + c];
  sums[row][lane] = s;
  __syncthreads();
  // warp `row` adds up channel `row` of the 32
  s = sums[lane][row];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int to = c - lane + row;
  if (lane == 0 && to < H) out[to] = which ? s : *alpha * s;
}

// 8-bit checkpoints alone: VEC channels to a thread, 32 / VEC threads to a group
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
pack_kernel(Rows<const T> t, int64_t M, int H, uint8_t* __restrict__ codes,
            uint8_t* __restrict__ scales) {
  const int groups = (H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP;
  const int64_t k = (blockIdx.x * (int64_t)256 + threadIdx.x) * VEC;
  const int64_t group = k / GLR_CKPT_GROUP;
  const int64_t row = group / groups;
  const int c = (int)(group % groups) * GLR_CKPT_GROUP + (int)(k % GLR_CKPT_GROUP);
  const bool on = row < M && c < H;
  float v[VEC] = {};
  if (on) load<T, VEC>(t.at(row, c), v);
  keep<VEC>(v, on, codes + row * H + c, scales + group);
}
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
unpack_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t M,
              int H, Rows<T> t) {
  const int groups = (H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP;
  const int64_t k = (blockIdx.x * (int64_t)256 + threadIdx.x) * VEC;
  const int64_t group = k / GLR_CKPT_GROUP;
  const int64_t row = group / groups;
  const int c = (int)(group % groups) * GLR_CKPT_GROUP + (int)(k % GLR_CKPT_GROUP);
  if (row >= M || c >= H) return;
  float v[VEC];
  kept<VEC>(*reinterpret_cast<const pack<uint8_t, VEC>*>(codes + row * H + c), scales[group], v);
  store<T, VEC>(t.at(row, c), v);
}

template <typename T, typename P>
Rows<T> rows(P* p, int64_t st) {
  return {static_cast<T*>(p), st};
}

// 16-byte accesses of `size`-byte elements: every row begins on a 16-byte boundary and H is a
// whole number of them
bool wide(const void* p, int64_t st, int64_t size) {
  return !p || ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(st * size)) & 15u) == 0;
}

// Threads of a row and rows of a block, for NV accesses of a thread.
dim3 row_block(int64_t H, int vec, int nv) {
  const int R = (int)(((H + vec * nv - 1) / (vec * nv) + 31) / 32 * 32);
  return dim3(R, R >= 128 ? 1 : 128 / R);
}

constexpr size_t kMostSmem = 220 * 1024;  // of an SM for the staged rows

// Blocks that go over M rows: as many as the GPU holds of them, by their threads and shared memory.
cudaError_t row_blocks(int64_t M, dim3 block, int threads, size_t smem, unsigned* blocks) {
  int dev = 0, sms = 0;
  const int most = std::max(1, threads / (int)(block.x * block.y));
  const int per_sm = smem ? std::max(1, std::min(most, (int)(kMostSmem / smem))) : most;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  *blocks = (unsigned)std::min<int64_t>((M + block.y - 1) / block.y, (int64_t)sms * per_sm);
  return e;
}

template <typename T, int VEC, int NV, int kThreads, int kBlocks>
cudaError_t join_n(const glr_join_args& a, cudaStream_t s) {
  const JoinArgs j{a.M, (int)a.H, (int)a.norm, (int)a.act, (float)a.eps, a.w, a.alpha, a.v};
  const dim3 block = row_block(a.H, VEC, NV);
  constexpr size_t staged = kStages * 3 * NV * VEC * sizeof(T);  // of a thread
  constexpr bool kDirect = staged * kThreads > kMostSmem;
  constexpr size_t per = kDirect ? 0 : staged;
  constexpr auto kernel = join_kernel<T, VEC, NV, kDirect, kThreads, kBlocks>;
  unsigned blocks;
  cudaError_t e = row_blocks(a.M, block, kBlocks * kThreads, per * block.x * block.y, &blocks);
  if (e == cudaSuccess) e = max_smem_once<kernel>(per * kThreads);
  if (e != cudaSuccess) return e;
  kernel<<<blocks, block, per * block.x * block.y, s>>>(
      j, rows<const T>(a.x.data, a.x.stride_t), rows<const T>(a.h.data, a.h.stride_t),
      rows<const T>(a.g.data, a.g.stride_t), rows<T>(a.y.data, a.y.stride_t),
      rows<T>(a.n.data, a.n.stride_t), Ckpt{a.hc, a.hs, a.gc, a.gs});
  return cudaGetLastError();
}
// The accesses of a thread grow with the row: a block of 128 threads holds up to 16 floats of a row in each, which keeps
// four such blocks on an SM; longer rows take more threads.
template <typename T>
cudaError_t join_t(const glr_join_args& a, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  const int64_t z = sizeof(T);
  if (a.H % W == 0 && wide(a.x.data, a.x.stride_t, z) && wide(a.h.data, a.h.stride_t, z) &&
      wide(a.g.data, a.g.stride_t, z) && wide(a.y.data, a.y.stride_t, z) &&
      wide(a.n.data, a.n.stride_t, z) && wide(a.w, 0, 4) && wide(a.v, 0, 4) && wide(a.hc, 0, 1) &&
      wide(a.gc, 0, 1)) {
    if (a.H <= 16 * 128) return join_n<T, W, 16 / W, 128, 5>(a, s);
    if (a.H <= 16 * 256) return join_n<T, W, 16 / W, 256, 2>(a, s);
    if (a.H <= 16 * 512) return join_n<T, W, 16 / W, 512, 1>(a, s);
    return join_n<T, W, 16 / W, 1024, 1>(a, s);
  }
  if (a.H <= 4 * 128) return join_n<T, 1, 4, 128, 8>(a, s);
  if (a.H <= 8 * 256) return join_n<T, 1, 8, 256, 3>(a, s);
  return join_n<T, 1, 16, 1024, 1>(a, s);
}

template <typename T, int VEC, int NV, bool kKept, int kThreads, int kBlocks>
cudaError_t back_n(const glr_join_backward_args& a, cudaStream_t s) {
  const JoinArgs j{a.M, (int)a.H, (int)a.norm, (int)a.act, (float)a.eps, a.w, a.alpha, a.v};
  const dim3 block = row_block(a.H, VEC, NV);
  constexpr size_t staged = kStages * 5 * NV * VEC * sizeof(T);  // of a thread
  constexpr bool kDirect = staged * kThreads > kMostSmem;
  constexpr size_t per = kDirect ? 0 : staged;
  constexpr auto kernel = join_back<T, VEC, NV, kKept, kDirect, kThreads, kBlocks>;
  unsigned blocks = 0;
  cudaError_t e = row_blocks(a.M, block, kBlocks * kThreads, per * block.x * block.y, &blocks);
  blocks = std::min<unsigned>(blocks, kParts / block.y);
  if (e == cudaSuccess) e = max_smem_once<kernel>(per * kThreads);
  if (e != cudaSuccess) return e;
  float* part = static_cast<float*>(a.workspace);
  if (blocks > 0)
    kernel<<<blocks, block, per * block.x * block.y, s>>>(
        j, rows<const T>(a.dy.data, a.dy.stride_t), rows<const T>(a.dn.data, a.dn.stride_t),
        rows<const T>(a.x.data, a.x.stride_t), rows<const T>(a.h.data, a.h.stride_t),
        rows<const T>(a.g.data, a.g.stride_t),
        Ckpt{const_cast<uint8_t*>(a.hc), const_cast<uint8_t*>(a.hs), const_cast<uint8_t*>(a.gc),
             const_cast<uint8_t*>(a.gs)},
        rows<T>(a.dx.data, a.dx.stride_t), rows<T>(a.dh.data, a.dh.stride_t),
        rows<T>(a.dg.data, a.dg.stride_t), part);
  join_sums<<<(unsigned)(2 * ((a.H + 31) / 32) + 1), 1024, 0, s>>>(
      part, (int)(blocks * block.y), (int)a.H, a.alpha, a.dw, a.dv, a.dalpha);
  return cudaGetLastError();
}
template <typename T, bool kKept>
cudaError_t back_t(const glr_join_backward_args& a, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  const int64_t z = sizeof(T);
  if (a.H % W == 0 && wide(a.dy.data, a.dy.stride_t, z) && wide(a.dn.data, a.dn.stride_t, z) &&
      wide(a.x.data, a.x.stride_t, z) && wide(a.h.data, a.h.stride_t, z) &&
      wide(a.g.data, a.g.stride_t, z) && wide(a.dx.data, a.dx.stride_t, z) &&
      wide(a.dh.data, a.dh.stride_t, z) && wide(a.dg.data, a.dg.stride_t, z) &&
      wide(a.w, 0, 4) && wide(a.v, 0, 4) && wide(a.hc, 0, 1) && wide(a.gc, 0, 1)) {
    if (a.H <= 16 * 128) return back_n<T, W, 16 / W, kKept, 128, 4>(a, s);
    if (a.H <= 16 * 256) return back_n<T, W, 16 / W, kKept, 256, 2>(a, s);
    if (a.H <= 16 * 512) return back_n<T, W, 16 / W, kKept, 512, 1>(a, s);
    return back_n<T, W, 16 / W, kKept, 1024, 1>(a, s);
  }
  if (a.H <= 4 * 256) return back_n<T, 1, 4, kKept, 256, 3>(a, s);
  if (a.H <= 16 * 256) return back_n<T, 1, 16, kKept, 256, 2>(a, s);
  return back_n<T, 1, 16, kKept, 1024, 1>(a, s);
}
template <typename T>
cudaError_t back_k(const glr_join_backward_args& a, cudaStream_t s) {
  return a.hc ? back_t<T, true>(a, s) : back_t<T, false>(a, s);
}

template <typename T>
cudaError_t pack_t(int64_t M, int64_t H, const void* t, int64_t st, uint8_t* codes,
                   uint8_t* scales, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  const int64_t n = M * ((H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP) * GLR_CKPT_GROUP;
  const Rows<const T> r = rows<const T>(t, st);
  if (H % W == 0 && wide(t, st, sizeof(T)) && wide(codes, 0, 1))
    pack_kernel<T, W><<<(unsigned)((n / W + 255) / 256), 256, 0, s>>>(r, M, (int)H, codes, scales);
  else
    pack_kernel<T, 1><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(r, M, (int)H, codes, scales);
  return cudaGetLastError();
}
template <typename T>
cudaError_t unpack_t(int64_t M, int64_t H, const uint8_t* codes, const uint8_t* scales, void* t,
                     int64_t st, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  const int64_t n = M * ((H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP) * GLR_CKPT_GROUP;
  const Rows<T> r = rows<T>(t, st);
  if (H % W == 0 && wide(t, st, sizeof(T)) && wide(codes, 0, 1))
    unpack_kernel<T, W><<<(unsigned)((n / W + 255) / 256), 256, 0, s>>>(codes, scales, M, (int)H, r);
  else
    unpack_kernel<T, 1><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(codes, scales, M, (int)H, r);
  return cudaGetLastError();
}

}  // namespace

size_t join_backward_workspace_bytes(int64_t H) {
  return sizeof(float) * (size_t)kParts * (2 * (size_t)H + 1);
}

cudaError_t launch_join(const glr_join_args& a, cudaStream_t s) {
  if (a.type == GLR_BF16) return join_t<__nv_bfloat16>(a, s);
  if (a.type == GLR_F16) return join_t<__half>(a, s);
  return join_t<float>(a, s);
}
cudaError_t launch_join_backward(const glr_join_backward_args& a, cudaStream_t s) {
  if (a.type == GLR_BF16) return back_k<__nv_bfloat16>(a, s);
  if (a.type == GLR_F16) return back_k<__half>(a, s);
  return back_k<float>(a, s);
}
cudaError_t launch_pack(int64_t type, int64_t M, int64_t H, const void* t, int64_t st,
                        uint8_t* codes, uint8_t* scales, cudaStream_t s) {
  if (type == GLR_BF16) return pack_t<__nv_bfloat16>(M, H, t, st, codes, scales, s);
  if (type == GLR_F16) return pack_t<__half>(M, H, t, st, codes, scales, s);
  return pack_t<float>(M, H, t, st, codes, scales, s);
}
cudaError_t launch_unpack(int64_t type, int64_t M, int64_t H, const uint8_t* codes,
                          const uint8_t* scales, void* t, int64_t st, cudaStream_t s) {
  if (type == GLR_BF16) return unpack_t<__nv_bfloat16>(M, H, codes, scales, t, st, s);
  if (type == GLR_F16) return unpack_t<__half>(M, H, codes, scales, t, st, s);
  return unpack_t<float>(M, H, codes, scales, t, st, s);
}

}  // namespace glr
}  // namespace dlr
