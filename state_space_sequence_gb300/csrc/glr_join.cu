// glr_join.cu -- the end of a recurrent block fused with the norm that begins the next one
// (include/glr.h, glr_join), its gradients, and the 8-bit checkpoints of activations.
//
// A row of H channels belongs to R threads (a multiple of 32) and stays in their registers: item
// (j, v) of thread t is channel (j R + t) VEC + v. VEC elements make a 16-byte access when H, the
// strides and the pointers allow it, else VEC = 1. Every sum over a row is therefore taken from
// registers, in two passes where a mean has to come off first, and each activation is read once
// and written once.
#include "glr_ckpt.cuh"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 17;

namespace glr {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kParts = 1024;  // most partial sums of a channel in the gradients

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

// The sums of K values over the R = blockDim.x threads of a row; `buf` holds K floats for every
// warp of the block. All threads of the block call it.
template <int K>
__device__ __forceinline__ void row_sum(float (&s)[K], float* buf) {
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* mine = buf + threadIdx.y * warps * K;
  __syncthreads();  // the last sums have been read
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) mine[w * K + k] = s[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = 0.0f;
  for (int j = 0; j < warps; ++j)
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] += mine[j * K + k];
}

// The norm of a row in place: z -> zhat; returns 1 / the deviation. Channels past H hold 0 and
// are left at 0.
template <int VEC, int NV>
__device__ __forceinline__ float normalise(float (&z)[NV * VEC], bool layer, int H, float eps,
                                           float* buf) {
  const int R = blockDim.x;
  if (layer) {
    float m[1] = {0.0f};
#pragma unroll
    for (int e = 0; e < NV * VEC; ++e) m[0] += z[e];
    row_sum<1>(m, buf);
    const float mean = m[0] / (float)H;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        if ((j * R + (int)threadIdx.x) * VEC + v < H) z[j * VEC + v] -= mean;
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int e = 0; e < NV * VEC; ++e) q[0] = fmaf(z[e], z[e], q[0]);
  row_sum<1>(q, buf);
  const float rstd = 1.0f / sqrtf(q[0] / (float)H + eps);
#pragma unroll
  for (int e = 0; e < NV * VEC; ++e) z[e] *= rstd;
  return rstd;
}

// act(g) and, with `slope`, its derivative
__device__ __forceinline__ float gate_act(int act, float g, float* slope) {
  const float s = sigmoid(g);
  if (act == GLR_ACT_SILU) {
    // g sigmoid(g) is 0 at -inf
    const float gs = s == 0.0f ? 0.0f : g * s;
    if (slope) *slope = s + gs * (1.0f - s);
    return gs;
  }
  if (slope) *slope = s * (1.0f - s);
  return s;
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
#pragma unroll
  for (int v = 0; v < VEC; ++v) k.v[v] = (uint8_t)encode(t[v] * inv);
  *reinterpret_cast<pack<uint8_t, VEC>*>(codes) = k;
  if ((threadIdx.x & (32 / VEC - 1)) == 0) *scale = (uint8_t)b;
}
template <int VEC>
__device__ __forceinline__ void kept(const uint8_t* codes, const uint8_t* scale, float* out) {
  const pack<uint8_t, VEC> k = *reinterpret_cast<const pack<uint8_t, VEC>*>(codes);
  const float s = scale_of(*scale);
#pragma unroll
  for (int v = 0; v < VEC; ++v) out[v] = decode(k.v[v]) * s;
}

struct Ckpt {
  uint8_t *hc, *hs, *gc, *gs;
};

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads)
join_kernel(JoinArgs a, Rows<const T> x, Rows<const T> h, Rows<const T> g, Rows<T> y, Rows<T> n,
            Ckpt ck) {
  constexpr int E = VEC * NV;
  __shared__ float buf[32];
  const int R = blockDim.x, H = a.H;
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool here = row < a.M;
  const int groups = (H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP;
  const float alpha = h.p ? *a.alpha : 0.0f;
  float z[E], u[E];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * R + (int)threadIdx.x) * VEC;
    float hv[VEC] = {}, gv[VEC] = {}, xv[VEC] = {};
    const bool on = here && c < H;
    if (on) {
      load<T, VEC>(x.at(row, c), xv);
      if (h.p) load<T, VEC>(h.at(row, c), hv);
      if (g.p) load<T, VEC>(g.at(row, c), gv);
    }
    if (ck.hc)
      keep<VEC>(hv, on, ck.hc + row * H + c, ck.hs + row * groups + c / GLR_CKPT_GROUP);
    if (ck.gc)
      keep<VEC>(gv, on, ck.gc + row * H + c, ck.gs + row * groups + c / GLR_CKPT_GROUP);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      z[j * VEC + v] = xv[v];
      u[j * VEC + v] = on ? (g.p ? hv[v] * gate_act(a.act, gv[v], nullptr) : hv[v]) : 0.0f;
    }
  }
  if (h.p) {
    normalise<VEC, NV>(u, a.norm == GLR_NORM_LAYER, H, a.eps, buf);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * R + (int)threadIdx.x) * VEC;
      if (c >= H) continue;
      float wv[VEC];
      load<float, VEC>(a.w + c, wv);
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        z[j * VEC + v] = fmaf(alpha * wv[v], u[j * VEC + v], z[j * VEC + v]);
      if (here && DLR_IN(c + VEC - 1, H)) store<T, VEC>(y.at(row, c), &z[j * VEC]);
    }
  }
  if (!n.p) return;
  normalise<VEC, NV>(z, a.norm == GLR_NORM_LAYER, H, a.eps, buf);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * R + (int)threadIdx.x) * VEC;
    if (c >= H) continue;
    float vv[VEC];
    load<float, VEC>(a.v + c, vv);
#pragma unroll
    for (int v = 0; v < VEC; ++v) vv[v] *= z[j * VEC + v];
    if (here && DLR_IN(c + VEC - 1, H)) store<T, VEC>(n.at(row, c), vv);
  }
}

// q -> rstd (q - zhat mean(q zhat) [- mean(q)]), the gradient behind a norm; returns the sum of
// q zhat over the row
template <int VEC, int NV>
__device__ __forceinline__ float norm_grad(float (&q)[NV * VEC], const float (&zhat)[NV * VEC],
                                           float rstd, float scale, bool layer, int H, float* buf) {
  float s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < NV * VEC; ++e) {
    s[0] = fmaf(q[e], zhat[e], s[0]);
    s[1] += q[e];
  }
  row_sum<2>(s, buf);
  const float m = s[0] / (float)H, mean = layer ? s[1] / (float)H : 0.0f;
#pragma unroll
  for (int e = 0; e < NV * VEC; ++e) q[e] = scale * rstd * (q[e] - zhat[e] * m - mean);
  return s[0];
}

// part: [parts, 2, H] sums of D uhat and of dn yhat, then [parts] sums of w D uhat
template <typename T, int VEC, int NV, bool kKept>
__global__ void __launch_bounds__(kMaxThreads)
join_back(JoinArgs a, Rows<const T> dy, Rows<const T> dn, Rows<const T> x, Rows<const T> h,
          Rows<const T> g, Ckpt ck, Rows<T> dx, Rows<T> dh, Rows<T> dg, float* __restrict__ part) {
  constexpr int E = VEC * NV;
  __shared__ float buf[64];
  const int R = blockDim.x, H = a.H;
  const bool layer = a.norm == GLR_NORM_LAYER, block = a.w != nullptr;
  const bool gated = block && a.act != GLR_ACT_NONE;
  const int groups = (H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP;
  const float alpha = block ? *a.alpha : 0.0f;
  float sw[E] = {}, sv[E] = {};
  double sa = 0.0;  // one term a row, of either sign: its sum may cancel
  for (int64_t row0 = (int64_t)blockIdx.x * blockDim.y; row0 < a.M;
       row0 += (int64_t)gridDim.x * blockDim.y) {
    const int64_t row = row0 + threadIdx.y;
    const bool here = row < a.M;
    float z[E], u[E], hv[E] = {}, gv[E] = {}, d[E] = {}, q[E] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * R + (int)threadIdx.x) * VEC;
      const bool on = here && c < H;
      float xv[VEC] = {};
      if (on) {
        load<T, VEC>(x.at(row, c), xv);
        if (block) {
          if (kKept)
            kept<VEC>(ck.hc + row * H + c, ck.hs + row * groups + c / GLR_CKPT_GROUP, &hv[j * VEC]);
          else
            load<T, VEC>(h.at(row, c), &hv[j * VEC]);
        }
        if (gated) {
          if (kKept)
            kept<VEC>(ck.gc + row * H + c, ck.gs + row * groups + c / GLR_CKPT_GROUP, &gv[j * VEC]);
          else
            load<T, VEC>(g.at(row, c), &gv[j * VEC]);
        }
        if (dy.p) load<T, VEC>(dy.at(row, c), &d[j * VEC]);
        if (dn.p) load<T, VEC>(dn.at(row, c), &q[j * VEC]);
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        z[j * VEC + v] = xv[v];
        const float hh = hv[j * VEC + v];
        u[j * VEC + v] = on ? (gated ? hh * gate_act(a.act, gv[j * VEC + v], nullptr) : hh) : 0.0f;
      }
    }
    float ru = 0.0f;
    if (block) {
      ru = normalise<VEC, NV>(u, layer, H, a.eps, buf);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * R + (int)threadIdx.x) * VEC;
        if (c >= H) continue;
        float wv[VEC];
        load<float, VEC>(a.w + c, wv);
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          z[j * VEC + v] = fmaf(alpha * wv[v], u[j * VEC + v], z[j * VEC + v]);
      }
    }
    if (dn.p) {
      const float ry = normalise<VEC, NV>(z, layer, H, a.eps, buf);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * R + (int)threadIdx.x) * VEC;
        if (c >= H) continue;
        float vv[VEC];
        load<float, VEC>(a.v + c, vv);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          sv[j * VEC + v] = fmaf(q[j * VEC + v], z[j * VEC + v], sv[j * VEC + v]);
          q[j * VEC + v] *= vv[v];
        }
      }
      norm_grad<VEC, NV>(q, z, ry, 1.0f, layer, H, buf);
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] += q[e];
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * R + (int)threadIdx.x) * VEC;
      if (here && c < H && DLR_IN(c + VEC - 1, H)) store<T, VEC>(dx.at(row, c), &d[j * VEC]);
    }
    if (!block) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * R + (int)threadIdx.x) * VEC;
      float wv[VEC] = {};
      if (here && c < H) load<float, VEC>(a.w + c, wv);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const int e = j * VEC + v;
        if (c >= H || !here) d[e] = 0.0f;
        sw[e] = fmaf(d[e], u[e], sw[e]);
        d[e] *= wv[v];
      }
    }
    // the row's gradients behind its norm, times alpha (so that dalpha's sum needs no division)
    const float row_sa = norm_grad<VEC, NV>(d, u, ru, alpha, layer, H, buf);
    if (threadIdx.x == 0) sa += (double)row_sa;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * R + (int)threadIdx.x) * VEC;
      if (!here || c >= H) continue;
      float oh[VEC], og[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const int e = j * VEC + v;
        float slope = 0.0f;
        const float act = gated ? gate_act(a.act, gv[e], &slope) : 1.0f;
        oh[v] = d[e] * act;
        og[v] = d[e] * hv[e] * slope;
      }
      if (DLR_IN(c + VEC - 1, H)) {
        store<T, VEC>(dh.at(row, c), oh);
        if (gated) store<T, VEC>(dg.at(row, c), og);
      }
    }
  }
  const int64_t parts = (int64_t)gridDim.x * blockDim.y;
  const int64_t me = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (!DLR_IN(me, kParts)) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * R + (int)threadIdx.x) * VEC;
    if (c >= H) continue;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      part[(me * 2) * H + c + v] = sw[j * VEC + v];
      part[(me * 2 + 1) * H + c + v] = sv[j * VEC + v];
    }
  }
  if (threadIdx.x == 0) part[parts * 2 * H + me] = (float)sa;
}

// dw, dv and dalpha from the partial sums, in a fixed order: 32 channels of one of the two sums
// to a block, its 8 warps taking every 8th part; the last block takes dalpha
__global__ void __launch_bounds__(256)
join_sums(const float* __restrict__ part, int64_t parts, int H, const float* __restrict__ alpha,
          float* __restrict__ dw, float* __restrict__ dv, float* __restrict__ dalpha) {
  __shared__ float sums[8][32];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int per = (H + 31) / 32;
  float s = 0.0f;
  if ((int)blockIdx.x == 2 * per) {
    if (!dalpha) return;
    for (int64_t k = threadIdx.x; k < parts; k += 256) s += part[parts * 2 * H + k];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) sums[row][0] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int j = 1; j < 8; ++j) s += sums[j][0];
      *dalpha = s;
    }
    return;
  }
  const int which = blockIdx.x >= per ? 1 : 0;
  const int c = ((int)blockIdx.x - which * per) * 32 + lane;
  float* out = which ? dv : dw;
  if (!out) return;
  if (c < H)
    for (int64_t k = row; k < parts; k += 8) s += part[(k * 2 + which) * H + c];
  sums[row][lane] = s;
  __syncthreads();
  if (row == 0 && c < H) {
#pragma unroll
    for (int j = 1; j < 8; ++j) s += sums[j][lane];
    out[c] = which ? s : *alpha * s;
  }
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
  kept<VEC>(codes + row * H + c, scales + group, v);
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

// threads of a row and rows of a block for a row of `items` accesses, NV to a thread
dim3 row_block(int items, int nv) {
  const int R = ((items + nv - 1) / nv + 31) / 32 * 32;
  return dim3(R, R >= 128 ? 1 : 128 / R);
}

template <typename T, int VEC, int NV>
cudaError_t join_n(const glr_join_args& a, cudaStream_t s) {
  const JoinArgs j{a.M, (int)a.H, (int)a.norm, (int)a.act, (float)a.eps, a.w, a.alpha, a.v};
  const dim3 block = row_block((int)(a.H + VEC - 1) / VEC, NV);
  const int64_t blocks = (a.M + block.y - 1) / block.y;
  join_kernel<T, VEC, NV><<<(unsigned)blocks, block, 0, s>>>(
      j, rows<const T>(a.x.data, a.x.stride_t), rows<const T>(a.h.data, a.h.stride_t),
      rows<const T>(a.g.data, a.g.stride_t), rows<T>(a.y.data, a.y.stride_t),
      rows<T>(a.n.data, a.n.stride_t), Ckpt{a.hc, a.hs, a.gc, a.gs});
  return cudaGetLastError();
}
template <typename T>
cudaError_t join_t(const glr_join_args& a, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  const int64_t z = sizeof(T);
  if (a.H % W == 0 && wide(a.x.data, a.x.stride_t, z) && wide(a.h.data, a.h.stride_t, z) &&
      wide(a.g.data, a.g.stride_t, z) && wide(a.y.data, a.y.stride_t, z) &&
      wide(a.n.data, a.n.stride_t, z) && wide(a.w, 0, 4) && wide(a.v, 0, 4) && wide(a.hc, 0, 1) &&
      wide(a.gc, 0, 1)) {
    if (a.H <= W * kMaxThreads) return join_n<T, W, 1>(a, s);
    return join_n<T, W, 16 / W>(a, s);
  }
  if (a.H <= 4 * kMaxThreads) return join_n<T, 1, 4>(a, s);
  return join_n<T, 1, 16>(a, s);
}

template <typename T, int VEC, int NV, bool kKept>
cudaError_t back_n(const glr_join_backward_args& a, cudaStream_t s) {
  const JoinArgs j{a.M, (int)a.H, (int)a.norm, (int)a.act, (float)a.eps, a.w, a.alpha, a.v};
  const dim3 block = row_block((int)(a.H + VEC - 1) / VEC, NV);
  const int64_t most = kParts / block.y, need = (a.M + block.y - 1) / block.y;
  const int64_t blocks = need < most ? need : most;
  float* part = static_cast<float*>(a.workspace);
  if (blocks > 0)
    join_back<T, VEC, NV, kKept><<<(unsigned)blocks, block, 0, s>>>(
        j, rows<const T>(a.dy.data, a.dy.stride_t), rows<const T>(a.dn.data, a.dn.stride_t),
        rows<const T>(a.x.data, a.x.stride_t), rows<const T>(a.h.data, a.h.stride_t),
        rows<const T>(a.g.data, a.g.stride_t),
        Ckpt{const_cast<uint8_t*>(a.hc), const_cast<uint8_t*>(a.hs), const_cast<uint8_t*>(a.gc),
             const_cast<uint8_t*>(a.gs)},
        rows<T>(a.dx.data, a.dx.stride_t), rows<T>(a.dh.data, a.dh.stride_t),
        rows<T>(a.dg.data, a.dg.stride_t), part);
  join_sums<<<(unsigned)(2 * ((a.H + 31) / 32) + 1), 256, 0, s>>>(
      part, blocks * block.y, (int)a.H, a.alpha, a.dw, a.dv, a.dalpha);
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
    if (a.H <= W * kMaxThreads) return back_n<T, W, 1, kKept>(a, s);
    return back_n<T, W, 16 / W, kKept>(a, s);
  }
  if (a.H <= 4 * kMaxThreads) return back_n<T, 1, 4, kKept>(a, s);
  return back_n<T, 1, 16, kKept>(a, s);
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
