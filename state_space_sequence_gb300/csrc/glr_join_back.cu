// glr_join_back.cu -- the gradients of glr_join (include/glr.h). A row's statistics are computed
// again from x, h and g, which are read anyway; the sums over the rows (dw, dv, dalpha) stay in
// each block's registers to the end, go to the workspace once a block, and are added up in a fixed
// order (dalpha in 64 bits, at no cost in time).
//
// Five rows in and three out. 32768 x 2048 bfloat16 takes 215 us with the sums (5.0 TB/s, 73% of a
// plain copy's bandwidth): 71 instructions an element fill 58% of the issue slots, and with 16
// warps on an SM the rest goes on waiting between a row's sums; more warps with fewer registers
// spill (96 of them: 286 us; 8 channels to a thread: 385 us). From 8-bit checkpoints 65536 x 1024
// takes 233 us (60%), bound the same way with a quarter fewer bytes. 8191 x 515 float32 takes 64 us
// (31%). Rows of single channels from 769 on and all rows above 8192 channels spill (100 to 1640
// bytes a thread): 33520 x 1001 float32 884 us (18%), bfloat16 977 us (8%), 2730 x 12288 bfloat16
// 272 us (29%). glr_join.cuh has the layout.
#include "glr_join.cuh"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 19;

namespace glr {
namespace {

// part: [parts, 2, H] sums of D uhat and of dn yhat, then [parts] sums of w D uhat in 64 bits.
// dalpha is one sum over all rows and channels, of terms of either sign, and may come out far below
// the root of their squares' sum: a thread adds up its channels of a row in 32 bits, everything
// beyond them in 64.
template <typename T, int VEC, int NV, bool kKept, bool kDirect, int kThreads, int kResident>
__global__ void __launch_bounds__(kThreads, kResident / kThreads)
join_back(JoinArgs a, Rows<const T> dy, Rows<const T> dn, Rows<const T> x, Rows<const T> h,
          Rows<const T> g, Ckpt ck, Rows<T> dx, Rows<T> dh, Rows<T> dg, float* __restrict__ part) {
  constexpr int P = VEC * NV / 2;
  using St = Staged<T, VEC, NV, kDirect>;
  using Sc = Staged<uint8_t, VEC, NV, kDirect>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float buf[64 * kSums];
  __shared__ double own[32];
  const Items<VEC, NV> it{a.H, (int)blockDim.x};
  const int per = St::items();
  const bool layer = a.norm == GLR_NORM_LAYER, block = a.w != nullptr;
  const bool gated = block && a.act != GLR_ACT_NONE;
  const int groups = (a.H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP;
  const float alpha = block ? *a.alpha : 0.0f, inv_h = 1.0f / (float)a.H;
  int64_t row = blockIdx.x;
  // [kStages][x dy dn h g][items]; codes take the places of h and g
  auto at = [&](int k, int array) {
    return reinterpret_cast<typename St::item*>(smem) + (k * 5 + array) * per;
  };
  auto codes_at = [&](int k, int array) {
    return reinterpret_cast<typename Sc::item*>(at(k, array));
  };
  int scale_h[NV] = {}, scale_g[NV] = {};  // of the next row
  auto fetch = [&](int64_t r, int k) {
    if (r < a.M) {
      St::fetch_row(at(k, 0), it, x.at(r, 0));
      if (dy.p) St::fetch_row(at(k, 1), it, dy.at(r, 0));
      if (dn.p) St::fetch_row(at(k, 2), it, dn.at(r, 0));
      if constexpr (kKept) {
        Sc::fetch_row(codes_at(k, 3), it, ck.hc + r * a.H);
        if (gated) Sc::fetch_row(codes_at(k, 4), it, ck.gc + r * a.H);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int64_t s = r * groups + it.channel(j) / GLR_CKPT_GROUP;
          scale_h[j] = it.on(j) ? ck.hs[s] : 0;
          if (gated) scale_g[j] = it.on(j) ? ck.gs[s] : 0;
        }
      } else {
        if (block) St::fetch_row(at(k, 3), it, h.at(r, 0));
        if (gated) St::fetch_row(at(k, 4), it, g.at(r, 0));
      }
    }
    stage_end();
  };
  float2 sw[P] = {}, sv[P] = {};
  double sa = 0.0;  // of this thread's channels
  int turn = 0;
  fetch(row, 0);
  for (int k = 0; row < a.M; row += gridDim.x, k ^= 1) {
    int sch[NV], scg[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) sch[j] = scale_h[j], scg[j] = scale_g[j];
    fetch(row + gridDim.x, k ^ 1);
    stage_wait<1>();
    auto read = [&](int array, const int (&scale)[NV], float2 (&out)[P]) {  // 3: h, 4: g
      if constexpr (kKept) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float t[VEC];
          const uint8_t* src = (array == 3 ? ck.hc : ck.gc) + row * a.H + it.channel(j);
          kept<VEC>(Sc::one(codes_at(k, array), j, src, it.on(j)), scale[j], t);
          it.place(j, t, out);
        }
      } else {
        St::get(at(k, array), it, array == 3 ? h : g, row, out);
      }
    };
    float2 z[P], u[P], w[P];
    St::get(at(k, 0), it, x, row, z);
    float ru = 0.0f;
    if (block) {
      read(3, sch, u);
      if (gated) {
        float2 gv[P];
        read(4, scg, gv);
        apply_gate(a.act, u, gv);
      }
      ru = centre<VEC, NV>(it, u, layer, inv_h, a.eps, buf, turn);
      it.params(a.w, w);
      const float2 c = two(alpha * ru);
#pragma unroll
      for (int p = 0; p < P; ++p) z[p] = fma2(mul2(w[p], u[p]), c, z[p]);
    }
    float2 d[P];
    if (dn.p) {
      // the squares and the products with q = v dn go around together; yhat = ry z
      float2 q[P], v[P];
      if (layer) less_mean<VEC, NV>(it, z, inv_h, buf, turn);
      St::get(at(k, 2), it, dn, row, v);
      it.params(a.v, q);
#pragma unroll
      for (int p = 0; p < P; ++p) q[p] = mul2(q[p], v[p]);
      float sq = 0.0f, sz = dot(z, z), sqz = dot(q, z);
      if (layer) {
        float s[3] = {sz, sqz, total(q)};
        row_sum<3>(s, buf, turn);
        sz = s[0], sqz = s[1], sq = s[2];
      } else {
        float s[2] = {sz, sqz};
        row_sum<2>(s, buf, turn);
        sz = s[0], sqz = s[1];
      }
      const float ry = inverse_deviation(sz, inv_h, a.eps);
      St::get(at(k, 2), it, dn, row, v);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        z[p] = mul2(z[p], two(ry));
        sv[p] = fma2(v[p], z[p], sv[p]);
      }
      // what cancels does so before it is scaled
      const float2 m = two(-ry * sqz * inv_h), mean = two(-sq * inv_h);
#pragma unroll
      for (int p = 0; p < P; ++p) z[p] = mul2(fma2(z[p], m, add2(q[p], mean)), two(ry));
    }
    if (dy.p && dn.p) {
      St::get(at(k, 1), it, dy, row, d);
#pragma unroll
      for (int p = 0; p < P; ++p) d[p] = add2(d[p], z[p]);
    } else if (dy.p) {
      St::get(at(k, 1), it, dy, row, d);
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) d[p] = dn.p ? z[p] : two(0.0f);
    }
    it.put(dx, row, d);
    if (!block) continue;
    it.params(a.w, w);
    if (layer) it.clear(d);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      u[p] = mul2(u[p], two(ru));  // uhat
      sw[p] = fma2(d[p], u[p], sw[p]);
      d[p] = mul2(d[p], w[p]);
    }
    float s[2] = {dot(d, u), 0.0f};
    sa += (double)s[0];
    if (layer) {
      s[1] = total(d);
      row_sum<2>(s, buf, turn);
    } else {
      float one[1] = {s[0]};
      row_sum<1>(one, buf, turn);
      s[0] = one[0];
    }
    // alpha stands outside, so that dalpha's sum needs no division
    const float ar = alpha * ru;
    const float2 m = two(-s[0] * inv_h), mean = two(-s[1] * inv_h);
#pragma unroll
    for (int p = 0; p < P; ++p) d[p] = mul2(fma2(u[p], m, add2(d[p], mean)), two(ar));
    if (gated) {
      float2 hv[P], gv[P];
      read(3, sch, hv);
      read(4, scg, gv);
      // act' = s + g s (1 - s), or s (1 - s)
      if (a.act == GLR_ACT_SILU) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const float2 sg = sigmoid2(gv[p]), act = silu(gv[p], sg);
          const float2 slope = fma2(act, fma2(sg, two(-1.0f), two(1.0f)), sg);
          gv[p] = mul2(mul2(d[p], hv[p]), slope);
          d[p] = mul2(d[p], act);
        }
      } else {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const float2 sg = sigmoid2(gv[p]);
          const float2 slope = mul2(sg, fma2(sg, two(-1.0f), two(1.0f)));
          gv[p] = mul2(mul2(d[p], hv[p]), slope);
          d[p] = mul2(d[p], sg);
        }
      }
      it.put(dg, row, gv);
    }
    it.put(dh, row, d);
  }
  stage_wait<0>();
  const int64_t parts = gridDim.x, me = blockIdx.x;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (!it.on(j) || !DLR_IN((me * 2 + 1) * a.H + it.channel(j) + VEC - 1, parts * 2 * a.H))
      continue;
    float t[VEC];
    it.pick(j, sw, t);
    store<float, VEC == 8 ? 4 : VEC>(part + (me * 2) * a.H + it.channel(j), t);
    if constexpr (VEC == 8) store<float, 4>(part + (me * 2) * a.H + it.channel(j) + 4, t + 4);
    it.pick(j, sv, t);
    store<float, VEC == 8 ? 4 : VEC>(part + (me * 2 + 1) * a.H + it.channel(j), t);
    if constexpr (VEC == 8) store<float, 4>(part + (me * 2 + 1) * a.H + it.channel(j) + 4, t + 4);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sa += __shfl_xor_sync(0xffffffffu, sa, o);
  if ((threadIdx.x & 31) == 0) own[threadIdx.x >> 5] = sa;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int j = 1; j < (int)blockDim.x >> 5; ++j) sa += own[j];
    reinterpret_cast<double*>(part + parts * 2 * a.H)[me] = sa;
  }
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
    const double* each = reinterpret_cast<const double*>(part + (int64_t)parts * 2 * H);
    for (int k = lane; k < parts; k += 32) s += each[k];
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

// Blocks that go over the rows at most: a fixed number of threads, whatever the GPU, so that the
// workspace's size is the row's alone.
int most_parts(int R) { return 160 * std::max(1, 512 / R); }

template <typename T, int VEC, int NV, bool kKept, int kThreads, int kResident>
cudaError_t back_n(const glr_join_backward_args& a, cudaStream_t s) {
  const JoinArgs j{a.M, (int)a.H, (int)a.norm, (int)a.act, (float)a.eps, a.w, a.alpha, a.v};
  constexpr size_t staged = kStages * 5 * NV * VEC * sizeof(T);  // of a thread
  constexpr bool kDirect = staged * kThreads > kMostSmem;
  constexpr size_t per = kDirect ? 0 : staged;
  constexpr auto kernel = join_back<T, VEC, NV, kKept, kDirect, kThreads, kResident>;
  const int R = row_threads(a.H, VEC * NV);
  unsigned blocks = 0;
  cudaError_t e = row_blocks(a.M, R, kResident, per * R, &blocks);
  blocks = std::min<unsigned>(blocks, most_parts(R));
  if (e == cudaSuccess) e = max_smem_once<kernel>(per * kThreads);
  if (e != cudaSuccess) return e;
  float* part = static_cast<float*>(a.workspace);
  if (blocks > 0)
    kernel<<<blocks, R, per * R, s>>>(
        j, rows<const T>(a.dy.data, a.dy.stride_t), rows<const T>(a.dn.data, a.dn.stride_t),
        rows<const T>(a.x.data, a.x.stride_t), rows<const T>(a.h.data, a.h.stride_t),
        rows<const T>(a.g.data, a.g.stride_t),
        Ckpt{const_cast<uint8_t*>(a.hc), const_cast<uint8_t*>(a.hs), const_cast<uint8_t*>(a.gc),
             const_cast<uint8_t*>(a.gs)},
        rows<T>(a.dx.data, a.dx.stride_t), rows<T>(a.dh.data, a.dh.stride_t),
        rows<T>(a.dg.data, a.dg.stride_t), part);
  join_sums<<<(unsigned)(2 * ((a.H + 31) / 32) + 1), 1024, 0, s>>>(part, (int)blocks, (int)a.H,
                                                                    a.alpha, a.dw, a.dv, a.dalpha);
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
      wide(a.w, 0, 4) && wide(a.v, 0, 4) && wide(a.hc, 0, 1) && wide(a.gc, 0, 1) &&
      wide(a.workspace, 0, 1)) {
    if (a.H <= 16 * 128) return back_n<T, W, 16 / W, kKept, 128, 512>(a, s);
    if (a.H <= 16 * 512) return back_n<T, W, 16 / W, kKept, 512, 512>(a, s);
    return back_n<T, W, 16 / W, kKept, 1024, 1024>(a, s);
  }
  if (a.H <= 6 * 128) return back_n<T, 1, 6, kKept, 128, 640>(a, s);
  if (a.H <= 16 * 256) return back_n<T, 1, 16, kKept, 256, 512>(a, s);
  return back_n<T, 1, 16, kKept, 1024, 1024>(a, s);
}
template <typename T>
cudaError_t back_k(const glr_join_backward_args& a, cudaStream_t s) {
  return a.hc ? back_t<T, true>(a, s) : back_t<T, false>(a, s);
}

}  // namespace

size_t join_backward_workspace_bytes(int64_t H) {
  // the fewest threads that any layout above gives a row make the most parts
  return sizeof(float) * (size_t)most_parts(row_threads(H, 16)) * (2 * (size_t)H + 2);
}

cudaError_t launch_join_backward(const glr_join_backward_args& a, cudaStream_t s) {
  if (a.type == GLR_BF16) return back_k<__nv_bfloat16>(a, s);
  if (a.type == GLR_F16) return back_k<__half>(a, s);
  return back_k<float>(a, s);
}

}  // namespace glr
}  // namespace dlr
