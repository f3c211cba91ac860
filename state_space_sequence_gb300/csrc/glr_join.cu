// glr_join.cu -- the end of a recurrent block fused with the norm that begins the next one
// (include/glr.h, glr_join): u = h act(g), y = x + alpha w norm(u), n = v norm(y), with h and g
// kept in 8 bits on the way where the caller wants them for the gradients.
//
// Bound by memory: three rows in and two out. 32768 x 2048 bfloat16 takes 105 us (6.4 TB/s, 94% of
// a plain copy's bandwidth); with both checkpoints 65536 x 1024 takes 136 us (88%); 8191 x 515
// float32, single channels to an access, 26 us (47%: 6 channels to a thread do not hide its row's
// sums). glr_join.cuh has the layout.
#include "glr_join.cuh"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 17;

namespace glr {
namespace {

template <typename T, int VEC, int NV, bool kDirect, int kThreads, int kResident>
__global__ void __launch_bounds__(kThreads, kResident / kThreads)
join_kernel(JoinArgs a, Rows<const T> x, Rows<const T> h, Rows<const T> g, Rows<T> y, Rows<T> n,
            Ckpt ck) {
  constexpr int P = VEC * NV / 2;
  using St = Staged<T, VEC, NV, kDirect>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float buf[64 * kSums];
  // [kStages][x h g][items]
  typename St::item* const sm = reinterpret_cast<typename St::item*>(smem);
  const Items<VEC, NV> it{a.H, (int)blockDim.x};
  const int per = St::items();
  const bool layer = a.norm == GLR_NORM_LAYER;
  const int groups = (a.H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP;
  const float alpha = h.p ? *a.alpha : 0.0f, inv_h = 1.0f / (float)a.H;
  int64_t row = blockIdx.x;
  auto fetch = [&](int64_t r, int k) {
    if (r < a.M) {
      St::fetch_row(sm + (k * 3) * per, it, x.at(r, 0));
      if (h.p) St::fetch_row(sm + (k * 3 + 1) * per, it, h.at(r, 0));
      if (g.p) St::fetch_row(sm + (k * 3 + 2) * per, it, g.at(r, 0));
    }
    stage_end();
  };
  fetch(row, 0);
  int turn = 0;
  for (int k = 0; row < a.M; row += gridDim.x, k ^= 1) {
    fetch(row + gridDim.x, k ^ 1);
    stage_wait<1>();
    float2 z[P], u[P];
    if (h.p) {
      St::get(sm + (k * 3 + 1) * per, it, h, row, u);
      auto code = [&](int array, const Rows<const T>& r, uint8_t* codes, uint8_t* scales) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = it.channel(j);
          const bool on = it.on(j) && DLR_IN(row * a.H + c + VEC - 1, a.M * a.H);
          keep<T, VEC>(St::one(sm + (k * 3 + array) * per, j, r.at(row, c), on), on,
                       codes + row * a.H + c, scales + row * groups + c / GLR_CKPT_GROUP);
        }
      };
      if (ck.hc) code(1, h, ck.hc, ck.hs);
      if (g.p) {
        float2 gv[P];
        St::get(sm + (k * 3 + 2) * per, it, g, row, gv);
        apply_gate(a.act, u, gv);
        if (ck.gc) code(2, g, ck.gc, ck.gs);
      }
      const float ru = centre<VEC, NV>(it, u, layer, inv_h, a.eps, buf, turn);
      float2 w[P];
      it.params(a.w, w);
      St::get(sm + (k * 3) * per, it, x, row, z);
      const float2 c = two(alpha * ru);
#pragma unroll
      for (int p = 0; p < P; ++p) z[p] = fma2(mul2(w[p], u[p]), c, z[p]);
      it.put(y, row, z);
    } else {
      St::get(sm + (k * 3) * per, it, x, row, z);
    }
    if (n.p) {
      const float2 ry = two(centre<VEC, NV>(it, z, layer, inv_h, a.eps, buf, turn));
      float2 v[P];
      it.params(a.v, v);
#pragma unroll
      for (int p = 0; p < P; ++p) v[p] = mul2(v[p], mul2(z[p], ry));
      it.put(n, row, v);
    }
  }
  stage_wait<0>();
}


// kThreads: the block's most threads; kResident: threads that an SM holds.
template <typename T, int VEC, int NV, int kThreads, int kResident>
cudaError_t join_n(const glr_join_args& a, cudaStream_t s) {
  const JoinArgs j{a.M, (int)a.H, (int)a.norm, (int)a.act, (float)a.eps, a.w, a.alpha, a.v};
  constexpr size_t staged = kStages * 3 * NV * VEC * sizeof(T);  // of a thread
  constexpr bool kDirect = staged * kThreads > kMostSmem;
  constexpr size_t per = kDirect ? 0 : staged;
  constexpr auto kernel = join_kernel<T, VEC, NV, kDirect, kThreads, kResident>;
  const int R = row_threads(a.H, VEC * NV);
  unsigned blocks;
  cudaError_t e = row_blocks(a.M, R, kResident, per * R, &blocks);
  if (e == cudaSuccess) e = max_smem_once<kernel>(per * kThreads);
  if (e != cudaSuccess) return e;
  kernel<<<blocks, R, per * R, s>>>(
      j, rows<const T>(a.x.data, a.x.stride_t), rows<const T>(a.h.data, a.h.stride_t),
      rows<const T>(a.g.data, a.g.stride_t), rows<T>(a.y.data, a.y.stride_t),
      rows<T>(a.n.data, a.n.stride_t), Ckpt{a.hc, a.hs, a.gc, a.gs});
  return cudaGetLastError();
}
// 16 channels to a thread while the row's threads then fill an SM evenly; single channels (rows
// that allow no 16-byte access) 6 to a thread while the row is short, so that more threads share
// it.
template <typename T>
cudaError_t join_t(const glr_join_args& a, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  const int64_t z = sizeof(T);
  if (a.H % W == 0 && wide(a.x.data, a.x.stride_t, z) && wide(a.h.data, a.h.stride_t, z) &&
      wide(a.g.data, a.g.stride_t, z) && wide(a.y.data, a.y.stride_t, z) &&
      wide(a.n.data, a.n.stride_t, z) && wide(a.w, 0, 4) && wide(a.v, 0, 4) && wide(a.hc, 0, 1) &&
      wide(a.gc, 0, 1)) {
    if (a.H <= 16 * 128) return join_n<T, W, 16 / W, 128, 640>(a, s);
    if (a.H <= 16 * 512) return join_n<T, W, 16 / W, 512, 512>(a, s);
    return join_n<T, W, 16 / W, 1024, 1024>(a, s);
  }
  if (a.H <= 6 * 128) return join_n<T, 1, 6, 128, 768>(a, s);
  if (a.H <= 16 * 256) return join_n<T, 1, 16, 256, 512>(a, s);
  return join_n<T, 1, 16, 1024, 1024>(a, s);
}

}  // namespace

cudaError_t launch_join(const glr_join_args& a, cudaStream_t s) {
  if (a.type == GLR_BF16) return join_t<__nv_bfloat16>(a, s);
  if (a.type == GLR_F16) return join_t<__half>(a, s);
  return join_t<float>(a, s);
}

}  // namespace glr
}  // namespace dlr
