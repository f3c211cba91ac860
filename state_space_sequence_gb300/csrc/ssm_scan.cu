// ssm_scan.cu -- the selective scan of include/ssm.h over a sequence, and one token of it.
//
// Per channel N states go through h = exp(s A) h + s x Bm and come out as o = sum Cm h: of the bytes
// a token's channel brings (x, dt, z, y: 8 in 16 bits) little, of arithmetic much: at N = 16 sixteen
// exponentials and 64 multiply-adds. So the kernel is built around its inner loop (ssm_common.cuh has
// the layout), which issues for two states a product for the exponent, two exponentials, one
// multiply-add for the state, one for the output and one product for the input. Everything else is
// done once a tile of 16 steps, by pieces of rows: the step's softplus, the skip and the gate.
#include "ssm_scan.cuh"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 22;

namespace ssm {
namespace {

constexpr int kWarps = 4;  // of a block; each works by itself

template <typename T>
struct scan_params {
  inputs<T> in;
  view<T> y;
  float *h_last, *states;
};

// A warp's part of shared memory: the tile's steps s, inputs s x, outputs, Bm and Cm.
template <typename T, int LN>
struct scan_tile {
  using S = shape<T, LN>;
  float s[kT][S::kCW], u[kT][S::kCW], o[kT][S::kCW];
  float Bm[kT][S::kNP], Cm[kT][S::kNP];
  float bias[S::kCW], D[S::kCW];
};

// MAP: only the state that each split but the last adds, and the sum of its steps.
template <typename T, int LN, bool MAP>
__global__ void __launch_bounds__(32 * kWarps) scan_kernel(scan_params<T> q) {
  using S = shape<T, LN>;
  constexpr bool kPrecise = sizeof(T) == 4;
  constexpr int VE = S::VE, VB = S::VB;
  extern __shared__ float4 smem[];
  const inputs<T>& in = q.in;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  scan_tile<T, LN>& m = reinterpret_cast<scan_tile<T, LN>*>(smem)[warp];

  const int64_t id = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  const int per_row = in.blocks * in.G, n_split = MAP ? in.splits - 1 : in.splits;
  if (id >= (int64_t)per_row * n_split * in.B) return;
  const int cb = (int)(id % per_row);
  const int split = (int)(id / per_row % n_split);
  const int64_t b = id / per_row / n_split;
  const int group = cb / in.blocks, first = (cb % in.blocks) * S::kCW;
  const int c0 = group * in.Hg + first, n_ch = min(S::kCW, in.Hg - first);
  // this lane's channels and states
  const int at = lane % LN, cl = lane / LN * kChannels, n0 = at * kStates;
  const int my_ch = n_ch - cl;

  const bool whole = n_ch == S::kCW && pieces(in.x, c0, VE * sizeof(T)) &&
                     pieces(in.dt, c0, VE * sizeof(T));
  const bool whole_z = in.z.p && n_ch == S::kCW && pieces(in.z, c0, VE * sizeof(T));
  const bool whole_y = n_ch == S::kCW && pieces(q.y, c0, VE * sizeof(T));
  const bool whole_b = in.N % VB == 0 && pieces(in.Bm, (int64_t)group * in.N, VB * sizeof(T)) &&
                       pieces(in.Cm, (int64_t)group * in.N, VB * sizeof(T));

  for (int c = lane; c < S::kCW; c += 32) {
    m.bias[c] = in.bias && c < n_ch ? in.bias[c0 + c] : 0.0f;
    m.D[c] = in.D && c < n_ch ? in.D[c0 + c] : 0.0f;
  }
  float2 rate[kChannels][2], h[kChannels][2];
  load_rates(rate, in.A, in.N, c0 + cl, my_ch, n0);
  const int64_t HN = (int64_t)in.H * in.N, ch = (int64_t)(c0 + cl) * in.N;
  if (MAP || (split == 0 && !in.h0))
    load_states(h, nullptr, in.N, 0, 0);
  else if (split == 0)
    load_states(h, in.h0 + b * HN + ch, in.N, my_ch, n0);
  else
    load_states(h, in.ends + (b * in.splits + split - 1) * HN + ch, in.N, my_ch, n0);
  float sum[kChannels] = {};
  bool cut = false;
  __syncwarp();

  const int t_first = split * in.per_split, t_end = min(in.tiles, t_first + in.per_split);
  for (int tile = t_first; tile < t_end; ++tile) {
    const int64_t t0 = (int64_t)tile * kT;
    const uint32_t mark = marks(in.reset, b, t0, in.L, lane);
    // the steps and what they bring in
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
      const int p = k * 32 + lane, t = p / S::kRow, c = p % S::kRow * VE;
      if (t >= kT) break;
      float xv[VE], dv[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) xv[i] = dv[i] = 0.0f;
      const bool there = t0 + t < in.L && c < n_ch;
      if (there) {
        words<T, VE> wx, wd;
        get_piece<T, VE>(wx, in.x.row(b, t0 + t) + c0 + c, n_ch - c, whole);
        get_piece<T, VE>(wd, in.dt.row(b, t0 + t) + c0 + c, n_ch - c, whole);
        wx.to(xv);
        wd.to(dv);
      }
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        float sig, s = dv[i] + m.bias[c + i];
        if (in.softplus) s = softplus(s, sig);
        // steps and channels that do not exist leave the state as it is
        s = there && c + i < n_ch ? s : 0.0f;
        dv[i] = s;
        xv[i] = there && c + i < n_ch ? s * xv[i] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        m.s[t][c + i] = dv[i];
        m.u[t][c + i] = xv[i];
      }
    }
#pragma unroll
    for (int k = 0; k < S::NB; ++k) {
      const int p = k * 32 + lane, t = p / S::kRowB, n = p % S::kRowB * VB;
      if (t >= kT) break;
      float bv[VB], cv[VB];
#pragma unroll
      for (int i = 0; i < VB; ++i) bv[i] = cv[i] = 0.0f;
      if (t0 + t < in.L && n < in.N) {
        words<T, VB> wb, wc;
        const int64_t o = (int64_t)group * in.N + n;
        get_piece<T, VB>(wb, in.Bm.row(b, t0 + t) + o, in.N - n, whole_b);
        wb.to(bv);
        if (!MAP) {
          get_piece<T, VB>(wc, in.Cm.row(b, t0 + t) + o, in.N - n, whole_b);
          wc.to(cv);
        }
      }
#pragma unroll
      for (int i = 0; i < VB; ++i) {
        m.Bm[t][n + i] = bv[i];
        if (!MAP) m.Cm[t][n + i] = cv[i];
      }
    }
    __syncwarp();
    if (!MAP && q.states)
      store_states(q.states + (b * in.tiles + tile) * HN + ch, h, in.N, my_ch, n0);

#pragma unroll 4
    for (int t = 0; t < kT; ++t) {
      const float4 s4 = *reinterpret_cast<const float4*>(&m.s[t][cl]);
      const float4 u4 = *reinterpret_cast<const float4*>(&m.u[t][cl]);
      const float4 b4 = *reinterpret_cast<const float4*>(&m.Bm[t][n0]);
      const float4 c4 = *reinterpret_cast<const float4*>(&m.Cm[t][n0]);
      const float s[4] = {s4.x, s4.y, s4.z, s4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
      const float2 bp[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
      const float2 cp[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
      if (mark >> t & 1) {
        load_states(h, nullptr, in.N, 0, 0);
        cut = true;
      }
      float o[kChannels];
#pragma unroll
      for (int i = 0; i < kChannels; ++i) {
        float2 acc = two(0.0f);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const decay<kPrecise> a(mul2(rate[i][p], two(s[i])));
          h[i][p] = a.of_plus(h[i][p], mul2(bp[p], two(u[i])));
          if (!MAP) acc = fma2(h[i][p], cp[p], acc);
        }
        o[i] = acc.x + acc.y;
        if (MAP) sum[i] += s[i];
      }
      if (!MAP) {
        sum4<1, LN>(o, at);
        put4<LN>(&m.o[t][cl], o, at);
      }
    }
    __syncwarp();
    // the skip, the gate, and out
#pragma unroll
    for (int k = 0; k < (MAP ? 0 : S::NV); ++k) {
      const int p = k * 32 + lane, t = p / S::kRow, c = p % S::kRow * VE;
      if (t >= kT) break;
      if (t0 + t >= in.L || c >= n_ch) continue;
      float o[VE], v[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) o[i] = m.o[t][c + i];
      words<T, VE> w;
      if (in.D) {
        get_piece<T, VE>(w, in.x.row(b, t0 + t) + c0 + c, n_ch - c, whole);
        w.to(v);
#pragma unroll
        for (int i = 0; i < VE; ++i) o[i] = fmaf(m.D[c + i], v[i], o[i]);
      }
      if (in.z.p) {
        get_piece<T, VE>(w, in.z.row(b, t0 + t) + c0 + c, n_ch - c, whole_z);
        w.to(v);
#pragma unroll
        for (int i = 0; i < VE; ++i) o[i] *= v[i] * glr::sigmoid(v[i]);
      }
      put_piece<T, VE>(q.y.row(b, t0 + t) + c0 + c, o, n_ch - c, whole_y);
    }
    __syncwarp();
  }
  if (MAP) {
    store_states(in.ends + (b * in.splits + split) * HN + ch, h, in.N, my_ch, n0);
    if (at == 0)
#pragma unroll
      for (int i = 0; i < kChannels; ++i)
        if (i < my_ch)
          in.sums[(b * in.splits + split) * in.H + c0 + cl + i] =
              cut ? __int_as_float(0x7fffffff) : sum[i];
  } else if (split == in.splits - 1 && q.h_last) {
    store_states(q.h_last + b * HN + ch, h, in.N, my_ch, n0);
  }
}

template <typename T, int LN>
cudaError_t run_scan(scan_params<T> q, cudaStream_t s) {
  using S = shape<T, LN>;
  q.in.blocks = (q.in.Hg + S::kCW - 1) / S::kCW;
  const int64_t units = (int64_t)q.in.blocks * q.in.G * q.in.B;
  constexpr size_t bytes = sizeof(scan_tile<T, LN>) * kWarps;
  auto grid = [](int64_t warps) { return (unsigned)((warps + kWarps - 1) / kWarps); };
  cudaError_t e;
  if (q.in.splits > 1) {
    if ((e = max_smem_once<scan_kernel<T, LN, true>>(bytes)) != cudaSuccess) return e;
    scan_kernel<T, LN, true><<<grid(units * (q.in.splits - 1)), 32 * kWarps, bytes, s>>>(q);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int64_t HN = (int64_t)q.in.H * q.in.N;
    join_splits<false><<<(unsigned)((q.in.B * HN + 127) / 128), 128, 0, s>>>(
        q.in.A, q.in.h0, q.in.ends, q.in.sums, q.in.B, q.in.splits, HN, q.in.N);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = max_smem_once<scan_kernel<T, LN, false>>(bytes)) != cudaSuccess) return e;
  scan_kernel<T, LN, false><<<grid(units * q.in.splits), 32 * kWarps, bytes, s>>>(q);
  return cudaGetLastError();
}

template <typename T>
cudaError_t scan_of(const ssm_scan_args& a, cudaStream_t s) {
  scan_params<T> q{make_inputs<T>(a), out_view<T>(a.y), a.h_last, a.states};
  q.in.ends = static_cast<float*>(a.workspace);
  q.in.sums = q.in.ends + a.B * q.in.splits * a.H * a.N;
  switch (lanes_for(a.N)) {
    case 1: return run_scan<T, 1>(q, s);
    case 2: return run_scan<T, 2>(q, s);
    case 4: return run_scan<T, 4>(q, s);
    case 8: return run_scan<T, 8>(q, s);
    default: return run_scan<T, 16>(q, s);
  }
}

// ---- one token ----------------------------------------------------------------------------

template <typename T>
struct step_params {
  int64_t B;
  int H, Hg, N, G, softplus;
  view<const T> x, dt, z, Bm, Cm;
  const float *A, *D, *bias, *h;
  const uint8_t* reset;
  view<T> y;
  float* h_out;
};

// LN lanes to a channel, 4 states to a lane; LN a power of two. The states go through memory once
// each way and are all there is to it: 134 MB at 256 x 4096 x 16.
template <typename T, int LN, bool QUADS>
__global__ void __launch_bounds__(256) step_kernel(step_params<T> q) {
  const int lane = threadIdx.x & 31, at = lane % LN, n0 = at * kStates;
  const int64_t unit = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LN;
  const bool there = unit < (int64_t)q.B * q.H;
  const int64_t b = there ? unit / q.H : 0;
  const int c = there ? (int)(unit - b * q.H) : 0, group = c / q.Hg;
  float sig, s = to_f(q.dt.row(b, 0)[c]) + (q.bias ? q.bias[c] : 0.0f);
  if (q.softplus) s = softplus(s, sig);
  const float x = to_f(q.x.row(b, 0)[c]), u = s * x;
  const bool fresh = q.reset && q.reset[b];
  float A[4], h[4], Bm[4], Cm[4];
  const int64_t o = (b * q.H + c) * q.N + n0;
  const T* pb = q.Bm.row(b, 0) + (int64_t)group * q.N + n0;
  const T* pc = q.Cm.row(b, 0) + (int64_t)group * q.N + n0;
  if (QUADS) {
    load_floats<4>(A, q.A + (int64_t)c * q.N + n0);
    load_floats<4>(h, q.h + o);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      A[j] = n0 + j < q.N ? q.A[(int64_t)c * q.N + n0 + j] : 0.0f;
      h[j] = n0 + j < q.N ? q.h[o + j] : 0.0f;
    }
  }
  float acc = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    Bm[j] = QUADS || n0 + j < q.N ? to_f(pb[j]) : 0.0f;
    Cm[j] = QUADS || n0 + j < q.N ? to_f(pc[j]) : 0.0f;
    const float a = expf(min_nan(s * A[j], 87.0f));
    h[j] = fresh ? u * Bm[j] : fmaf(a, h[j], u * Bm[j]);
    acc = fmaf(h[j], Cm[j], acc);
  }
#pragma unroll
  for (int d = 1; d < LN; d *= 2) acc += __shfl_xor_sync(0xffffffffu, acc, d);
  if (!there) return;
  if (QUADS) {
    store_floats<4>(q.h_out + o, h);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n0 + j < q.N) q.h_out[o + j] = h[j];
  }
  if (at) return;
  if (q.D) acc = fmaf(q.D[c], x, acc);
  if (q.z.p) {
    const float z = to_f(q.z.row(b, 0)[c]);
    acc *= z * glr::sigmoid(z);
  }
  q.y.row(b, 0)[c] = from_f<T>(acc);
}

template <typename T, int LN>
cudaError_t run_step(const step_params<T>& q, cudaStream_t s) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(q.A) | reinterpret_cast<uintptr_t>(q.h) |
                        reinterpret_cast<uintptr_t>(q.h_out);
  const unsigned grid = (unsigned)((q.B * q.H * LN + 255) / 256);
  if (q.N == 4 * LN && (all & 15) == 0)
    step_kernel<T, LN, true><<<grid, 256, 0, s>>>(q);
  else
    step_kernel<T, LN, false><<<grid, 256, 0, s>>>(q);
  return cudaGetLastError();
}

template <typename T>
cudaError_t step_of(const ssm_step_args& a, cudaStream_t s) {
  auto in = [](const glr_view& v) {
    return view<const T>{static_cast<const T*>(v.data), v.stride_b, 0};
  };
  const step_params<T> q{a.B, (int)a.H, (int)(a.H / a.G), (int)a.N, (int)a.G, (int)a.softplus,
                         in(a.x), in(a.dt), in(a.z), in(a.Bm), in(a.Cm), a.A, a.D, a.dt_bias,
                         a.h, a.reset, out_view<T>(a.y), a.h_out};
  switch (lanes_for(a.N)) {
    case 1: return run_step<T, 1>(q, s);
    case 2: return run_step<T, 2>(q, s);
    case 4: return run_step<T, 4>(q, s);
    case 8: return run_step<T, 8>(q, s);
    default: return run_step<T, 16>(q, s);
  }
}

}  // namespace

size_t scan_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t N, int64_t G) {
  return (size_t)map_floats(B, H, N, splits_for(B, L, H, N, G)) * 4;
}

cudaError_t launch_scan(const ssm_scan_args& a, cudaStream_t s) {
  if (a.type == GLR_F32) return scan_of<float>(a, s);
  return a.type == GLR_BF16 ? scan_of<__nv_bfloat16>(a, s) : scan_of<__half>(a, s);
}

cudaError_t launch_step(const ssm_step_args& a, cudaStream_t s) {
  if (a.type == GLR_F32) return step_of<float>(a, s);
  return a.type == GLR_BF16 ? step_of<__nv_bfloat16>(a, s) : step_of<__half>(a, s);
}

}  // namespace ssm
}  // namespace dlr
