// ssm_scan_back.cu -- the gradients of the selective scan of include/ssm.h.
//
// Backwards in time with the gradient of the state carried along: G_t = g_t Cm_t + a_{t+1} G_{t+1}.
// Sums over the states (q, e, o) go over a channel's lanes, sums over the channels (dBm, dCm) over a
// warp's channels, then the block's warps, then the blocks of a group (through the workspace, added
// up by a second kernel); sums over time (dA, dD, ddt_bias) stay with the warp, one partial sum for
// each batch entry and split.
//
// The states are not kept but every 16 steps. A tile's second half needs them first: a run over the
// first half finds where it begins; then each half is run forwards, its states held in registers
// (8 steps x 16 numbers a lane), dCm and o formed on the way, and backwards. In all 2.5 exponentials
// a state and step instead of one, for an eighth of the memory that all states would take.
#include "ssm_scan.cuh"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 23;

namespace ssm {
namespace {

constexpr int kWarps = 4;   // of a block at most; they meet once a tile
constexpr int kHalf = kT / 2;

template <typename T>
struct back_params {
  inputs<T> in;
  view<const T> dy;
  view<T> dx, ddt, dz, dBm, dCm;
  const float *states, *dh_last;
  float *dA, *dD, *ddt_bias, *dh0;
  // parts: dBm and dCm [G, blocks, B, L, 2, NP] (NP = 4 LN), dA [B splits, H, N], dD and ddt_bias
  // [2, B splits, H]
  float *part_bc, *part_A, *part_c;
};

template <typename T, int LN>
struct back_tile {
  using S = shape<T, LN>;
  float s[kT][S::kCW], u[kT][S::kCW], g[kT][S::kCW];
  float q[kT][S::kCW], e[kT][S::kCW], o[kT][S::kCW];
  float Bm[kT][S::kNP], Cm[kT][S::kNP];
  float dBC[2][kT][2][S::kNP];  // two tiles in turn
  float bias[S::kCW], D[S::kCW];
};

template <bool PRECISE>
__device__ __forceinline__ void advance(float2 (&h)[kChannels][2],
                                        const float2 (&rate)[kChannels][2], const float (&s)[4],
                                        const float (&u)[4], const float2 (&bp)[2]) {
#pragma unroll
  for (int i = 0; i < kChannels; ++i)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const decay<PRECISE> a(mul2(rate[i][p], two(s[i])));
      h[i][p] = a.of_plus(h[i][p], mul2(bp[p], two(u[i])));
    }
}

__device__ __forceinline__ void clear(float2 (&h)[kChannels][2]) {
#pragma unroll
  for (int i = 0; i < kChannels; ++i) h[i][0] = h[i][1] = two(0.0f);
}

__device__ __forceinline__ void get4(float (&v)[4], const float* p) { load_floats<4>(v, p); }
__device__ __forceinline__ void get4(float2 (&v)[2], const float* p) {
  const float4 t = *reinterpret_cast<const float4*>(p);
  v[0] = make_float2(t.x, t.y);
  v[1] = make_float2(t.z, t.w);
}

// MAP: only the gradient that each split but the first sends on, and the sum of its steps.
template <typename T, int LN, bool MAP>
__global__ void __launch_bounds__(32 * kWarps) back_kernel(back_params<T> q) {
  using S = shape<T, LN>;
  constexpr bool kPrecise = sizeof(T) == 4;
  constexpr int VE = S::VE, VB = S::VB, CL = 32 / LN;
  extern __shared__ float4 smem[];
  const inputs<T>& in = q.in;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  back_tile<T, LN>* all = reinterpret_cast<back_tile<T, LN>*>(smem);
  back_tile<T, LN>& m = all[warp];

  // a block: `warps` neighbouring warps of one group, split and batch entry
  const int per_row = in.blocks * in.G, n_split = MAP ? in.splits - 1 : in.splits;
  const int cb = (int)(blockIdx.x % per_row);
  const int split = (int)(blockIdx.x / per_row % n_split) + (MAP ? 1 : 0);
  const int64_t b = blockIdx.x / per_row / n_split;
  const int group = cb / in.blocks, block = cb % in.blocks;
  const int first = (block * warps + warp) * S::kCW;
  const int c0 = group * in.Hg + first, n_ch = max(0, min(S::kCW, in.Hg - first));
  const int at = lane % LN, cg = lane / LN, cl = cg * kChannels, n0 = at * kStates;
  const int my_ch = n_ch - cl;

  const bool full = n_ch == S::kCW;
  const bool whole = full && pieces(in.x, c0, VE * sizeof(T)) &&
                     pieces(in.dt, c0, VE * sizeof(T)) && pieces(q.dy, c0, VE * sizeof(T));
  const bool whole_z = in.z.p && full && pieces(in.z, c0, VE * sizeof(T));
  const bool whole_o = full && pieces(q.dx, c0, VE * sizeof(T)) &&
                       pieces(q.ddt, c0, VE * sizeof(T)) &&
                       (!in.z.p || pieces(q.dz, c0, VE * sizeof(T)));
  const bool whole_b = in.N % VB == 0 && pieces(in.Bm, (int64_t)group * in.N, VB * sizeof(T)) &&
                       pieces(in.Cm, (int64_t)group * in.N, VB * sizeof(T));

  for (int c = lane; c < S::kCW; c += 32) {
    m.bias[c] = in.bias && c < n_ch ? in.bias[c0 + c] : 0.0f;
    m.D[c] = in.D && c < n_ch ? in.D[c0 + c] : 0.0f;
  }
  float2 rate[kChannels][2], carry[kChannels][2], dA[kChannels][2];
  load_rates(rate, in.A, in.N, c0 + cl, my_ch, n0);
  clear(dA);
  const int64_t HN = (int64_t)in.H * in.N, ch = (int64_t)(c0 + cl) * in.N;
  const int64_t row_map = b * in.splits + split;
  if (MAP)
    clear(carry);
  else if (split == in.splits - 1)
    load_states(carry, q.dh_last ? q.dh_last + b * HN + ch : nullptr, in.N, my_ch, n0);
  else
    load_states(carry, in.ends + (row_map + 1) * HN + ch, in.N, my_ch, n0);
  float sum[kChannels] = {};
  float sum_c[(S::kCW + 31) / 32][2] = {};  // of channel lane + 32 k: ddt and g x
  bool cut = false;
  __syncwarp();

  const int t_first = split * in.per_split, t_end = min(in.tiles, t_first + in.per_split);
  for (int tile = t_end - 1; tile >= t_first; --tile) {
    const int64_t t0 = (int64_t)tile * kT;
    const uint32_t mark = marks(in.reset, b, t0, in.L, lane);
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
      const int p = k * 32 + lane, t = p / S::kRow, c = p % S::kRow * VE;
      if (t >= kT) break;
      float xv[VE], dv[VE], gv[VE], zv[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) xv[i] = dv[i] = gv[i] = zv[i] = 0.0f;
      const bool there = t0 + t < in.L && c < n_ch;
      if (there) {
        words<T, VE> w;
        get_piece<T, VE>(w, in.x.row(b, t0 + t) + c0 + c, n_ch - c, whole);
        w.to(xv);
        get_piece<T, VE>(w, in.dt.row(b, t0 + t) + c0 + c, n_ch - c, whole);
        w.to(dv);
        get_piece<T, VE>(w, q.dy.row(b, t0 + t) + c0 + c, n_ch - c, whole);
        w.to(gv);
        if (in.z.p) {
          get_piece<T, VE>(w, in.z.row(b, t0 + t) + c0 + c, n_ch - c, whole_z);
          w.to(zv);
        }
      }
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const bool ok = there && c + i < n_ch;
        float sig, s = dv[i] + m.bias[c + i];
        if (in.softplus) s = softplus(s, sig);
        m.s[t][c + i] = ok ? s : 0.0f;
        m.u[t][c + i] = ok ? s * xv[i] : 0.0f;
        const float gate = in.z.p ? zv[i] * glr::sigmoid(zv[i]) : 1.0f;
        m.g[t][c + i] = ok ? gv[i] * gate : 0.0f;
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
        words<T, VB> w;
        const int64_t o = (int64_t)group * in.N + n;
        get_piece<T, VB>(w, in.Bm.row(b, t0 + t) + o, in.N - n, whole_b);
        w.to(bv);
        get_piece<T, VB>(w, in.Cm.row(b, t0 + t) + o, in.N - n, whole_b);
        w.to(cv);
      }
#pragma unroll
      for (int i = 0; i < VB; ++i) {
        m.Bm[t][n + i] = bv[i];
        m.Cm[t][n + i] = cv[i];
      }
    }
    __syncwarp();

    if constexpr (MAP) {
#pragma unroll 4
      for (int t = kT - 1; t >= 0; --t) {
        float s[4], g[4];
        float2 cp[2];
        get4(s, &m.s[t][cl]);
        get4(g, &m.g[t][cl]);
        get4(cp, &m.Cm[t][n0]);
#pragma unroll
        for (int i = 0; i < kChannels; ++i) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const decay<kPrecise> a(mul2(rate[i][p], two(s[i])));
            carry[i][p] = a.of(fma2(cp[p], two(g[i]), carry[i][p]));
          }
          sum[i] += s[i];
        }
        if (mark >> t & 1) {
          clear(carry);
          cut = true;
        }
      }
      __syncwarp();
    } else {
      const float* start = q.states + (b * in.tiles + tile) * HN + ch;
      float (*dBC)[2][S::kNP] = m.dBC[tile & 1];
#pragma unroll 1
      for (int half = 1; half >= 0; --half) {
        float2 h[kChannels][2], hist[kHalf][kChannels][2];
        load_states(h, start, in.N, my_ch, n0);
        if (half)
#pragma unroll 2
          for (int t = 0; t < kHalf; ++t) {
            float s[4], u[4];
            float2 bp[2];
            get4(s, &m.s[t][cl]);
            get4(u, &m.u[t][cl]);
            get4(bp, &m.Bm[t][n0]);
            if (mark >> t & 1) clear(h);
            advance<kPrecise>(h, rate, s, u, bp);
          }
        const int first_t = half * kHalf;
#pragma unroll
        for (int k = 0; k < kHalf; ++k) {
          const int t = first_t + k;
          float s[4], u[4], g[4];
          float2 bp[2], cp[2];
          get4(s, &m.s[t][cl]);
          get4(u, &m.u[t][cl]);
          get4(g, &m.g[t][cl]);
          get4(bp, &m.Bm[t][n0]);
          get4(cp, &m.Cm[t][n0]);
          if (mark >> t & 1) clear(h);
#pragma unroll
          for (int i = 0; i < kChannels; ++i) hist[k][i][0] = h[i][0], hist[k][i][1] = h[i][1];
          advance<kPrecise>(h, rate, s, u, bp);
          float2 dc[2] = {two(0.0f), two(0.0f)};
#pragma unroll
          for (int i = 0; i < kChannels; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p) dc[p] = fma2(h[i][p], two(g[i]), dc[p]);
          float v[4] = {dc[0].x, dc[0].y, dc[1].x, dc[1].y};
          sum4<LN, CL>(v, cg);
          put4<CL>(&dBC[t][1][n0], v, cg);
          if (in.z.p) {
            float o[4];
#pragma unroll
            for (int i = 0; i < kChannels; ++i) {
              const float2 acc = fma2(h[i][1], cp[1], mul2(h[i][0], cp[0]));
              o[i] = acc.x + acc.y;
            }
            sum4<1, LN>(o, at);
            put4<LN>(&m.o[t][cl], o, at);
          }
        }
#pragma unroll
        for (int k = kHalf - 1; k >= 0; --k) {
          const int t = first_t + k;
          float s[4], u[4], g[4], qv[4], ev[4];
          float2 bp[2], cp[2], db[2] = {two(0.0f), two(0.0f)};
          get4(s, &m.s[t][cl]);
          get4(u, &m.u[t][cl]);
          get4(g, &m.g[t][cl]);
          get4(bp, &m.Bm[t][n0]);
          get4(cp, &m.Cm[t][n0]);
          const bool stop = mark >> t & 1;
#pragma unroll
          for (int i = 0; i < kChannels; ++i) {
            float2 qs = two(0.0f), es = two(0.0f);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const float2 G = fma2(cp[p], two(g[i]), carry[i][p]);
              qs = fma2(G, bp[p], qs);
              db[p] = fma2(G, two(u[i]), db[p]);
              const decay<kPrecise> a(mul2(rate[i][p], two(s[i])));
              float2 c = a.of(G);
              if (stop) c = two(0.0f);
              carry[i][p] = c;
              const float2 r = mul2(c, hist[k][i][p]);
              es = fma2(r, rate[i][p], es);
              dA[i][p] = fma2(r, two(s[i]), dA[i][p]);
            }
            qv[i] = qs.x + qs.y;
            ev[i] = es.x + es.y;
          }
          sum4<1, LN>(qv, at);
          put4<LN>(&m.q[t][cl], qv, at);
          sum4<1, LN>(ev, at);
          put4<LN>(&m.e[t][cl], ev, at);
          float v[4] = {db[0].x, db[0].y, db[1].x, db[1].y};
          sum4<LN, CL>(v, cg);
          put4<CL>(&dBC[t][0][n0], v, cg);
        }
      }
      __syncwarp();
      // what the channels' gradients take besides, by pieces of rows
#pragma unroll
      for (int k = 0; k < S::NV; ++k) {
        const int p = k * 32 + lane, t = p / S::kRow, c = p % S::kRow * VE;
        if (t >= kT) break;
        const bool there = t0 + t < in.L && c < n_ch;
        if (there) {
          float xv[VE], dv[VE], dxv[VE];
          words<T, VE> w;
          get_piece<T, VE>(w, in.x.row(b, t0 + t) + c0 + c, n_ch - c, whole);
          w.to(xv);
          get_piece<T, VE>(w, in.dt.row(b, t0 + t) + c0 + c, n_ch - c, whole);
          w.to(dv);
#pragma unroll
          for (int i = 0; i < VE; ++i) {
            const float qv = m.q[t][c + i], g = m.g[t][c + i];
            float sig = 1.0f, s = dv[i] + m.bias[c + i];
            if (in.softplus) s = softplus(s, sig);
            // e was summed with the rates in powers of two
            const float slope = m.e[t][c + i] * (1.0f / kLog2e);
            dxv[i] = fmaf(s, qv, m.D[c + i] * g);
            dv[i] = fmaf(xv[i], qv, slope) * sig;
            m.q[t][c + i] = c + i < n_ch ? dv[i] : 0.0f;
            m.e[t][c + i] = c + i < n_ch ? g * xv[i] : 0.0f;
          }
          put_piece<T, VE>(q.dx.row(b, t0 + t) + c0 + c, dxv, n_ch - c, whole_o);
          put_piece<T, VE>(q.ddt.row(b, t0 + t) + c0 + c, dv, n_ch - c, whole_o);
          if (in.z.p) {
            float zv[VE], yv[VE];
            get_piece<T, VE>(w, in.z.row(b, t0 + t) + c0 + c, n_ch - c, whole_z);
            w.to(zv);
            get_piece<T, VE>(w, q.dy.row(b, t0 + t) + c0 + c, n_ch - c, whole);
            w.to(yv);
#pragma unroll
            for (int i = 0; i < VE; ++i) {
              const float sig = glr::sigmoid(zv[i]);
              const float o = fmaf(m.D[c + i], xv[i], m.o[t][c + i]);
              yv[i] *= o * fmaf(zv[i] * sig, 1.0f - sig, sig);
            }
            put_piece<T, VE>(q.dz.row(b, t0 + t) + c0 + c, yv, n_ch - c, whole_o);
          }
        } else {
#pragma unroll
          for (int i = 0; i < VE; ++i) m.q[t][c + i] = m.e[t][c + i] = 0.0f;
        }
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < (S::kCW + 31) / 32; ++k) {
        const int c = lane + 32 * k;
        if (c < S::kCW)
          for (int t = 0; t < kT; ++t) {
            sum_c[k][0] += m.q[t][c];
            sum_c[k][1] += m.e[t][c];
          }
      }
      // the warps' sums over their channels
      __syncthreads();
      const int64_t pitch = 2 * S::kNP;
      float* part = q.part_bc + (((int64_t)group * in.blocks + block) * in.B + b) * in.L * pitch;
      for (int i = threadIdx.x; i < kT * pitch; i += blockDim.x) {
        const int t = i / pitch;
        float v = 0.0f;
        for (int w = 0; w < warps; ++w) v += (&all[w].dBC[tile & 1][0][0][0])[i];
        if (t0 + t < in.L) part[t0 * pitch + i] = v;
      }
    }
  }
  if constexpr (MAP) {
    store_states(in.ends + row_map * HN + ch, carry, in.N, my_ch, n0);
    if (at == 0)
#pragma unroll
      for (int i = 0; i < kChannels; ++i)
        if (i < my_ch)
          in.sums[row_map * in.H + c0 + cl + i] = cut ? __int_as_float(0x7fffffff) : sum[i];
  } else {
    store_states(q.part_A + row_map * HN + ch, dA, in.N, my_ch, n0);
#pragma unroll
    for (int k = 0; k < (S::kCW + 31) / 32; ++k) {
      const int c = lane + 32 * k;
      if (c < n_ch) {
        q.part_c[row_map * in.H + c0 + c] = sum_c[k][0];
        q.part_c[((int64_t)in.B * in.splits + row_map) * in.H + c0 + c] = sum_c[k][1];
      }
    }
    if (split == 0 && q.dh0) store_states(q.dh0 + b * HN + ch, carry, in.N, my_ch, n0);
  }
}

// dBm and dCm from the blocks' parts: a thread for a state of a group and step.
template <typename T>
__global__ void sum_maps(const float* part, view<T> dBm, view<T> dCm, int64_t B, int64_t L, int G,
                         int N, int NP, int blocks) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, pitch = 2 * NP;
  const int64_t rows = B * L;
  if (i >= rows * G * pitch) return;
  const int n = (int)(i % pitch);
  const int64_t row = i / pitch % rows;
  const int g = (int)(i / pitch / rows);
  if (n % NP >= N) return;
  float v = 0.0f;
  for (int k = 0; k < blocks; ++k) v += part[(((int64_t)g * blocks + k) * rows + row) * pitch + n];
  const int64_t b = row / L, t = row - b * L;
  (n < NP ? dBm : dCm).row(b, t)[(int64_t)g * N + n % NP] = from_f<T>(v);
}

// The parameters' gradients from the parts of `rows` batch entries and splits.
__global__ void sum_params(const float* part_A, const float* part_c, float* dA, float* dbias,
                           float* dD, int64_t rows, int64_t H, int64_t HN) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const float* p;
  float* to;
  int64_t k, pitch;
  if (i < HN)
    p = part_A, to = dA, k = i, pitch = HN;
  else if (i < HN + H)
    p = part_c, to = dbias, k = i - HN, pitch = H;
  else if (i < HN + 2 * H)
    p = part_c + rows * H, to = dD, k = i - HN - H, pitch = H;
  else
    return;
  if (!to) return;
  float v = 0.0f;
#pragma unroll 4
  for (int64_t r = 0; r < rows; ++r) v += p[r * pitch + k];
  to[k] = v;
}

struct back_plan {
  int64_t warps, blocks, NP, splits;  // warps of a block, blocks of a group
  int64_t bc, A, c, map;              // floats of the parts and the splits' maps
};
back_plan plan(int64_t B, int64_t L, int64_t H, int64_t N, int64_t G) {
  back_plan p;
  const int64_t ln = lanes_for(N), cw = 128 / ln, units = (H / G + cw - 1) / cw;
  p.warps = std::min<int64_t>(kWarps, units);
  p.blocks = (units + p.warps - 1) / p.warps;
  p.NP = 4 * ln;
  const int64_t want = splits_for(B, L, H, N, G), tiles = (L + kT - 1) / kT;
  const int64_t per = (tiles + want - 1) / want;
  p.splits = (tiles + per - 1) / per;
  p.bc = G * p.blocks * B * L * 2 * p.NP;
  p.A = B * p.splits * H * N;
  p.c = 2 * B * p.splits * H;
  p.map = map_floats(B, H, N, p.splits);
  return p;
}

template <typename T, int LN>
cudaError_t run_back(back_params<T> q, const back_plan& p, cudaStream_t s) {
  q.in.blocks = (int)p.blocks;
  const int threads = 32 * (int)p.warps;
  const size_t bytes = sizeof(back_tile<T, LN>) * (size_t)p.warps;
  const int64_t units = p.blocks * q.in.G * q.in.B;
  const int64_t HN = (int64_t)q.in.H * q.in.N;
  cudaError_t e;
  if (q.in.splits > 1) {
    if ((e = max_smem_once<back_kernel<T, LN, true>>(sizeof(back_tile<T, LN>) * kWarps)) !=
        cudaSuccess)
      return e;
    back_kernel<T, LN, true><<<(unsigned)(units * (q.in.splits - 1)), threads, bytes, s>>>(q);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    join_splits<true><<<(unsigned)((q.in.B * HN + 127) / 128), 128, 0, s>>>(
        q.in.A, q.dh_last, q.in.ends, q.in.sums, q.in.B, q.in.splits, HN, q.in.N);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = max_smem_once<back_kernel<T, LN, false>>(sizeof(back_tile<T, LN>) * kWarps)) !=
      cudaSuccess)
    return e;
  back_kernel<T, LN, false><<<(unsigned)(units * q.in.splits), threads, bytes, s>>>(q);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t n = q.in.B * q.in.L * q.in.G * 2 * p.NP;
  sum_maps<T><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(q.part_bc, q.dBm, q.dCm, q.in.B, q.in.L,
                                                          q.in.G, q.in.N, (int)p.NP, (int)p.blocks);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  sum_params<<<(unsigned)((HN + 2 * q.in.H + 127) / 128), 128, 0, s>>>(
      q.part_A, q.part_c, q.dA, q.ddt_bias, q.dD, q.in.B * q.in.splits, q.in.H, HN);
  return cudaGetLastError();
}

template <typename T>
cudaError_t back_of(const ssm_scan_backward_args& a, cudaStream_t s) {
  back_params<T> q{};
  q.in = make_inputs<T>(a);
  q.dy = view<const T>{static_cast<const T*>(a.dy.data), a.dy.stride_b, a.dy.stride_t};
  q.dx = out_view<T>(a.dx), q.ddt = out_view<T>(a.ddt), q.dz = out_view<T>(a.dz);
  q.dBm = out_view<T>(a.dBm), q.dCm = out_view<T>(a.dCm);
  q.states = a.states, q.dh_last = a.dh_last;
  q.dA = a.dA, q.dD = a.dD, q.ddt_bias = a.ddt_bias, q.dh0 = a.dh0;
  const back_plan p = plan(a.B, a.L, a.H, a.N, a.G);
  float* w = static_cast<float*>(a.workspace);
  q.part_bc = w, w += p.bc;
  q.part_A = w, w += p.A;
  q.part_c = w, w += p.c;
  q.in.ends = w, w += a.B * p.splits * a.H * a.N;
  q.in.sums = w;
  switch (lanes_for(a.N)) {
    case 1: return run_back<T, 1>(q, p, s);
    case 2: return run_back<T, 2>(q, p, s);
    case 4: return run_back<T, 4>(q, p, s);
    case 8: return run_back<T, 8>(q, p, s);
    default: return run_back<T, 16>(q, p, s);
  }
}

}  // namespace

size_t scan_backward_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t N, int64_t G) {
  const back_plan p = plan(B, L, H, N, G);
  return (size_t)(p.bc + p.A + p.c + p.map) * 4;
}

cudaError_t launch_scan_backward(const ssm_scan_backward_args& a, cudaStream_t s) {
  if (a.type == GLR_F32) return back_of<float>(a, s);
  return a.type == GLR_BF16 ? back_of<__nv_bfloat16>(a, s) : back_of<__half>(a, s);
}

}  // namespace ssm
}  // namespace dlr
