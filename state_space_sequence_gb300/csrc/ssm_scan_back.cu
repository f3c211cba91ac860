// ssm_scan_back.cu -- the gradients of the selective scan of include/ssm.h.
//
// Backwards in time with the gradient of the state carried along: G_t = g_t Cm_t + a_{t+1} G_{t+1}.
// Sums over the states (q, e, o) go over a channel's lanes, sums over the channels (dBm, dCm) over a
// unit's lanes, then the block's units, then the blocks of a group (through the workspace, added up
// by a second kernel); sums over time stay with the unit's two warps, one partial sum for each batch
// entry and split.
//
// The states are not kept but every 16 steps. A tile's second half needs them first: a run over the
// first half finds where it begins; then each half is run forwards, its states held in registers (8
// steps x 8 numbers a lane), dCm and o formed on the way, and backwards. In all 2.5 exponentials a
// state and step instead of one, for a sixteenth of the memory that all states would take.
//
// B4 L4096 H4096 N16 bfloat16 takes 1512 to 1520 us (and 22 for the two kernels behind it), bound by issue slots (55%, 66% on the 128 SMs that have
// units): 52 instructions for 64 states and steps, 15% of the time for the sums over channels, 14% for the
// helpers' ends of the gradients, 4% for the second run over a first half.
//
// The sums over a unit's channels for dBm and dCm, 8 values over 16 lanes a step at N = 16, go
// through the tensor cores (mma.sync, the only form that takes registers): a product with a matrix
// of ones adds up four lanes, and four steps share one accumulator, so that the rest takes three
// exchanges for four steps. The operands have 11 bits, so each value goes in two parts, which keep 21.
// A value that is not finite spreads over its four steps that way (zero times it is no zero); tiles
// with marks, past which nothing may come, add up by exchanges alone.
#include <type_traits>

#include "ssm_scan.cuh"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 23;

namespace ssm {
namespace {

constexpr int kHalf = kT / 2;  // steps whose states are in registers at a time
constexpr int kUnitWarps = kHalves + 1;  // two run a unit, one stages and finishes

// Units of a block: four, each on a quarter of an SM.
constexpr int kUnits = 4;
// Lanes of a channel: two also for N <= 8, where half of the states are then zeros. Units of 64 channels
// with one lane each take more than a quarter of shared memory: with two of them to a block B4 L4096
// H4096 N8 bfloat16 took 1833 us, now 1550.
int back_lanes(int64_t N) { return std::max(2, lanes_for(N)); }

template <typename T>
struct back_params {
  inputs<T> in;
  view<const T> dy;
  view<T> dx, ddt, dz, dBm, dCm;
  const float *states, *dh_last;
  float *dA, *dD, *ddt_bias, *dh0;
  // parts: dBm and dCm [G, blocks, B, L, 2, NP] (NP = 8 LN), dA [B splits, H, N], ddt_bias and dD
  // [2, B splits, H]
  float *part_bc, *part_A, *part_c;
};

// A unit's part of shared memory: what a tile's steps read and what they leave, two tiles in turn.
// MAP needs s, g and Cm alone.
template <int LN, bool MAP>
struct back_tile {
  using S = shape<LN>;
  static constexpr int kN = MAP ? 1 : 2, kSteps = MAP ? 1 : kT;
  float s[2][kT][S::kCW], g[2][kT][S::kCW], u[2][kT][S::kCW];
  float Bm[kN][kSteps][S::kNP], Cm[2][kT][S::kNP];
  float h[kN][MAP ? 1 : S::kCW][S::kNP];  // the tile's first states
  float q[kN][kSteps][kHalves][S::kCW], e[kN][kSteps][kHalves][S::kCW];
  float o[kN][kSteps][kHalves][S::kCW];
  float dBC[kN][kSteps][2][S::kNP];
};

// Sums over the unit's channels of a lane's 4 values for each of 4 steps: take() for step k of them,
// then finish() writes them to p[k * pitch + 0 .. 4) (p the place of the lane's first state).
struct channel_sums {
  float c[4];
  __device__ __forceinline__ void clear() { c[0] = c[1] = c[2] = c[3] = 0.0f; }
  __device__ __forceinline__ void mma(const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  // A's rows are the quads of lanes (twice), its columns their four lanes (twice); column 2k of the
  // ones picks the first four, 2k + 1 the others, into columns 2k and 2k + 1 of the sums.
  __device__ __forceinline__ void take(const float2 (&v)[kPairs], int k, int lane) {
    const uint32_t one = __float_as_uint(1.0f);
    const uint32_t b0 = lane >> 2 == 2 * k ? one : 0u, b1 = lane >> 2 == 2 * k + 1 ? one : 0u;
    constexpr uint32_t kTop = 0xffffe000u;  // sign, exponent and the 10 leading bits
    const float2 x = v[0], y = v[1];
    const uint32_t hi[4] = {__float_as_uint(x.x) & kTop, __float_as_uint(y.x) & kTop,
                            __float_as_uint(x.y) & kTop, __float_as_uint(y.y) & kTop};
    const float2 lx =
        fma2(make_float2(__uint_as_float(hi[0]), __uint_as_float(hi[2])), two(-1.0f), x);
    const float2 ly =
        fma2(make_float2(__uint_as_float(hi[1]), __uint_as_float(hi[3])), two(-1.0f), y);
    const uint32_t lo[4] = {__float_as_uint(lx.x), __float_as_uint(ly.x), __float_as_uint(lx.y),
                            __float_as_uint(ly.y)};
    mma(lo, b0, b1);
    mma(hi, b0, b1);
  }
  // The other quads of the lane's states are added up; its place in the quad is the step.
  template <int CL>
  __device__ __forceinline__ void finish(float* p, int pitch, int lane) {
    const int quad = (lane >> 2) % (CL / 4);
    sum_lanes<4, 4, CL / 4>(c, quad);
    put_lanes<4, CL / 4>(p + (lane & 3) * pitch, c, quad);
  }
};

template <bool PRECISE>
__device__ __forceinline__ void advance(float2 (&h)[kChannels][kPairs],
                                        const float2 (&rate)[kChannels][kPairs],
                                        const float (&s)[kChannels], const float (&u)[kChannels],
                                        const float2 (&bp)[kPairs]) {
#pragma unroll
  for (int i = 0; i < kChannels; ++i)
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      const decay<PRECISE> a(rate[i][p], two(s[i]));
      h[i][p] = a.of_plus(h[i][p], bp[p], two(u[i]));
    }
}

// MAP: only the gradient that each split but the first sends on, and the sum of its steps.
template <typename T, int LN, bool MAP>
__global__ void __launch_bounds__(32 * kUnitWarps * kUnits, 1) back_kernel(back_params<T> q) {
  using S = shape<LN>;
  constexpr bool kPrecise = sizeof(T) == 4;
  constexpr int CL = 32 / LN;
  extern __shared__ float4 smem[];
  const inputs<T>& in = q.in;
  using tile_t = back_tile<LN, MAP>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp % kUnits;
  tile_t* all = reinterpret_cast<tile_t*>(smem);
  tile_t& m = all[mine];

  // a block: kUnits neighbouring units of one group, split and batch entry (all of them run, also
  // those without channels, for the helpers' meetings)
  const int per_row = in.blocks * in.G, n_split = MAP ? in.splits - 1 : in.splits;
  const int cb = (int)(blockIdx.x % per_row), block = cb % in.blocks;
  unit<T, LN> u;
  u.split = (int)(blockIdx.x / per_row % n_split) + (MAP ? 1 : 0);
  u.b = blockIdx.x / per_row / n_split;
  u.place(in, cb / in.blocks, (block * kUnits + mine) * S::kCW);
  u.whole = u.whole && u.pieces(q.dy);
  const int t_first = u.split * in.per_split, t_end = min(in.tiles, t_first + in.per_split);
  const int64_t HN = (int64_t)in.H * in.N, row_map = u.b * in.splits + u.split;

  if (warp >= kHalves * kUnits) {
    const bool full = u.n_ch == S::kCW, ok_z = full && u.pieces(in.z);
    const bool ok_o = full && u.pieces(q.dx) && u.pieces(q.ddt) && u.pieces(q.dz);
    const int c = u.channel(lane);
    float bias[kPiece], D[kPiece];
    load_channels(bias, in.bias, u, lane);
    load_channels(D, in.D, u, lane);
    // what is staged is read a tile before, where registers hold it
    constexpr bool kAhead = S::NV * sizeof(T) <= 8;
    using piece = words<T, kPiece>;
    piece wx[S::NV], wd[S::NV], wy[S::NV], wz[S::NV], wb[S::NB], wc[S::NB];
    float4 first[4];  // a tile's first states: quads of the unit's kCW x NP
    const bool whole_h = quads(q.states, in.N);
    auto fetch = [&](int tile) {
      const int64_t t0 = (int64_t)tile * kT;
      if (!MAP) u.fetch(wx, in.x, t0, in.L, lane, u.whole);
      u.fetch(wd, in.dt, t0, in.L, lane, u.whole);
      u.fetch(wy, q.dy, t0, in.L, lane, u.whole);
      if (in.z.p) u.fetch(wz, in.z, t0, in.L, lane, ok_z);
      u.fetch_b(wc, in.Cm, t0, in.L, in.N, lane);
      if constexpr (!MAP) {
        u.fetch_b(wb, in.Bm, t0, in.L, in.N, lane);
        const float* src = q.states + (u.b * in.tiles + (DLR_IN(tile, in.tiles) ? tile : 0)) * HN +
                           (int64_t)u.c0 * in.N;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = (k * 32 + lane) * 4, ci = i / S::kNP;
          first[k] = ci < u.n_ch ? get_quad(src + (int64_t)ci * in.N, i % S::kNP, in.N, whole_h)
                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
      }
    };
    auto stage = [&](int tile) {
      const int j = tile & 1;
      stage_steps<S::NV, 1>(u, in.softplus, (int64_t)tile * kT, in.L, lane, bias, MAP ? wd : wx, wd,
                         m.s[j], m.u[j]);
      u.put_b(m.Cm[j], wc, lane);
#pragma unroll
      for (int k = 0; k < S::NV; ++k) {
        float yv[kPiece], zv[kPiece];
        wy[k].to(yv);  // zeros where there is no channel or step
        if (in.z.p) {
          wz[k].to(zv);
#pragma unroll
          for (int i = 0; i < kPiece; i += 2) {
            const float2 z = make_float2(zv[i], zv[i + 1]), g = mul2(z, glr::sigmoid2(z));
            yv[i] *= g.x, yv[i + 1] *= g.y;
          }
        }
        store4(&m.g[j][u.step(k, lane)][c], yv);
      }
      if constexpr (!MAP) {
        u.put_b(m.Bm[j], wb, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<float4*>(&m.h[j][0][0] + (k * 32 + lane) * 4) = first[k];
      }
    };
    // of this lane's channels: ddt and g x summed over time
    float2 sum_t[2] = {two(0.0f), two(0.0f)}, sum_x[2] = {two(0.0f), two(0.0f)};
    auto pair4 = [&](float2 (&v)[2], const float* p) {
      const float4 t = *reinterpret_cast<const float4*>(p);
      v[0] = make_float2(t.x, t.y);
      v[1] = make_float2(t.z, t.w);
    };
    auto both = [&](float2 (&v)[2], const float (*p)[S::kCW]) {  // the two halves' sum
      float2 w[2];
      pair4(v, &p[0][c]);
      pair4(w, &p[1][c]);
      v[0] = add2(v[0], w[0]);
      v[1] = add2(v[1], w[1]);
    };
    auto pairs_of = [](float2 (&v)[2], const piece& w) {
      float t[kPiece];
      w.to(t);
      v[0] = make_float2(t[0], t[1]);
      v[1] = make_float2(t[2], t[3]);
    };
    // the units' dBm and dCm, and what the channels' gradients take besides, by pieces of rows
    auto finish = [&](int tile) {
      const int64_t t0 = (int64_t)tile * kT;
      const int j = tile & 1;
      piece fx[S::NV], fd[S::NV], fy[S::NV], fz[S::NV];
      u.fetch(fx, in.x, t0, in.L, lane, u.whole);
      u.fetch(fd, in.dt, t0, in.L, lane, u.whole);
      if (in.z.p) {
        u.fetch(fy, q.dy, t0, in.L, lane, u.whole);
        u.fetch(fz, in.z, t0, in.L, lane, ok_z);
      }
      meet_finishing<kUnits>();
      constexpr int pitch = 2 * S::kNP, share = kT * pitch / kUnits;
      float* part = q.part_bc +
                    ((((int64_t)u.group * in.blocks + block) * in.B + u.b) * in.L + t0) * pitch;
#pragma unroll
      for (int k = 0; k < (share + 127) / 128; ++k) {
        const int i = mine * share + (k * 32 + lane) * 4;
        if (share % 128 && (k * 32 + lane) * 4 >= share) break;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kUnits; ++w) {
          const float4 p = *reinterpret_cast<const float4*>(&all[w].dBC[j][0][0][0] + i);
          v = make_float4(v.x + p.x, v.y + p.y, v.z + p.z, v.w + p.w);
        }
        if (t0 + i / pitch < in.L &&
            DLR_IN(part + i + 3 - q.part_bc, (int64_t)in.G * in.blocks * in.B * in.L * pitch))
          *reinterpret_cast<float4*>(part + i) = v;
      }
      const bool all_there = ok_o && t0 + kT <= in.L;
      auto out = [&](const view<T>& v, int k, const float2 (&o)[2]) {
        const int64_t t = t0 + u.step(k, lane);
        T* p = v.p + (u.b * v.sb + t * v.st + u.c0 + c);
        const float y[kPiece] = {o[0].x, o[0].y, o[1].x, o[1].y};
        if (!DLR_IN(all_there ? t : 0, in.L) || !DLR_IN(all_there ? c + kPiece - 1 : 0, S::kCW)) return;
        if (all_there)
          put_piece<T, kPiece>(p, y, kPiece, true);
        else if (t < in.L && c < u.n_ch)
          put_piece<T, kPiece>(p, y, u.n_ch - c, ok_o);
      };
      // steps and channels that do not exist add nothing to the sums
#pragma unroll
      for (int k = 0; k < S::NV; ++k) {
        const int t = u.step(k, lane);
        const bool there = full ? t0 + t < in.L : t0 + t < in.L && c < u.n_ch;
        float2 xv[2], dv[2], gv[2], qv[2], ev[2], sv[2];
        pairs_of(xv, fx[k]);
        pairs_of(dv, fd[k]);
        both(qv, m.q[j][t]);
        both(ev, m.e[j][t]);
        pair4(gv, &m.g[j][t][c]);
        pair4(sv, &m.s[j][t][c]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // e was summed with the rates in powers of two
          float2 d = fma2(xv[i], qv[i], mul2(ev[i], two(1.0f / kLog2e)));
          if (in.softplus)
            d = mul2(d, glr::sigmoid2(add2(dv[i], make_float2(bias[2 * i], bias[2 * i + 1]))));
          dv[i] = d;
          if (!full) {
            if (c + 2 * i >= u.n_ch) d.x = 0.0f;
            if (c + 2 * i + 1 >= u.n_ch) d.y = 0.0f;
          }
          if (there) {
            sum_t[i] = add2(sum_t[i], d);
            sum_x[i] = fma2(gv[i], xv[i], sum_x[i]);
          }
          qv[i] = fma2(sv[i], qv[i], mul2(make_float2(D[2 * i], D[2 * i + 1]), gv[i]));
        }
        out(q.ddt, k, dv);
        out(q.dx, k, qv);
        if (in.z.p) {
          float2 zv[2];
          pairs_of(zv, fz[k]);
          pairs_of(gv, fy[k]);
          both(qv, m.o[j][t]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 s = glr::sigmoid2(zv[i]);
            const float2 slope = fma2(mul2(zv[i], s), fma2(s, two(-1.0f), two(1.0f)), s);
            const float2 o = fma2(make_float2(D[2 * i], D[2 * i + 1]), xv[i], qv[i]);
            gv[i] = mul2(gv[i], mul2(o, slope));
          }
          out(q.dz, k, gv);
        }
      }
    };
    fetch(t_end - 1);
    stage(t_end - 1);
    if (kAhead && t_end - 2 >= t_first) fetch(t_end - 2);
    meet_unit<kUnitWarps>(mine);
    for (int tile = t_end - 1; tile >= t_first; --tile) {
      if constexpr (!MAP)
        if (tile < t_end - 1) finish(tile + 1);  // reads s and g, whose place the next stage takes
      if (tile - 1 >= t_first) {
        if (!kAhead) fetch(tile - 1);
        stage(tile - 1);
        if (kAhead && tile - 2 >= t_first) fetch(tile - 2);
      }
      // no unit goes on, and over its dBC, before all helpers have read it
      if (!MAP) meet_finishing<kUnits>();
      meet_unit<kUnitWarps>(mine);
    }
    if constexpr (!MAP) {
      finish(t_first);
      float sum[2][kPiece] = {{sum_t[0].x, sum_t[0].y, sum_t[1].x, sum_t[1].y},
                              {sum_x[0].x, sum_x[0].y, sum_x[1].x, sum_x[1].y}};
#pragma unroll
      for (int i = 0; i < kPiece; ++i)
#pragma unroll
        for (int d = S::kRow; d < 32; d *= 2) {
          sum[0][i] += __shfl_xor_sync(0xffffffffu, sum[0][i], d);
          sum[1][i] += __shfl_xor_sync(0xffffffffu, sum[1][i], d);
        }
      if (lane < S::kRow) {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
          if (c + i < u.n_ch) {
            float* p = q.part_c + row_map * in.H + u.c0 + c + i;
            p[0] = sum[0][i];
            p[in.B * in.splits * in.H] = sum[1][i];
          }
      }
    }
    return;
  }

  // the recurrence: this lane's channels and states
  const int half_of = warp / kUnits, at = lane / CL, cl = lane % CL * kChannels;
  const int n0 = (half_of * LN + at) * kStates;
  const int my_ch = u.n_ch - cl;
  const int64_t ch = (int64_t)(u.c0 + cl) * in.N;
  float2 rate[kChannels][kPairs], carry[kChannels][kPairs];
  load_rates(rate, in.A, in.N, u.c0 + cl, my_ch, n0);
  clear(carry);
  if (!MAP) {
    if (q.dh_last) load_states(carry, q.dh_last + u.b * HN + ch, in.N, my_ch, n0);
    enter<true>(carry, in, u.b, u.split, u.c0 + cl, my_ch, n0, rate);
  }
  meet_unit<kUnitWarps>(mine);

  // A tile without marks goes without looking for them: a branch would keep the steps apart that are
  // to overlap. A step's words are read a step ahead (the last ones for nothing).
  if constexpr (MAP) {
    float sum[kChannels] = {};
    bool cut = false;
    for (int tile = t_end - 1; tile >= t_first; --tile) {
      const uint32_t mark = marks(in.reset, u.b, (int64_t)tile * kT, in.L, lane);
      const int j = tile & 1;
      auto steps = [&](auto marks_here) {
        constexpr bool MARKS = decltype(marks_here)::value;
        float s_next[kChannels], g_next[kChannels];
        float2 c_next[kPairs];
        auto read = [&](int t) {
          get_channels(s_next, &m.s[j][t][cl]);
          get_channels(g_next, &m.g[j][t][cl]);
          get_map(c_next, &m.Cm[j][t][n0]);
        };
        read(kT - 1);
#pragma unroll 4
        for (int t = kT - 1; t >= 0; --t) {
          float s[kChannels], g[kChannels];
          float2 cp[kPairs];
#pragma unroll
          for (int i = 0; i < kChannels; ++i) s[i] = s_next[i], g[i] = g_next[i];
#pragma unroll
          for (int p = 0; p < kPairs; ++p) cp[p] = c_next[p];
          read((t + kT - 1) % kT);
#pragma unroll
          for (int i = 0; i < kChannels; ++i) {
#pragma unroll
            for (int p = 0; p < kPairs; ++p) {
              const decay<kPrecise> a(rate[i][p], two(s[i]));
              carry[i][p] = a.of(fma2(cp[p], two(g[i]), carry[i][p]));
            }
            sum[i] += s[i];
          }
          if (MARKS && (mark >> t & 1)) clear(carry);
        }
      };
      if (mark) {
        steps(std::true_type{});
        cut = true;
      } else {
        steps(std::false_type{});
      }
      meet_unit<kUnitWarps>(mine);
    }
    store_states(in.ends + row_map * HN + ch, carry, in.N, my_ch, n0);
    if (n0 == 0)
#pragma unroll
      for (int i = 0; i < kChannels; ++i)
        if (i < my_ch)
          in.sums[row_map * in.H + u.c0 + cl + i] = cut ? __int_as_float(0x7fffffff) : sum[i];
  } else {
    float2 dA[kChannels][kPairs];
    clear(dA);
    for (int tile = t_end - 1; tile >= t_first; --tile) {
      const uint32_t mark = marks(in.reset, u.b, (int64_t)tile * kT, in.L, lane);
      const int j = tile & 1;
      float (*dBC)[2][S::kNP] = m.dBC[j];
      auto steps = [&](auto marks_here) {
        constexpr bool MARKS = decltype(marks_here)::value;
        float2 h[kChannels][kPairs];
        float s_next[kChannels], x_next[kChannels], g_next[kChannels];
        float2 b_next[kPairs], c_next[kPairs];
        auto read = [&](int t) {
          get_channels(s_next, &m.s[j][t][cl]);
          get_channels(x_next, &m.u[j][t][cl]);
          get_map(b_next, &m.Bm[j][t][n0]);
        };
        auto read_all = [&](int t) {
          read(t);
          get_channels(g_next, &m.g[j][t][cl]);
          get_map(c_next, &m.Cm[j][t][n0]);
        };
        // where the second half begins
#pragma unroll
        for (int i = 0; i < kChannels; ++i) get_map(h[i], &m.h[j][cl + i][n0]);
        read(0);
#pragma unroll 4
        for (int t = 0; t < kHalf; ++t) {
          float s[kChannels], x[kChannels];
          float2 bp[kPairs];
#pragma unroll
          for (int i = 0; i < kChannels; ++i) s[i] = s_next[i], x[i] = x_next[i];
#pragma unroll
          for (int p = 0; p < kPairs; ++p) bp[p] = b_next[p];
          read(t + 1);
          if (MARKS && (mark >> t & 1)) clear(h);
          advance<kPrecise>(h, rate, s, x, bp);
        }
#pragma unroll 1
        for (int half = 1; half >= 0; --half) {
          const int t_half = half * kHalf;
          float2 hist[kHalf][kChannels][kPairs];
          channel_sums sums;
          read_all(t_half);
          if (half == 0)
#pragma unroll
            for (int i = 0; i < kChannels; ++i) get_map(h[i], &m.h[j][cl + i][n0]);
#pragma unroll
          for (int k = 0; k < kHalf; ++k) {
            const int t = t_half + k;
            asm volatile("" ::: "memory");  // words read further ahead would cost registers
            float s[kChannels], x[kChannels], g[kChannels], o[kChannels];
            float2 bp[kPairs], cp[kPairs], d[kPairs];
#pragma unroll
            for (int i = 0; i < kChannels; ++i)
              s[i] = s_next[i], x[i] = x_next[i], g[i] = g_next[i];
#pragma unroll
            for (int p = 0; p < kPairs; ++p) bp[p] = b_next[p], cp[p] = c_next[p];
            read_all(k + 1 < kHalf ? t + 1 : t);
            if (MARKS && (mark >> t & 1)) clear(h);
#pragma unroll
            for (int i = 0; i < kChannels; ++i)
#pragma unroll
              for (int p = 0; p < kPairs; ++p) hist[k][i][p] = h[i][p];
            advance<kPrecise>(h, rate, s, x, bp);
            if (k % 4 == 0) sums.clear();
#pragma unroll
            for (int p = 0; p < kPairs; ++p)
              d[p] = fma2(h[1][p], two(g[1]), mul2(h[0][p], two(g[0])));
            if constexpr (MARKS) {
              float v[4] = {d[0].x, d[0].y, d[1].x, d[1].y};
              sum_lanes<1, 4, CL>(v, lane % CL);
              put_lanes<4, CL>(&dBC[t][1][n0], v, lane % CL);
            } else {
              sums.take(d, k % 4, lane);
            }
#pragma unroll
            for (int i = 0; i < kChannels; ++i) {
              const float2 acc = fma2(h[i][1], cp[1], mul2(h[i][0], cp[0]));
              o[i] = acc.x + acc.y;
            }
            sum_lanes<CL, kChannels, LN>(o, at);
            put_lanes<kChannels, LN>(&m.o[j][t][half_of][cl], o, at);
            if (!MARKS && k % 4 == 3) sums.finish<CL>(&dBC[t - 3][1][n0], 2 * S::kNP, lane);
          }
#pragma unroll
          for (int k = kHalf - 1; k >= 0; --k) {
            const int t = t_half + k;
            asm volatile("" ::: "memory");
            float s[kChannels], x[kChannels], g[kChannels], qv[kChannels], ev[kChannels];
            float2 bp[kPairs], cp[kPairs], db[kPairs];
#pragma unroll
            for (int i = 0; i < kChannels; ++i)
              s[i] = s_next[i], x[i] = x_next[i], g[i] = g_next[i];
#pragma unroll
            for (int p = 0; p < kPairs; ++p) bp[p] = b_next[p], cp[p] = c_next[p];
            if (k) read_all(t - 1);
            if (k % 4 == 3) sums.clear();
#pragma unroll
            for (int i = 0; i < kChannels; ++i) {
              float2 qs, es;
#pragma unroll
              for (int p = 0; p < kPairs; ++p) {
                const float2 G = fma2(cp[p], two(g[i]), carry[i][p]);
                qs = p ? fma2(G, bp[p], qs) : mul2(G, bp[p]);
                db[p] = i ? fma2(G, two(x[i]), db[p]) : mul2(G, two(x[i]));
                const decay<kPrecise> a(rate[i][p], two(s[i]));
                const float2 c = a.of(G), r = mul2(c, hist[k][i][p]);
                carry[i][p] = c;
                es = p ? fma2(r, rate[i][p], es) : mul2(r, rate[i][p]);
                dA[i][p] = fma2(r, two(s[i]), dA[i][p]);
              }
              qv[i] = qs.x + qs.y;
              ev[i] = es.x + es.y;
            }
            if (MARKS && (mark >> t & 1)) clear(carry);
            if constexpr (MARKS) {
              float v[4] = {db[0].x, db[0].y, db[1].x, db[1].y};
              sum_lanes<1, 4, CL>(v, lane % CL);
              put_lanes<4, CL>(&dBC[t][0][n0], v, lane % CL);
            } else {
              sums.take(db, k % 4, lane);
            }
            sum_lanes<CL, kChannels, LN>(qv, at);
            put_lanes<kChannels, LN>(&m.q[j][t][half_of][cl], qv, at);
            sum_lanes<CL, kChannels, LN>(ev, at);
            put_lanes<kChannels, LN>(&m.e[j][t][half_of][cl], ev, at);
            if (!MARKS && k % 4 == 0) sums.finish<CL>(&dBC[t][0][n0], 2 * S::kNP, lane);
          }
        }
      };
      if (mark)
        steps(std::true_type{});
      else
        steps(std::false_type{});
      meet_unit<kUnitWarps>(mine);
    }
    store_states(q.part_A + row_map * HN + ch, dA, in.N, my_ch, n0);
    if (u.split == 0 && q.dh0) store_states(q.dh0 + u.b * HN + ch, carry, in.N, my_ch, n0);
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
  int64_t blocks, NP, splits;  // blocks of a group
  int64_t bc, A, c, map;       // floats of the parts and the splits' maps
};
back_plan plan(int64_t B, int64_t L, int64_t H, int64_t N, int64_t G) {
  back_plan p;
  const int64_t ln = back_lanes(N), cw = 64 / ln, units = (H / G + cw - 1) / cw;
  p.blocks = (units + kUnits - 1) / kUnits;
  p.NP = kHalves * kStates * ln;
  const int64_t want = splits_for(B, L, H, G, (int)ln, kUnits, 0.25), tiles = (L + kT - 1) / kT;
  const int64_t per = (tiles + want - 1) / want;
  p.splits = (tiles + per - 1) / per;
  p.bc = G * p.blocks * B * L * 2 * p.NP;
  p.A = (B * p.splits * H * N + 3) / 4 * 4;
  p.c = (2 * B * p.splits * H + 3) / 4 * 4;
  p.map = map_floats(B, H, N, p.splits);
  return p;
}

template <typename T, int LN>
cudaError_t run_back(back_params<T> q, const back_plan& p, cudaStream_t s) {
  q.in.blocks = (int)p.blocks;
  const int64_t units = p.blocks * q.in.G * q.in.B;
  const int64_t HN = (int64_t)q.in.H * q.in.N;
  cudaError_t e;
  if (q.in.splits > 1) {
    constexpr size_t bytes = sizeof(back_tile<LN, true>) * kUnits;
    if ((e = max_smem_once<back_kernel<T, LN, true>>(bytes)) != cudaSuccess) return e;
    back_kernel<T, LN, true><<<(unsigned)(units * (q.in.splits - 1)), 32 * kUnitWarps * kUnits, bytes, s>>>(q);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  constexpr size_t bytes = sizeof(back_tile<LN, false>) * kUnits;
  static_assert(bytes <= 232448, "shared memory");
  if ((e = max_smem_once<back_kernel<T, LN, false>>(bytes)) != cudaSuccess) return e;
  back_kernel<T, LN, false><<<(unsigned)(units * q.in.splits), 32 * kUnitWarps * kUnits, bytes, s>>>(q);
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
  q.in = make_inputs<T>(a, (int)plan(a.B, a.L, a.H, a.N, a.G).splits);
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
  switch (back_lanes(a.N)) {
    case 2: return run_back<T, 2>(q, p, s);
    case 4: return run_back<T, 4>(q, p, s);
    default: return run_back<T, 8>(q, p, s);
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
