// ssm_scan.cu -- the selective scan of include/ssm.h over a sequence, and one token of it.
//
// Per channel N states go through h = exp(s A) h + s x Bm and come out as o = sum Cm h: of the bytes
// a token's channel brings (x, dt, z, y: 8 in 16 bits) little, of arithmetic much: at N = 16 sixteen
// exponentials and 64 multiply-adds. So the kernel is built around its inner loop (ssm_common.cuh has
// the layout), which issues for two states a product for the exponent, two exponentials, one
// multiply-add for the state, one for the output and one product for the input. Everything else is
// done once a tile of 16 steps, by pieces of rows: the step's softplus, the skip and the gate.
//
// B4 L4096 H4096 N16 bfloat16 with its states kept takes 424 us (1.9 TB/s): issue slots (52%, 61% where an
// SM has four units; the others have three) and shared memory (67%) bound it; its exponentials alone are
// 115 us. Float32 at B1 L65536 H256 N64 takes 531 us, and 431 for the maps of its 19 splits: its decays
// bound it (the multiply-adds' pipe is busy for 64 and 68% of the time).
#include <type_traits>

#include "ssm_scan.cuh"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 22;

namespace ssm {
namespace {

template <typename T>
struct scan_params {
  inputs<T> in;
  view<T> y;
  float *h_last, *states;
};

// Of a unit: two warps that run it, two that stage, each every other piece of a tile, and two that
// finish. With one of each the case above took 437 us: a helper alone, mostly waiting for itself, took
// as long for a tile as the running warps.
constexpr int kHelpers = 2, kUnitWarps = kHalves + 2 * kHelpers;
// Units of a block, of which an SM has four units' worth. In 16 bits one: where there are few they then
// spread over the SMs (B1 L333 H1024 N16 16 -> 13 us, the case above 423 -> 421). Four for float32, each
// on a quarter of an SM, whose multiply-adds then are not left to chance (B1 L16384 H1024 N16 246 us,
// with one 289), and above 32 states, whose maps are most of what is read and stay in the L1 for all
// four (B4 L4096 H1024 N64 bfloat16 463 us, with one 487).
constexpr int units_of(size_t element, int lanes) { return element == 2 && lanes <= 4 ? 1 : 4; }
template <typename T, int LN>
constexpr int kUnitsOf = units_of(sizeof(T), LN);
// The maps take 0.70 of the scan's time in 16 bits, 0.80 in float32.
int splits_of(size_t element, int64_t B, int64_t L, int64_t H, int64_t N, int64_t G) {
  const int lanes = lanes_for(N);
  return splits_for(B, L, H, G, lanes, units_of(element, lanes), element == 2 ? 0.7 : 0.8);
}

// A unit's part of shared memory: what a tile's steps read (s, s x, Bm, Cm), and the outputs, for two
// tiles in turn.
template <int LN, bool MAP>
struct scan_tile {
  using S = shape<LN>;
  float s[2][kT][S::kCW], u[2][kT][S::kCW];
  float Bm[2][kT][S::kNP];
  float Cm[MAP ? 1 : 2][MAP ? 1 : kT][S::kNP];
  float o[MAP ? 1 : 2][MAP ? 1 : kT][kHalves * LN][S::kCW];  // sums, in the parts of the lanes
};

// MAP: only the state that each split but the last adds, and the sum of its steps.
template <typename T, int LN, bool MAP>
__global__ void __launch_bounds__(32 * kUnitWarps * kUnitsOf<T, LN>, 4 / kUnitsOf<T, LN>)
scan_kernel(scan_params<T> q) {
  using S = shape<LN>;
  constexpr bool kPrecise = sizeof(T) == 4;
  constexpr int CL = 32 / LN, kUnits = kUnitsOf<T, LN>;
  extern __shared__ float4 smem[];
  const inputs<T>& in = q.in;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp % kUnits;
  scan_tile<LN, MAP>& m = reinterpret_cast<scan_tile<LN, MAP>*>(smem)[mine];
  unit<T, LN> u;
  if (!u.find(in, (int64_t)blockIdx.x * kUnits + mine, MAP ? in.splits - 1 : in.splits)) return;
  const int t_first = u.split * in.per_split, t_end = min(in.tiles, t_first + in.per_split);
  const int64_t HN = (int64_t)in.H * in.N, row_map = u.b * in.splits + u.split;

  // a helper's part of the pieces of a tile: every second one, or all of one piece
  constexpr int kMany = S::NV > 1 ? S::NV / kHelpers : 1, kStep = S::NV > 1 ? kHelpers : 1;
  const int part = (warp - kHalves * kUnits) / kUnits % kHelpers;
  const int from = S::NV > 1 ? part : 0;
  const bool busy = S::NV > 1 || part == 0;

  if (warp >= (kHalves + kHelpers) * kUnits) {  // finishes: the sum of the lanes' parts, the skip, the gate
    if constexpr (MAP) {
      for (int tile = t_first; tile <= t_end; ++tile) meet_unit<kUnitWarps>(mine);
    } else {
      const bool full = u.n_ch == S::kCW, ok_z = full && u.pieces(in.z), ok_y = full && u.pieces(q.y);
      const int c = u.channel(lane);
      float D[kPiece];
      load_channels(D, in.D, u, lane);
      words<T, kPiece> wx[kMany], wz[kMany];  // read a tile before their use
      auto fetch = [&](int tile) {
        const int64_t t0 = (int64_t)tile * kT;
        if (!busy) return;
        if (in.D) u.fetch<kMany, kStep>(wx, in.x, t0, in.L, lane, u.whole, from);
        if (!in.z.p) return;
        u.fetch<kMany, kStep>(wz, in.z, t0, in.L, lane, ok_z, from);
      };
      auto finish = [&](int tile) {
        const int64_t t0 = (int64_t)tile * kT;
        if (!busy) return;
        T* py = q.y.p + (u.b * q.y.sb + (t0 + u.step(from, lane)) * q.y.st + u.c0 + c);
        const bool all = ok_y && t0 + kT <= in.L;
#pragma unroll
        for (int k = 0; k < kMany; ++k) {
          const int t = u.step(from + k * kStep, lane);
          float2 o[2] = {two(0.0f), two(0.0f)};
#pragma unroll
          for (int l = 0; l < kHalves * LN; ++l) {
            float v[kPiece];
            load4(v, &m.o[tile & 1][t][l][c]);
            o[0] = l ? add2(o[0], make_float2(v[0], v[1])) : make_float2(v[0], v[1]);
            o[1] = l ? add2(o[1], make_float2(v[2], v[3])) : make_float2(v[2], v[3]);
          }
          if (in.D) {
            float v[kPiece];
            wx[k].to(v);
            o[0] = fma2(make_float2(D[0], D[1]), make_float2(v[0], v[1]), o[0]);
            o[1] = fma2(make_float2(D[2], D[3]), make_float2(v[2], v[3]), o[1]);
          }
          if (in.z.p) {
            float v[kPiece];
            wz[k].to(v);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 z = make_float2(v[2 * i], v[2 * i + 1]);
              o[i] = mul2(o[i], mul2(z, glr::sigmoid2(z)));
            }
          }
          const float y[kPiece] = {o[0].x, o[0].y, o[1].x, o[1].y};
          if (!DLR_IN(c, S::kCW) || !DLR_IN(all ? t0 + t : 0, in.L)) continue;
          if (all)
            put_piece<T, kPiece>(py + k * kStep * (32 / S::kRow) * q.y.st, y, kPiece, true);
          else if (t0 + t < in.L && c < u.n_ch)
            put_piece<T, kPiece>(py + k * kStep * (32 / S::kRow) * q.y.st, y, u.n_ch - c, ok_y);
        }
      };
      meet_unit<kUnitWarps>(mine);
      for (int tile = t_first; tile < t_end; ++tile) {
        if (tile > t_first) finish(tile - 1);
        fetch(tile);
        meet_unit<kUnitWarps>(mine);
      }
      finish(t_end - 1);
    }
    return;
  }
  if (warp >= kHalves * kUnits) {  // stages: its pieces of s and s x, and one of the maps
    float bias[kPiece];
    load_channels(bias, in.bias, u, lane);
    words<T, kPiece> wx[kMany], wd[kMany], wm[S::NB];  // read a tile before their use
    const view<const T>& map = part ? in.Cm : in.Bm;
    auto fetch = [&](int tile) {
      const int64_t t0 = (int64_t)tile * kT;
      if (busy) {
        u.fetch<kMany, kStep>(wx, in.x, t0, in.L, lane, u.whole, from);
        u.fetch<kMany, kStep>(wd, in.dt, t0, in.L, lane, u.whole, from);
      }
      if (!MAP || part == 0) u.fetch_b(wm, map, t0, in.L, in.N, lane);
    };
    auto stage = [&](int tile) {
      if (busy)
        stage_steps<kMany, kStep>(u, in.softplus, (int64_t)tile * kT, in.L, lane, bias, wx, wd,
                                  m.s[tile & 1], m.u[tile & 1], from);
      if constexpr (MAP) {
        if (part == 0) u.put_b(m.Bm[tile & 1], wm, lane);
      } else {
        u.put_b(part ? m.Cm[tile & 1] : m.Bm[tile & 1], wm, lane);
      }
    };
    fetch(t_first);
    stage(t_first);
    if (t_first + 1 < t_end) fetch(t_first + 1);
    meet_unit<kUnitWarps>(mine);
    for (int tile = t_first; tile < t_end; ++tile) {
      if (tile + 1 < t_end) stage(tile + 1);
      if (tile + 2 < t_end) fetch(tile + 2);
      meet_unit<kUnitWarps>(mine);
    }
    return;
  }

  // the recurrence: this lane's channels and states
  const int at = warp / kUnits * LN + lane / CL, cl = lane % CL * kChannels, n0 = at * kStates;
  const int my_ch = u.n_ch - cl;
  const int64_t ch = (int64_t)(u.c0 + cl) * in.N;
  float2 rate[kChannels][kPairs], h[kChannels][kPairs];
  load_rates(rate, in.A, in.N, u.c0 + cl, my_ch, n0);
  clear(h);
  if (!MAP) {
    if (in.h0) load_states(h, in.h0 + u.b * HN + ch, in.N, my_ch, n0);
    enter<false>(h, in, u.b, u.split, u.c0 + cl, my_ch, n0, rate);
  }
  float sum[kChannels] = {};
  bool cut = false;
  float* keep = q.states + (u.b * in.tiles + t_first) * HN + ch + n0;
  const bool keep_whole = my_ch >= kChannels && n0 < in.N && quads(q.states, in.N);
  meet_unit<kUnitWarps>(mine);
  for (int tile = t_first; tile < t_end; ++tile) {
    const int64_t t0 = (int64_t)tile * kT;
    const uint32_t mark = marks(in.reset, u.b, t0, in.L, lane);
    const float (*ms)[S::kCW] = m.s[tile & 1];
    const float (*mu)[S::kCW] = m.u[tile & 1];
    const float (*mb)[S::kNP] = m.Bm[tile & 1];
    const float (*mc)[S::kNP] = m.Cm[MAP ? 0 : tile & 1];
    float (*mo)[kHalves * LN][S::kCW] = m.o[MAP ? 0 : tile & 1];
    if (!MAP && q.states && DLR_IN(tile, in.tiles)) {
      if (keep_whole) {
#pragma unroll
        for (int i = 0; i < kChannels; ++i)
          *reinterpret_cast<float4*>(keep + i * in.N) =
              make_float4(h[i][0].x, h[i][0].y, h[i][1].x, h[i][1].y);
      } else {
        store_states(keep - n0, h, in.N, my_ch, n0);
      }
      keep += HN;
    }
    // A tile without marks goes without looking for them: a branch would keep the steps apart that
    // are to overlap.
    auto steps = [&](auto marks_here) {
      constexpr bool MARKS = decltype(marks_here)::value;
      // a step's words are read a step ahead
      float s_next[kChannels], x_next[kChannels];
      float2 b_next[kPairs], c_next[kPairs];
      auto read = [&](int t) {
        get_channels(s_next, &ms[t][cl]);
        get_channels(x_next, &mu[t][cl]);
        get_map(b_next, &mb[t][n0]);
        if (!MAP) get_map(c_next, &mc[t][n0]);
      };
      read(0);
#pragma unroll 8
      for (int t = 0; t < kT; ++t) {
        float s[kChannels], x[kChannels], o[kChannels];
        float2 bp[kPairs], cp[kPairs];
#pragma unroll
        for (int i = 0; i < kChannels; ++i) s[i] = s_next[i], x[i] = x_next[i];
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
          bp[p] = b_next[p];
          if (!MAP) cp[p] = c_next[p];
        }
        read((t + 1) % kT);  // the last one for nothing
        if (MARKS && (mark >> t & 1)) clear(h);
#pragma unroll
        for (int i = 0; i < kChannels; ++i) {
          float2 acc;
#pragma unroll
          for (int p = 0; p < kPairs; ++p) {
            const decay<kPrecise> a(rate[i][p], two(s[i]));
            h[i][p] = a.of_plus(h[i][p], bp[p], two(x[i]));
            if (!MAP) acc = p ? fma2(h[i][p], cp[p], acc) : mul2(h[i][p], cp[p]);
          }
          if (!MAP) o[i] = acc.x + acc.y;
          if (MAP) sum[i] += s[i];
        }
        if (!MAP) *reinterpret_cast<float2*>(&mo[t][at][cl]) = make_float2(o[0], o[1]);
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
  if (MAP) {
    store_states(in.ends + row_map * HN + ch, h, in.N, my_ch, n0);
    if (at == 0)
#pragma unroll
      for (int i = 0; i < kChannels; ++i)
        if (i < my_ch)
          in.sums[row_map * in.H + u.c0 + cl + i] = cut ? __int_as_float(0x7fffffff) : sum[i];
  } else if (u.split == in.splits - 1 && q.h_last) {
    store_states(q.h_last + u.b * HN + ch, h, in.N, my_ch, n0);
  }
}

template <typename T, int LN>
cudaError_t run_scan(scan_params<T> q, cudaStream_t s) {
  using S = shape<LN>;
  constexpr int kUnits = kUnitsOf<T, LN>;
  q.in.blocks = (q.in.Hg + S::kCW - 1) / S::kCW;
  const int64_t units = (int64_t)q.in.blocks * q.in.G * q.in.B;
  auto grid = [](int64_t n) { return (unsigned)((n + kUnits - 1) / kUnits); };
  cudaError_t e;
  if (q.in.splits > 1) {
    constexpr size_t bytes = sizeof(scan_tile<LN, true>) * kUnits;
    if ((e = max_smem_once<scan_kernel<T, LN, true>>(bytes)) != cudaSuccess) return e;
    scan_kernel<T, LN, true><<<grid(units * (q.in.splits - 1)), 32 * kUnitWarps * kUnits, bytes, s>>>(q);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  constexpr size_t bytes = sizeof(scan_tile<LN, false>) * kUnits;
  if ((e = max_smem_once<scan_kernel<T, LN, false>>(bytes)) != cudaSuccess) return e;
  scan_kernel<T, LN, false><<<grid(units * q.in.splits), 32 * kUnitWarps * kUnits, bytes, s>>>(q);
  return cudaGetLastError();
}

template <typename T>
cudaError_t scan_of(const ssm_scan_args& a, cudaStream_t s) {
  scan_params<T> q{make_inputs<T>(a, splits_of(sizeof(T), a.B, a.L, a.H, a.N, a.G)), out_view<T>(a.y), a.h_last, a.states};
  q.in.ends = static_cast<float*>(a.workspace);
  q.in.sums = q.in.ends + a.B * q.in.splits * a.H * a.N;
  switch (lanes_for(a.N)) {
    case 1: return run_scan<T, 1>(q, s);
    case 2: return run_scan<T, 2>(q, s);
    case 4: return run_scan<T, 4>(q, s);
    default: return run_scan<T, 8>(q, s);
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

// LN lanes to a channel, Q quads of states to a lane (the lanes' quads in turn, so that a channel's lie
// beside one another), of R batch entries (the rates are then read once for all of them). The states
// go through memory once each way and are all there is to it: 134 MB at 256 x 4096 x 16, which took
// 36 us with one quad to a lane and its maps read one by one (the steps and gates, formed by every
// lane of a channel, bound it then), and takes 27 with two quads, in blocks of 128 threads (5.4 TB/s).
constexpr int kStepThreads = 128;
template <typename T, int LN, int Q, bool QUADS, int R>
__global__ void __launch_bounds__(kStepThreads) step_kernel(step_params<T> q) {
  constexpr int P = 2 * Q;  // pairs of states
  const unsigned columns = (unsigned)(q.H + kStepThreads / LN - 1) / (kStepThreads / LN);
  const int at = threadIdx.x % LN, n0 = 4 * at;
  const int c0 = (int)(blockIdx.x % columns) * (kStepThreads / LN) + threadIdx.x / LN, c = min(c0, q.H - 1);
  const int64_t b0 = (int64_t)(blockIdx.x / columns) * R;
  const int group = c / q.Hg;
  float2 rate[P], h[R][P], bm[R][P], cm[R][P];
  float s[R], x[R], z[R];
  auto quad = [&](float2 (&v)[P], const float* p) {
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      const float4 t = get_quad(p, n0 + 4 * LN * k, q.N, QUADS);
      v[2 * k] = make_float2(t.x, t.y);
      v[2 * k + 1] = make_float2(t.z, t.w);
    }
  };
  auto map = [&](float2 (&v)[P], const T* p) {
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      words<T, 4> w;
      float t[4];
      get_piece<T, 4>(w, p + n0 + 4 * LN * k, q.N - n0 - 4 * LN * k, QUADS);
      w.to(t);
      v[2 * k] = make_float2(t[0], t[1]);
      v[2 * k + 1] = make_float2(t[2], t[3]);
    }
  };
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t b = min(b0 + r, q.B - 1);
    quad(h[r], q.h + (b * q.H + c) * q.N);
    if (q.reset && q.reset[b])
#pragma unroll
      for (int p = 0; p < P; ++p) h[r][p] = two(0.0f);
    s[r] = to_f(q.dt.row(b, 0)[c]);
    x[r] = to_f(q.x.row(b, 0)[c]);
    z[r] = q.z.p ? to_f(q.z.row(b, 0)[c]) : 0.0f;
    map(bm[r], q.Bm.row(b, 0) + (int64_t)group * q.N);
    map(cm[r], q.Cm.row(b, 0) + (int64_t)group * q.N);
  }
  quad(rate, q.A + (int64_t)c * q.N);
#pragma unroll
  for (int p = 0; p < P; ++p) rate[p] = mul2(rate[p], two(kLog2e));
  const float bias = q.bias ? q.bias[c] : 0.0f, D = q.D ? q.D[c] : 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t b = b0 + r;
    s[r] += bias;
    if (q.softplus) s[r] = softplus2(two(s[r])).x;
    float2 acc;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const decay<sizeof(T) == 4> a(rate[p], two(s[r]));
      h[r][p] = a.of_plus(h[r][p], bm[r][p], two(s[r] * x[r]));
      acc = p ? fma2(h[r][p], cm[r][p], acc) : mul2(h[r][p], cm[r][p]);
    }
    float o = acc.x + acc.y;
#pragma unroll
    for (int d = 1; d < LN; d *= 2) o += __shfl_xor_sync(0xffffffffu, o, d);
    if (b >= q.B || c0 >= q.H || !DLR_IN(QUADS ? n0 + 4 * LN * (Q - 1) + 3 : 0, q.N)) continue;
    float* to = q.h_out + (b * q.H + c) * q.N;
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      const int n = n0 + 4 * LN * k;
      const float2 lo = h[r][2 * k], hi = h[r][2 * k + 1];
      if constexpr (QUADS) {
        *reinterpret_cast<float4*>(to + n) = make_float4(lo.x, lo.y, hi.x, hi.y);
      } else {
        const float v[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < q.N) to[n + j] = v[j];
      }
    }
    if (at) continue;
    if (q.D) o = fmaf(D, x[r], o);
    if (q.z.p) o *= z[r] * glr::sigmoid(z[r]);
    q.y.row(b, 0)[c] = from_f<T>(o);
  }
}

template <typename T, int LN, int Q>
cudaError_t run_step(const step_params<T>& q, cudaStream_t s) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(q.A) | reinterpret_cast<uintptr_t>(q.h) |
                        reinterpret_cast<uintptr_t>(q.h_out);
  const uintptr_t maps = reinterpret_cast<uintptr_t>(q.Bm.p) | reinterpret_cast<uintptr_t>(q.Cm.p) |
                         (uintptr_t)((q.Bm.sb | q.Cm.sb) * (int64_t)sizeof(T));
  const unsigned columns = (unsigned)((q.H + kStepThreads / LN - 1) / (kStepThreads / LN));
  if (q.N == 4 * LN * Q && (all & 15) == 0 && (maps & (4 * sizeof(T) - 1)) == 0) {
    // two entries to a thread where that leaves every SM some blocks
    if (columns * q.B >= 2 * 152 * 4)
      step_kernel<T, LN, Q, true, 2><<<columns * (unsigned)((q.B + 1) / 2), kStepThreads, 0, s>>>(q);
    else
      step_kernel<T, LN, Q, true, 1><<<columns * (unsigned)q.B, kStepThreads, 0, s>>>(q);
  } else {
    step_kernel<T, LN, Q, false, 1><<<columns * (unsigned)q.B, kStepThreads, 0, s>>>(q);
  }
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
  if (a.N <= 4) return run_step<T, 1, 1>(q, s);
  switch (lanes_for(a.N)) {
    case 1: return run_step<T, 1, 2>(q, s);
    case 2: return run_step<T, 2, 2>(q, s);
    case 4: return run_step<T, 4, 2>(q, s);
    default: return run_step<T, 8, 2>(q, s);
  }
}

}  // namespace

size_t scan_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t N, int64_t G) {
  // enough for either type
  return (size_t)map_floats(B, H, N, std::max(splits_of(2, B, L, H, N, G),
                                              splits_of(4, B, L, H, N, G))) * 4;
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
