// ssm_conv.cu -- the short causal convolution of include/ssm.h: over a sequence, its gradients, and
// one token.
//
// Memory bounds all three: two arrays go through it forwards and three backwards, and a tap is one
// multiply-add. A thread takes VE neighbouring channels over a run of steps, a few steps at a time with
// the K - 1 inputs before them in registers, and reads the next few meanwhile: each input is read once
// by its run and, of the K - 1 before the run, once more (from the cache: the run before is the
// neighbouring warp's). B4 L16384 H2048 K4 bfloat16 with marks: 92 us forwards (5.8 TB/s), 186 backwards
// and 6 for its sums (4.2 TB/s; fixed latencies at 12 warps an SM), one token of 256 x 4096 5 us.
#include <algorithm>
#include <type_traits>

#include "ssm_common.cuh"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 24;

namespace ssm {
namespace {

constexpr int kWarps = 4;  // of a block: neighbouring runs of the same channels

template <typename T>
struct conv_params {
  int64_t B, L, H;
  int K, act;
  view<const T> x, dy;
  const float *w, *bias;
  const T *state, *dlast;
  const uint8_t* reset;
  view<T> y;  // backwards: dx
  T *last, *dstate;
  float* part;  // [K + 1, parts, H]: a block's sums for the taps and the bias
  int64_t parts;
  int64_t runs;      // of a row
  int run;           // steps of a run
  unsigned columns;  // blocks beside one another over the channels
};

// Steps of a run: long ones repeat less (the inputs before a run, backwards the steps behind it and
// the writing of its sums), short ones where there are few threads.
int run_for(int64_t B, int64_t L, int64_t columns, int lo, int hi) {
  int run = hi;
  while (run > lo && B * ((L + run - 1) / run) * columns < 152 * 32) run /= 2;
  return run;
}
int forward_run(int64_t B, int64_t L, int64_t H) { return run_for(B, L, (H + 127) / 128, 8, 64); }
int back_run(int64_t B, int64_t L, int64_t H) { return run_for(B, L, (H + 63) / 64, 16, 128); }

// VE channels as pairs, on which one instruction works at a time (a single channel pairs with zero).
template <int VE>
struct piece {
  static constexpr int kP = (VE + 1) / 2;
  float2 p[kP];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kP; ++i) p[i] = two(0.0f);
  }
  __device__ __forceinline__ void fma(const piece& a, const piece& b) {
#pragma unroll
    for (int i = 0; i < kP; ++i) p[i] = fma2(a.p[i], b.p[i], p[i]);
  }
  __device__ __forceinline__ void add(const piece& a) {
#pragma unroll
    for (int i = 0; i < kP; ++i) p[i] = add2(p[i], a.p[i]);
  }
  __device__ __forceinline__ void mul(const piece& a) {
#pragma unroll
    for (int i = 0; i < kP; ++i) p[i] = mul2(p[i], a.p[i]);
  }
  template <typename T>
  __device__ __forceinline__ void from(const words<T, VE>& w) {
    float v[VE];
    w.to(v);
    set(v);
  }
  __device__ __forceinline__ void set(const float* v) {
#pragma unroll
    for (int i = 0; i < kP; ++i) p[i] = make_float2(v[2 * i], 2 * i + 1 < VE ? v[2 * i + 1] : 0.0f);
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = i & 1 ? p[i / 2].y : p[i / 2].x;
  }
  template <typename T>
  __device__ __forceinline__ void put(T* to) const {
    float v[VE];
    get(v);
    words<T, VE> w;
    w.from(v);
    w.put(to);
  }
  __device__ __forceinline__ void silu() {
#pragma unroll
    for (int i = 0; i < kP; ++i) p[i] = mul2(p[i], glr::sigmoid2(p[i]));
  }
  __device__ __forceinline__ void silu_slope() {  // s + p s (1 - s)
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const float2 s = glr::sigmoid2(p[i]);
      p[i] = fma2(mul2(p[i], s), fma2(s, two(-1.0f), two(1.0f)), s);
    }
  }
};

// The input of step t (which may lie before the first): x, the carried state or zero.
template <typename T, int VE>
__device__ __forceinline__ void input(piece<VE>& v, const conv_params<T>& q, int64_t b, int64_t t,
                                      int64_t c) {
  words<T, VE> w;
  if (!DLR_IN(c + VE - 1, q.H) || !DLR_IN(t + q.K - 1, q.L + q.K - 1)) t = 0, c = 0;
  if (t >= 0)
    w.get(q.x.row(b, t) + c);
  else if (q.state)
    w.get(q.state + (b * (q.K - 1) + t + q.K - 1) * q.H + c);
  v.from(w);
}

// Taps of a thread's channels: w[j] of x_{t-j}.
template <typename T, int VE, int KM>
__device__ __forceinline__ void taps(piece<VE> (&w)[KM], piece<VE>& bias, const conv_params<T>& q,
                                     int64_t c) {
  float v[VE];
#pragma unroll
  for (int i = 0; i < VE; ++i) v[i] = q.bias ? q.bias[c + i] : 0.0f;
  bias.set(v);
  if (KM == 4 && q.K == 4 && (reinterpret_cast<uintptr_t>(q.w) & 15) == 0) {
    float4 t[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) t[i] = *reinterpret_cast<const float4*>(q.w + (c + i) * 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int i = 0; i < VE; ++i) v[i] = j == 0 ? t[i].w : j == 1 ? t[i].z : j == 2 ? t[i].y : t[i].x;
      w[j < KM ? j : 0].set(v);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < KM; ++j) {
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = j < q.K ? q.w[(c + i) * q.K + q.K - 1 - j] : 0.0f;
    w[j].set(v);
  }
}

// The marks around step t, the same in all lanes: bit l is step t - 16 + l.
template <typename T>
__device__ __forceinline__ uint32_t marks_around(const conv_params<T>& q, int64_t b, int64_t t,
                                                 int lane) {
  if (!q.reset) return 0;
  const int64_t s = t - 16 + lane;
  return __ballot_sync(0xffffffffu, s >= 0 && s < q.L && q.reset[b * q.L + s] != 0);
}
// The marks of 16 steps at a time, as a warp walks over them (t = 0, CH, .. from t0 on): the next
// ones are read meanwhile, so that no step waits for them.
template <typename T>
struct marks_ahead {
  const conv_params<T>& q;
  const uint8_t* row;
  int64_t at;  // the step whose mark this lane has in `next`
  uint8_t next = 0;
  uint32_t bits = 0;
  __device__ __forceinline__ marks_ahead(const conv_params<T>& q, int64_t b, int64_t t0, int lane)
      : q(q), row(q.reset ? q.reset + b * q.L : nullptr), at(t0 - 16 + lane) {
    fetch();
  }
  __device__ __forceinline__ void fetch() { next = row && at >= 0 && at < q.L ? row[at] : 0; }
  // those around step t0 + t: bit l is step t0 + t - 16 + l, as far as the 16 steps go
  __device__ __forceinline__ uint32_t around(int t) {
    if (!row) return 0;
    if ((t & 15) == 0) {
      bits = __ballot_sync(0xffffffffu, next != 0);
      at += 16;
      fetch();
    }
    return bits >> (t & 15);
  }
};
// Whether step t + i sees the input j steps before it: no mark on the way.
__device__ __forceinline__ bool sees(uint32_t bits, int i, int j) {
  return (bits >> (17 + i - j) & ((1u << j) - 1)) == 0;
}

// CH steps at a time: v[KM - 1 + i] is the input of step t + i. EXACT: K = KM. Otherwise taps end at
// K: what a tap of zero meets may be infinite.
template <typename T, int VE, int KM, bool EXACT>
__global__ void __launch_bounds__(32 * kWarps) conv_kernel(conv_params<T> q) {
  constexpr int CH = 8, HALO = KM - 1;
  const int lane = threadIdx.x & 31;
  const int64_t c0 = ((int64_t)(blockIdx.x % q.columns) * 32 + lane) * VE;
  const int64_t run = (int64_t)(blockIdx.x / q.columns) * kWarps + (threadIdx.x >> 5);
  const int64_t b = run / q.runs, t0 = (run - b * q.runs) * q.run;
  if (b >= q.B) return;
  const bool there = c0 < q.H;  // the other lanes vote for the marks
  const int64_t c = there ? c0 : 0;
  piece<VE> w[KM], bias, v[HALO + CH];
  taps<T, VE, KM>(w, bias, q, c);
#pragma unroll
  for (int j = 1; j <= HALO; ++j) {
    v[HALO - j].clear();
    if (EXACT || j < q.K) input<T, VE>(v[HALO - j], q, b, t0 - j, c);
  }
  const int steps_here = (int)min(q.L - t0, (int64_t)q.run);
  marks_ahead<T> ahead(q, b, t0, lane);
  words<T, VE> next[CH];
  const T* px = q.x.row(b, t0) + c;
  T* py = q.y.row(b, t0) + c;
  auto fetch = [&](int t) {
    if (t + CH <= steps_here) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (DLR_IN(t0 + t + i, q.L)) next[i].get(px + i * q.x.st);
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (t + i < steps_here) next[i].get(px + i * q.x.st);
    }
    px += CH * q.x.st;
  };
  fetch(0);
  for (int t = 0; t < steps_here; t += CH) {
#pragma unroll
    for (int i = 0; i < CH; ++i) v[HALO + i].from(next[i]);
    if (t + CH < steps_here) fetch(t + CH);
    const uint32_t bits = ahead.around(t);
    // PLAIN: all CH steps are there and no mark is near
    auto steps = [&](auto plain) {
      constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (!PLAIN && t + i >= steps_here) break;
        piece<VE> o = bias;
#pragma unroll
        for (int j = HALO; j >= 0; --j) {
          if (!EXACT && j >= q.K) continue;
          if (!PLAIN && !sees(bits, i, j)) continue;
          o.fma(w[j], v[HALO + i - j]);
        }
        if (q.act == SSM_ACT_SILU) o.silu();
        if (there && DLR_IN(t0 + t + i, q.L) && DLR_IN(c + VE - 1, q.H)) o.put(py + i * q.y.st);
      }
    };
    if (bits || t + CH > steps_here)
      steps(std::false_type{});
    else
      steps(std::true_type{});
    py += CH * q.y.st;
#pragma unroll
    for (int j = 0; j < HALO; ++j) v[j] = v[CH + j];
  }
  if (t0 + steps_here == q.L && q.last) {
    const uint32_t bits = marks_around(q, b, q.L - 1, lane);
    for (int j = 0; j < q.K - 1; ++j) {
      piece<VE> o;
      o.clear();
      if (sees(bits, 0, j)) input<T, VE>(o, q, b, q.L - 1 - j, c);
      if (there) o.put(q.last + (b * (q.K - 1) + q.K - 2 - j) * q.H + c);
    }
  }
}

// The same backwards in what it forms, not in time: g of a run's steps and of the K - 1 behind it;
// dx of a step is complete K - 1 steps later. g[HALO + i] is that of step t + i.
template <typename T, int VE, int KM, bool EXACT>
__global__ void __launch_bounds__(32 * kWarps, KM == 4 ? 3 : 1) conv_back(conv_params<T> q) {
  constexpr int CH = 4, HALO = KM - 1;
  __shared__ float sums[kWarps][32 * VE];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned column = blockIdx.x % q.columns, part = blockIdx.x / q.columns;
  const int64_t c0 = ((int64_t)column * 32 + lane) * VE;
  const int64_t run = (int64_t)part * kWarps + warp;
  const int64_t b = run / q.runs, t0 = (run - b * q.runs) * q.run;
  const bool there = c0 < q.H;
  const int64_t c = there ? c0 : 0;
  const int halo = EXACT ? HALO : q.K - 1;
  piece<VE> dw[KM], db;
  db.clear();
#pragma unroll
  for (int j = 0; j < KM; ++j) dw[j].clear();
  if (b < q.B) {
    piece<VE> w[KM], bias, v[HALO + CH], g[HALO + CH];
    taps<T, VE, KM>(w, bias, q, c);
#pragma unroll
    for (int j = 1; j <= HALO; ++j) {
      v[HALO - j].clear();
      g[HALO - j].clear();
      if (EXACT || j < q.K) input<T, VE>(v[HALO - j], q, b, t0 - j, c);
    }
    // counted from t0: the run's end, the row's, and where what is read ends
    const int left = (int)min(q.L - t0, (int64_t)(q.run + SSM_MAX_TAPS + CH)), end = min(left, q.run);
    const int stop = min(left, end + halo);
    // the first run also closes the steps of the carried state
    const int from = t0 == 0 ? -halo : 0;
    marks_ahead<T> ahead(q, b, t0, lane);
    words<T, VE> nx[CH], ng[CH];
    const T* px = q.x.row(b, t0) + c;
    const T* pg = q.dy.row(b, t0) + c;
    T* py = q.y.p + b * q.y.sb + (t0 - halo) * q.y.st + c;  // of step t - halo
    auto fetch = [&](int t) {
      if (t + CH <= stop) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          if (!DLR_IN(t0 + t + i, q.L)) continue;
          nx[i].get(px + i * q.x.st);
          ng[i].get(pg + i * q.dy.st);
        }
      } else {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          nx[i] = ng[i] = words<T, VE>();
          if (t + i < stop) {
            nx[i].get(px + i * q.x.st);
            ng[i].get(pg + i * q.dy.st);
          }
        }
      }
      px += CH * q.x.st;
      pg += CH * q.dy.st;
    };
    fetch(0);
    for (int t = 0; t < end + halo; t += CH) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        v[HALO + i].from(nx[i]);
        g[HALO + i].from(ng[i]);
      }
      fetch(t + CH);
      const uint32_t bits = ahead.around(t);
      // PLAIN: all CH steps are the run's own, the steps that they complete too, and no mark is near
      auto steps = [&](auto plain) {
        constexpr bool PLAIN = decltype(plain)::value;
        if (q.act == SSM_ACT_SILU) {
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            piece<VE> p = bias;
#pragma unroll
            for (int j = HALO; j >= 0; --j) {
              if (!EXACT && j > halo) continue;
              if (!PLAIN && !sees(bits, i, j)) continue;
              p.fma(w[j], v[HALO + i - j]);
            }
            p.silu_slope();
            g[HALO + i].mul(p);
            // what is behind the row may have been formed of anything
            if (!PLAIN && t + i >= left) g[HALO + i].clear();
          }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          if (!PLAIN && t + i >= end) continue;
          db.add(g[HALO + i]);
#pragma unroll
          for (int j = 0; j <= HALO; ++j) {
            if (!EXACT && j > halo) continue;
            if (!PLAIN && !sees(bits, i, j)) continue;
            dw[j].fma(g[HALO + i], v[HALO + i - j]);
          }
        }
        // steps t + i - halo are complete
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int done = t + i - halo;
          if (!PLAIN && (done < from || done >= end)) continue;
          piece<VE> o;
          o.clear();
#pragma unroll
          for (int j = 0; j <= HALO; ++j) {  // what step done + j gives it
            if (!EXACT && j > halo) continue;
            if (!PLAIN && !sees(bits, i - halo + j, j)) continue;
            if constexpr (EXACT) {
              o.fma(w[j], g[i + j]);
            } else {  // indexed without an address
#pragma unroll
              for (int m = 0; m < HALO + CH; ++m)
                if (m == HALO - halo + i + j) o.fma(w[j], g[m]);
            }
          }
          if (!PLAIN && q.dlast && done >= left - halo) {
            const int j = left - 1 - done;
            if (sees(marks_around(q, b, q.L - 1, lane), 0, j)) {
              words<T, VE> wl;
              piece<VE> d;
              wl.get(q.dlast + (b * halo + done - (left - halo)) * q.H + c);
              d.from(wl);
              o.add(d);
            }
          }
          if (!there || !DLR_IN(t0 + done + halo, q.L + halo) || !DLR_IN(c + VE - 1, q.H)) continue;
          if (PLAIN || done >= 0)
            o.put(py + i * q.y.st);
          else if (q.dstate)
            o.put(q.dstate + (b * halo + done + halo) * q.H + c);
        }
      };
      if (bits || t + CH > end || t < halo || (q.dlast && t + CH > left - halo))
        steps(std::false_type{});
      else
        steps(std::true_type{});
      py += CH * q.y.st;
#pragma unroll
      for (int j = 0; j < HALO; ++j) {
        v[j] = v[CH + j];
        g[j] = g[CH + j];
      }
    }
  }
  // the block's sums for its channels, tap by tap, the warps in order
#pragma unroll
  for (int j = 0; j <= KM; ++j) {
    if (j < KM && j >= q.K) continue;
    float mine[VE];
    (j < KM ? dw[j < KM ? j : 0] : db).get(mine);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VE; ++i) sums[warp][lane * VE + i] = mine[i];
    __syncthreads();
    for (int k = threadIdx.x; k < 32 * VE; k += 32 * kWarps) {
      const int64_t ch = (int64_t)column * 32 * VE + k;
      float v = 0.0f;
      for (int u = 0; u < kWarps; ++u) v += sums[u][k];
      const int row = j < KM ? q.K - 1 - j : q.K;
      if (ch < q.H && DLR_IN(part, q.parts)) q.part[((int64_t)row * q.parts + part) * q.H + ch] = v;
    }
  }
}

// dw [H, K] and dbias [H] from the blocks' parts: 32 channels to a block, its 8 warps share the
// parts and meet in order.
__global__ void __launch_bounds__(256) conv_sums(const float* part, float* dw, float* dbias,
                                                 int64_t parts, int64_t H, int K) {
  __shared__ float sums[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (c < H)
#pragma unroll 4
    for (int64_t p = warp; p < parts; p += 8) v += part[((int64_t)row * parts + p) * H + c];
  sums[warp][lane] = v;
  __syncthreads();
  if (warp || c >= H) return;
  for (int u = 1; u < 8; ++u) v += sums[u][lane];
  if (row < K)
    dw[c * K + row] = v;
  else if (dbias)
    dbias[c] = v;
}

// A thread has its channels of R batch entries, so that the taps, 16 bytes a channel where an entry's
// inputs and output are 10 (K = 4 in 16 bits), are read once for all of them.
template <typename T, int VE, int KM, int R>
__global__ void __launch_bounds__(128) conv_step(conv_params<T> q) {
  const int64_t c = ((int64_t)(blockIdx.x % q.columns) * 32 + (threadIdx.x & 31)) * VE;
  const int64_t b0 = ((int64_t)(blockIdx.x / q.columns) * 4 + (threadIdx.x >> 5)) * R;
  if (b0 >= q.B || c >= q.H) return;
  piece<VE> w[KM], bias, win[R][KM];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t b = min(b0 + r, q.B - 1);
    const bool fresh = q.reset && q.reset[b] != 0;
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      win[r][j].clear();
      if (j == 0 || (j < q.K && !fresh)) input<T, VE>(win[r][j], q, b, -j, c);
    }
  }
  taps<T, VE, KM>(w, bias, q, c);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t b = b0 + r;
    if (b >= q.B) return;
    piece<VE> o = bias;
#pragma unroll
    for (int j = 0; j < KM; ++j) o.fma(w[j], win[r][j]);
    if (!DLR_IN(c + VE - 1, q.H)) return;
    if (q.act == SSM_ACT_SILU) o.silu();
    o.put(q.y.row(b, 0) + c);
#pragma unroll
    for (int j = 0; j < KM - 1; ++j)
      if (j < q.K - 1) win[r][j].put(q.last + (b * (q.K - 1) + q.K - 2 - j) * q.H + c);
  }
}

// Whether rows of H channels go in pieces of `bytes`: every row begins on a multiple of it.
template <typename T>
bool whole_rows(const conv_params<T>& q, int64_t bytes) {
  auto ok = [&](const auto& v) {
    return !v.p || ((reinterpret_cast<uintptr_t>(v.p) | (uintptr_t)(v.sb * sizeof(T)) |
                     (uintptr_t)(v.st * sizeof(T))) & (uintptr_t)(bytes - 1)) == 0;
  };
  const uintptr_t rest = reinterpret_cast<uintptr_t>(q.state) | reinterpret_cast<uintptr_t>(q.dlast) |
                         reinterpret_cast<uintptr_t>(q.last) | reinterpret_cast<uintptr_t>(q.dstate);
  return (q.H * (int64_t)sizeof(T)) % bytes == 0 && (rest & (uintptr_t)(bytes - 1)) == 0 &&
         ok(q.x) && ok(q.dy) && ok(q.y);
}

enum Dir { kForward, kBack, kStep };

template <typename T, int VE, int KM, bool EXACT, Dir DIR>
void go(conv_params<T> q, cudaStream_t s) {
  q.columns = (unsigned)((q.H + 32 * VE - 1) / (32 * VE));
  if constexpr (DIR == kStep) {
    // four entries to a thread where that leaves every SM its warps
    if (KM == 4 && (int64_t)q.columns * q.B >= 4 * 152 * 8)
      conv_step<T, VE, KM, 4><<<q.columns * (unsigned)((q.B + 15) / 16), 128, 0, s>>>(q);
    else
      conv_step<T, VE, KM, 1><<<q.columns * (unsigned)((q.B + 3) / 4), 128, 0, s>>>(q);
  } else {
    const unsigned grid = q.columns * (unsigned)((q.B * q.runs + kWarps - 1) / kWarps);
    if constexpr (DIR == kForward)
      conv_kernel<T, VE, KM, EXACT><<<grid, 32 * kWarps, 0, s>>>(q);
    else
      conv_back<T, VE, KM, EXACT><<<grid, 32 * kWarps, 0, s>>>(q);
  }
}

// Pieces of 8 bytes; single channels where rows do not stand on multiples of them. Backwards four
// channels in 16 bits leave an SM 12 warps and take 186 us at B4 L16384 H2048, two leave it 16 and take
// 215: what a step costs besides its channels is then shared by fewer.
template <typename T, int KM, bool EXACT, Dir DIR>
void by_piece(const conv_params<T>& q, cudaStream_t s) {
  constexpr int VE = 8 / (int)sizeof(T), kBytes = 8;
  if (whole_rows(q, kBytes))
    go<T, VE, KM, EXACT, DIR>(q, s);
  else
    go<T, 1, KM, EXACT, DIR>(q, s);
}

template <typename T, Dir DIR>
cudaError_t by_taps(const conv_params<T>& q, cudaStream_t s) {
  if (q.K == 4)
    by_piece<T, 4, true, DIR>(q, s);
  else if (q.K < 4)
    by_piece<T, 4, false, DIR>(q, s);
  else
    by_piece<T, SSM_MAX_TAPS, false, DIR>(q, s);
  return cudaGetLastError();
}

template <Dir DIR, typename F>
cudaError_t by_type(int64_t type, F fill, cudaStream_t s) {
  if (type == GLR_F32) return by_taps<float, DIR>(fill(float{}), s);
  if (type == GLR_BF16) return by_taps<__nv_bfloat16, DIR>(fill(__nv_bfloat16{}), s);
  return by_taps<__half, DIR>(fill(__half{}), s);
}

int64_t back_parts(int64_t B, int64_t L, int64_t H) {
  const int64_t run = back_run(B, L, H);
  return (B * ((L + run - 1) / run) + kWarps - 1) / kWarps;
}

}  // namespace

// No more blocks than this to a launch.
int64_t conv_blocks(int64_t B, int64_t L, int64_t H) {
  return ((B * ((L + 7) / 8) + kWarps - 1) / kWarps) * ((H + 31) / 32);
}

size_t conv_backward_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t K) {
  return (size_t)((K + 1) * back_parts(B, L, H) * H) * 4;
}

cudaError_t launch_conv(const ssm_conv_args& a, cudaStream_t s) {
  return by_type<kForward>(a.type, [&](auto t) {
    using T = decltype(t);
    conv_params<T> q{};
    q.B = a.B, q.L = a.L, q.H = a.H, q.K = (int)a.K, q.act = (int)a.act;
    q.x = view<const T>{static_cast<const T*>(a.x.data), a.x.stride_b, a.x.stride_t};
    q.y = view<T>{static_cast<T*>(a.y.data), a.y.stride_b, a.y.stride_t};
    q.w = a.w, q.bias = a.bias, q.reset = a.reset;
    q.state = static_cast<const T*>(a.state), q.last = static_cast<T*>(a.last);
    q.run = forward_run(a.B, a.L, a.H), q.runs = (a.L + q.run - 1) / q.run;
    return q;
  }, s);
}

cudaError_t launch_conv_backward(const ssm_conv_backward_args& a, cudaStream_t s) {
  const int64_t parts = back_parts(a.B, a.L, a.H);
  const cudaError_t e = by_type<kBack>(a.type, [&](auto t) {
    using T = decltype(t);
    conv_params<T> q{};
    q.B = a.B, q.L = a.L, q.H = a.H, q.K = (int)a.K, q.act = (int)a.act;
    q.x = view<const T>{static_cast<const T*>(a.x.data), a.x.stride_b, a.x.stride_t};
    q.dy = view<const T>{static_cast<const T*>(a.dy.data), a.dy.stride_b, a.dy.stride_t};
    q.y = view<T>{static_cast<T*>(a.dx.data), a.dx.stride_b, a.dx.stride_t};
    q.w = a.w, q.bias = a.bias, q.reset = a.reset;
    q.state = static_cast<const T*>(a.state), q.dlast = static_cast<const T*>(a.dlast);
    q.dstate = static_cast<T*>(a.dstate);
    q.part = static_cast<float*>(a.workspace), q.parts = parts;
    q.run = back_run(a.B, a.L, a.H), q.runs = (a.L + q.run - 1) / q.run;
    return q;
  }, s);
  if (e != cudaSuccess) return e;
  conv_sums<<<dim3((unsigned)((a.H + 31) / 32), (unsigned)a.K + 1), 256, 0, s>>>(
      static_cast<const float*>(a.workspace), a.dw, a.dbias, parts, a.H, (int)a.K);
  return cudaGetLastError();
}

cudaError_t launch_conv_step(const ssm_conv_step_args& a, cudaStream_t s) {
  return by_type<kStep>(a.type, [&](auto t) {
    using T = decltype(t);
    conv_params<T> q{};
    q.B = a.B, q.L = 1, q.H = a.H, q.K = (int)a.K, q.act = (int)a.act;
    q.x = view<const T>{static_cast<const T*>(a.x.data), a.x.stride_b, 0};
    q.y = view<T>{static_cast<T*>(a.y.data), a.y.stride_b, 0};
    q.w = a.w, q.bias = a.bias, q.reset = a.reset;
    q.state = static_cast<const T*>(a.state), q.last = static_cast<T*>(a.state_out);
    return q;
  }, s);
}

}  // namespace ssm
}  // namespace dlr
