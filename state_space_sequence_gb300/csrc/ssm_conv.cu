// ssm_conv.cu -- the short causal convolution of include/ssm.h: over a sequence, its gradients, and
// one token.
//
// Memory bounds all three: two arrays go through it forwards and three backwards, and a tap is one
// multiply-add. A thread takes VE neighbouring channels over a run of steps, the last K inputs in a
// window of registers: each input is read once by its run and, of the K - 1 before the run, once
// more (from the cache: the run before is the neighbouring warp's). A marked step empties the window.
#include <algorithm>

#include "ssm_common.cuh"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 24;

namespace ssm {
namespace {

constexpr int kWarps = 8;      // of a block: neighbouring runs of the same channels
constexpr int kRun = 16;       // steps of a run, forwards
constexpr int kRunBack = 32;   // and backwards, where a run's sums are written out at its end

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
  int64_t runs;  // of a row
  unsigned columns;  // blocks beside one another over the channels
};

// The input of step t (which may lie before the first): x, the carried state or zero.
template <typename T, int VE>
__device__ __forceinline__ void input(float (&v)[VE], const conv_params<T>& q, int64_t b, int64_t t,
                                      int64_t c) {
  words<T, VE> w;
#pragma unroll
  for (int i = 0; i < VE; ++i) v[i] = 0.0f;
  const T* p = nullptr;
  if (t >= 0)
    p = q.x.row(b, t) + c;
  else if (q.state)
    p = q.state + (b * (q.K - 1) + t + q.K - 1) * q.H + c;
  if (!p) return;
  get_piece<T, VE>(w, p, VE, true);
  w.to(v);
}

// Taps of a thread's channels: w[j] of x_{t-j}.
template <typename T, int VE, int KM>
__device__ __forceinline__ void taps(float (&w)[KM][VE], float (&bias)[VE], const conv_params<T>& q,
                                     int64_t c) {
#pragma unroll
  for (int i = 0; i < VE; ++i) bias[i] = q.bias ? q.bias[c + i] : 0.0f;
#pragma unroll
  for (int j = 0; j < KM; ++j)
#pragma unroll
    for (int i = 0; i < VE; ++i)
      w[j][i] = j < q.K ? q.w[(c + i) * q.K + q.K - 1 - j] : 0.0f;
}

template <typename T>
__device__ __forceinline__ bool marked(const conv_params<T>& q, int64_t b, int64_t t) {
  return q.reset && t >= 0 && q.reset[b * q.L + t] != 0;
}

// EXACT: K = KM. Otherwise the window ends at K: what a tap of zero meets may be infinite.
template <typename T, int VE, int KM, bool EXACT>
__global__ void __launch_bounds__(32 * kWarps) conv_kernel(conv_params<T> q) {
  const int64_t c = ((int64_t)(blockIdx.x % q.columns) * 32 + (threadIdx.x & 31)) * VE;
  const int64_t run = (int64_t)(blockIdx.x / q.columns) * kWarps + (threadIdx.x >> 5);
  const int64_t b = run / q.runs, t0 = (run - b * q.runs) * kRun;
  if (b >= q.B || c >= q.H) return;
  float w[KM][VE], bias[VE], win[KM][VE];  // win[j]: the input j steps before
  taps<T, VE, KM>(w, bias, q, c);
#pragma unroll
  for (int j = 0; j < KM; ++j)
#pragma unroll
    for (int i = 0; i < VE; ++i) win[j][i] = 0.0f;
  const int64_t end = min(q.L, t0 + kRun);
#pragma unroll
  for (int j = KM - 1; j >= 1; --j) {
    if (j >= q.K) continue;
    const int64_t t = t0 - j;
    if (marked(q, b, t))
#pragma unroll
      for (int k = j + 1; k < KM; ++k)
#pragma unroll
        for (int i = 0; i < VE; ++i) win[k][i] = 0.0f;
    input<T, VE>(win[j], q, b, t, c);
  }
  // win[j] for j >= 1 is now the input of t0 - j; the loop moves it on before each step
#pragma unroll
  for (int j = 0; j < KM - 1; ++j)
#pragma unroll
    for (int i = 0; i < VE; ++i) win[j][i] = win[j + 1][i];
#pragma unroll 4
  for (int64_t t = t0; t < end; ++t) {
    float v[VE];
    input<T, VE>(v, q, b, t, c);
    if (marked(q, b, t))
#pragma unroll
      for (int j = 0; j < KM; ++j)
#pragma unroll
        for (int i = 0; i < VE; ++i) win[j][i] = 0.0f;
#pragma unroll
    for (int j = KM - 1; j >= 1; --j)
#pragma unroll
      for (int i = 0; i < VE; ++i) win[j][i] = EXACT || j < q.K ? win[j - 1][i] : 0.0f;
#pragma unroll
    for (int i = 0; i < VE; ++i) win[0][i] = v[i];
    float o[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      o[i] = bias[i];
#pragma unroll
      for (int j = 0; j < KM; ++j) o[i] = fmaf(w[j][i], win[j][i], o[i]);
      if (q.act == SSM_ACT_SILU) o[i] *= glr::sigmoid(o[i]);
    }
    put_piece<T, VE>(q.y.row(b, t) + c, o, VE, true);
  }
  if (end == q.L && q.last) {
#pragma unroll
    for (int j = 0; j < KM - 1; ++j)
      if (j < q.K - 1)
        put_piece<T, VE>(q.last + (b * (q.K - 1) + q.K - 2 - j) * q.H + c, win[j], VE, true);
  }
}

// A run's steps t0 .. t0 + kRunBack - 1: dx of those, from the g of those and of the K - 1 behind
// them. dx of step t is complete K - 1 steps later: `open[j]` is dx of the step j before, so far.
template <typename T, int VE, int KM, bool EXACT>
__global__ void __launch_bounds__(32 * kWarps) conv_back(conv_params<T> q) {
  __shared__ float sums[kWarps][32 * VE];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned column = blockIdx.x % q.columns, part = blockIdx.x / q.columns;
  const int64_t c = ((int64_t)column * 32 + lane) * VE;
  const int64_t run = (int64_t)part * kWarps + warp;
  const int64_t b = run / q.runs, t0 = (run - b * q.runs) * kRunBack;
  const bool there = b < q.B && c < q.H;
  const int halo = EXACT ? KM - 1 : q.K - 1;
  float w[KM][VE], bias[VE], win[KM][VE], open[KM][VE], dw[KM][VE], db[VE];
#pragma unroll
  for (int i = 0; i < VE; ++i) {
    db[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < KM; ++j) win[j][i] = open[j][i] = dw[j][i] = 0.0f;
  }
  if (there) {
    taps<T, VE, KM>(w, bias, q, c);
    int seen = halo;  // inputs before the current one that it sees
#pragma unroll
    for (int j = KM - 1; j >= 1; --j) {
      if (j >= q.K) continue;
      const int64_t t = t0 - j;
      seen = marked(q, b, t) ? 0 : min(seen + 1, halo);
      input<T, VE>(win[j], q, b, t, c);
    }
#pragma unroll
    for (int j = 0; j < KM - 1; ++j)
#pragma unroll
      for (int i = 0; i < VE; ++i) win[j][i] = win[j + 1][i];
    const int64_t end = min(q.L, t0 + kRunBack);
    // the first run also closes the steps of the carried state
    const int64_t from = t0 == 0 ? -halo : t0;
#pragma unroll 2
    for (int64_t t = t0; t < end + halo; ++t) {
      float v[VE], g[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) v[i] = g[i] = 0.0f;
      const bool real = t < q.L;
      if (real) {
        words<T, VE> wg;
        input<T, VE>(v, q, b, t, c);
        get_piece<T, VE>(wg, q.dy.row(b, t) + c, VE, true);
        wg.to(g);
      }
      seen = real && marked(q, b, t) ? 0 : min(seen + 1, halo);
#pragma unroll
      for (int j = KM - 1; j >= 1; --j)
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          win[j][i] = j > seen ? 0.0f : win[j - 1][i];
          open[j][i] = open[j - 1][i];
        }
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        win[0][i] = v[i];
        open[0][i] = 0.0f;
      }
      if (q.act == SSM_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          float p = bias[i];
#pragma unroll
          for (int j = 0; j < KM; ++j) p = fmaf(w[j][i], win[j][i], p);
          const float s = glr::sigmoid(p);
          g[i] *= fmaf(p * s, 1.0f - s, s);
        }
      }
      if (real)
#pragma unroll
        for (int j = 0; j < KM; ++j)
          if (j <= seen)
#pragma unroll
            for (int i = 0; i < VE; ++i) open[j][i] = fmaf(w[j][i], g[i], open[j][i]);
      if (t < end) {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          db[i] += g[i];
#pragma unroll
          for (int j = 0; j < KM; ++j) dw[j][i] = fmaf(g[i], win[j][i], dw[j][i]);
        }
      }
      // step t - halo is complete
      const int64_t done = t - halo;
      if (done < from || done >= end) continue;
      float o[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        o[i] = open[0][i];
#pragma unroll
        for (int j = 1; j < KM; ++j)
          if (j == halo) o[i] = open[j][i];
      }
      if (q.dlast && done >= q.L - halo) {
        bool cut = false;
        for (int64_t s = max(done + 1, (int64_t)0); s < q.L; ++s) cut |= marked(q, b, s);
        if (!cut) {
          words<T, VE> wl;
          float d[VE];
          get_piece<T, VE>(wl, q.dlast + (b * halo + done - (q.L - halo)) * q.H + c, VE, true);
          wl.to(d);
#pragma unroll
          for (int i = 0; i < VE; ++i) o[i] += d[i];
        }
      }
      if (done >= 0)
        put_piece<T, VE>(q.y.row(b, done) + c, o, VE, true);
      else if (q.dstate)
        put_piece<T, VE>(q.dstate + (b * halo + done + halo) * q.H + c, o, VE, true);
    }
  }
  // the block's sums for its channels, tap by tap, the warps in order
#pragma unroll
  for (int j = 0; j <= KM; ++j) {
    if (j < KM && j >= q.K) continue;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VE; ++i) sums[warp][lane * VE + i] = j < KM ? dw[j < KM ? j : 0][i] : db[i];
    __syncthreads();
    for (int k = threadIdx.x; k < 32 * VE; k += 32 * kWarps) {
      const int64_t ch = (int64_t)column * 32 * VE + k;
      float v = 0.0f;
      for (int u = 0; u < kWarps; ++u) v += sums[u][k];
      const int row = j < KM ? q.K - 1 - j : q.K;
      if (ch < q.H) q.part[((int64_t)row * q.parts + part) * q.H + ch] = v;
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

template <typename T, int VE, int KM>
__global__ void __launch_bounds__(128) conv_step(conv_params<T> q) {
  const int64_t per = (q.H + VE - 1) / VE;
  const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
  const int64_t b = i / per, c = (i - b * per) * VE;
  if (b >= q.B) return;
  float w[KM][VE], bias[VE], win[KM][VE];
  taps<T, VE, KM>(w, bias, q, c);
  const bool fresh = q.reset && q.reset[b] != 0;
#pragma unroll
  for (int j = 0; j < KM; ++j) {
#pragma unroll
    for (int k = 0; k < VE; ++k) win[j][k] = 0.0f;
    if (j == 0 || (j < q.K && !fresh)) input<T, VE>(win[j], q, b, -j, c);
  }
  float o[VE];
#pragma unroll
  for (int k = 0; k < VE; ++k) {
    o[k] = bias[k];
#pragma unroll
    for (int j = 0; j < KM; ++j) o[k] = fmaf(w[j][k], win[j][k], o[k]);
    if (q.act == SSM_ACT_SILU) o[k] *= glr::sigmoid(o[k]);
  }
  put_piece<T, VE>(q.y.row(b, 0) + c, o, VE, true);
#pragma unroll
  for (int j = 0; j < KM - 1; ++j)
    if (j < q.K - 1)
      put_piece<T, VE>(q.last + (b * (q.K - 1) + q.K - 2 - j) * q.H + c, win[j], VE, true);
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
    const int64_t n = q.B * ((q.H + VE - 1) / VE);
    conv_step<T, VE, KM><<<(unsigned)((n + 127) / 128), 128, 0, s>>>(q);
  } else {
    const unsigned grid = q.columns * (unsigned)((q.B * q.runs + kWarps - 1) / kWarps);
    if constexpr (DIR == kForward)
      conv_kernel<T, VE, KM, EXACT><<<grid, 32 * kWarps, 0, s>>>(q);
    else
      conv_back<T, VE, KM, EXACT><<<grid, 32 * kWarps, 0, s>>>(q);
  }
}

// Pieces of 16 bytes forwards, 8 backwards (its windows and sums take three times the registers);
// single channels where rows do not stand on multiples of them.
template <typename T, int KM, bool EXACT, Dir DIR>
void by_piece(const conv_params<T>& q, cudaStream_t s) {
  constexpr int kBytes = DIR == kBack ? 8 : 16, VE = kBytes / (int)sizeof(T);
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

int64_t back_parts(int64_t B, int64_t L) {
  return (B * ((L + kRunBack - 1) / kRunBack) + kWarps - 1) / kWarps;
}

}  // namespace

// No more blocks than this to a launch.
int64_t conv_blocks(int64_t B, int64_t L, int64_t H) {
  return ((B * ((L + kRun - 1) / kRun) + kWarps - 1) / kWarps) * ((H + 31) / 32);
}

size_t conv_backward_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t K) {
  return (size_t)((K + 1) * back_parts(B, L) * H) * 4;
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
    q.runs = (a.L + kRun - 1) / kRun;
    return q;
  }, s);
}

cudaError_t launch_conv_backward(const ssm_conv_backward_args& a, cudaStream_t s) {
  const int64_t parts = back_parts(a.B, a.L);
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
    q.runs = (a.L + kRunBack - 1) / kRunBack;
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
