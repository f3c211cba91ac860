// glr_scan.cu -- the gated linear recurrence of include/glr.h: h_t = abar_t h_{t-1} + b_t per
// channel with a decay that the token chooses, its gradients, and one token from a carried state.
//
// A stretch of steps maps the state before it to the state after it by h -> A h + e, A the product
// of its decays and e its end state from zero; stretches compose in the same form. The gradients
// run backwards in time with G_t = dy_t + abar_{t+1} G_{t+1}: a stretch maps the gradient that
// enters behind it to the one that leaves before it by G -> A G + C with the same A.
//
// Each direction is one launch that reads every input once. A block takes a tile of GLR_STATE_STEPS steps
// of 32 VEC channels, each warp S of the steps with its gates in registers; the warps' maps meet in
// shared memory, the tiles of a row in a chain through global memory: a tile publishes its map, looks
// back over the maps of the tiles before it to the nearest one whose end value is there, and
// publishes its own end value. End values are always formed in the same order (each from the one before
// it), so the results do not depend on which of them a tile found. A tile that begins a sequence
// knows its end from its own steps.
#include "glr_common.cuh"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 16;

int* device_status_word();

namespace glr {
namespace {

constexpr int kTile = GLR_STATE_STEPS;  // steps of a tile: it begins at a kept state
constexpr int kHead = 64;               // words of the chain's workspace before its flags

// Flags of a tile: nothing yet, its map is there, its end value is there.
constexpr uint32_t kHasMap = 1, kHasEnd = 2;
constexpr uint64_t kWaitNs = 1000ull * 1000ull * 1000ull;  // a longer wait is a fault
constexpr int kLook = 32;  // tiles looked back over, one for each lane

__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ uint64_t timer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// What the two directions share. head: a ticket counter, then the flags [chains, tiles], all zero
// at the launch. A chain is the row of tiles of one batch entry and group of 32 VEC channels.
template <typename T>
struct Job {
  view<const T> x, r, i;
  const float* p;
  const uint8_t* reset;
  float* in;     // [B, tiles, H]: the value that enters each tile
  float2* maps;  // [B, tiles, H]: each tile's map
  uint32_t* head;
  int* status;
  int64_t B, L, H, chains;
  int groups, tiles;
  float c;
};

struct Tile {
  int64_t b, chain;
  int group, tile;
};

// Tiles are handed out by a counter, the first tile of every chain before the second of any. A
// block waits for tiles handed out before its own only, and their blocks are running or done,
// whatever order the GPU starts blocks in.
template <bool kChain, typename J>
__device__ __forceinline__ Tile take_tile(const J& q, bool backwards, uint32_t* shared) {
  int64_t k = blockIdx.x;
  if (kChain) {
    if (threadIdx.x == 0) *shared = atomicAdd(q.head, 1u);
    __syncthreads();
    k = *shared;
  }
  Tile at;
  at.tile = (int)(k / q.chains);
  if (backwards) at.tile = q.tiles - 1 - at.tile;
  at.chain = k % q.chains;
  at.group = (int)(at.chain % q.groups);
  at.b = at.chain / q.groups;
  return at;
}

// Called by one warp whose lanes have stored what the flag announces.
__device__ __forceinline__ void publish(uint32_t* flag, uint32_t what) {
  __threadfence();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) store_release(flag, what);
}

// Called by one warp. Waits until one of the `back` <= 32 tiles before this one (lane l looks l + 1
// tiles back, `step` flags from one to the next) has its end value and all those between have
// their maps. Returns how far back it is, or 0 when the wait ran out.
__device__ __forceinline__ int look_back(const uint32_t* flag, int back, int step) {
  const int lane = threadIdx.x & 31;
  uint64_t t0 = 0;
  for (;;) {
    const uint32_t f = lane < back ? load_acquire(flag - (int64_t)step * (lane + 1)) : 0u;
    const uint32_t ends = __ballot_sync(0xffffffffu, f == kHasEnd);
    const uint32_t none = __ballot_sync(0xffffffffu, f == 0u);
    if (ends) {
      const int l = __ffs(ends) - 1;
      if (!(none & ((1u << l) - 1u))) return l + 1;
    }
    const uint64_t t = timer_ns();
    if (t0 == 0) t0 = t;
    if (__any_sync(0xffffffffu, t - t0 > kWaitNs)) return 0;
  }
}

// Called by one warp: the value s that enters the tile, and `end`, the one that leaves it, from
// the tile's map (A, e); `cut`: the map does not depend on what enters. row: the lane's first
// element of in and maps, dir = 1 forwards, -1 backwards. The first tile of the chain has its s.
template <bool kChain, int VEC, typename J>
__device__ __forceinline__ void chain(const J& q, const Tile& at, int64_t row, int dir, bool on,
                                      const float (&A)[VEC], const float (&e)[VEC], bool cut,
                                      float (&s)[VEC], float (&end)[VEC]) {
  const int done = dir > 0 ? at.tile : q.tiles - 1 - at.tile;  // tiles of the chain before this
  const bool last = done == q.tiles - 1;
  const int64_t dH = dir * q.H;
  uint32_t* flag = q.head + kHead + at.chain * q.tiles + at.tile;
  if (kChain && done > 0) {
    if (!last) {
      if (on)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          if (cut)
            q.in[row + dH + v] = e[v];
          else
            q.maps[row + v] = make_float2(A[v], e[v]);
        }
      publish(flag, cut ? kHasEnd : kHasMap);
    }
    const int far = look_back(flag, min(done, kLook), dir);
    if (far == 0 && (threadIdx.x & 31) == 0) report_status(q.status, DLR_ERR_TIMEOUT);
#pragma unroll
    for (int v = 0; v < VEC; ++v)
      s[v] = on && far ? __ldcg(&q.in[row - (far - 1) * dH + v]) : 0.0f;
    for (int k = far - 1; k >= 1; --k)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float2 m = on ? __ldcg(&q.maps[row - k * dH + v]) : make_float2(0.0f, 0.0f);
        s[v] = fmaf(m.x, s[v], m.y);
      }
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) end[v] = cut ? e[v] : fmaf(A[v], s[v], e[v]);
  if (last) return;
  if (!(kChain && done > 0 && cut)) {
    if (on)
#pragma unroll
      for (int v = 0; v < VEC; ++v) q.in[row + dH + v] = end[v];
    if (kChain) publish(flag, kHasEnd);
  }
}

// bits of the n steps from t on that begin a sequence
__device__ __forceinline__ uint32_t cuts(const uint8_t* reset, int64_t first, int n) {
  if (!reset) return 0u;
  const int lane = threadIdx.x & 31;
  return __ballot_sync(0xffffffffu, lane < n && reset[first + lane] != 0);
}

// A decay in one register with its digits both next to 1 and next to 0: a - 1 (negative, with -0 for
// a = 1) where a > 1/2, else a.
__device__ __forceinline__ float keep_decay(const gate& g) { return g.a > 0.5f ? g.w : g.a; }
__device__ __forceinline__ float sign_one(float k) { return signbit(k) ? 1.0f : 0.0f; }
__device__ __forceinline__ float kept_decay(float k) { return k + sign_one(k); }
__device__ __forceinline__ float kept_rest(float k) {  // 1 - a^2
  const float s = sign_one(k);
  return fmaf(-k, fmaf(2.0f, s, k), 1.0f - s);
}

// S steps of VEC channels of an activation; steps from n on are left as they are
template <typename T, int VEC, int S>
__device__ __forceinline__ void load_steps(pack<T, VEC> (&out)[S], const T* p, int64_t st, int n) {
#pragma unroll
  for (int j = 0; j < S; ++j)
    if (j < n) out[j] = *reinterpret_cast<const pack<T, VEC>*>(p + j * st);
}

template <typename T, int VEC, int W, bool kChain>
__global__ void __launch_bounds__(W * 32, 16 / W)
scan_kernel(Job<T> q, view<T> y, const float* __restrict__ h0, float* __restrict__ h_last) {
  constexpr int S = kTile / W;
  __shared__ float2 map_s[W][32 * VEC];
  __shared__ float in_s[32 * VEC];
  __shared__ uint32_t cut_s[W], ticket_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Tile at = take_tile<kChain>(q, false, &ticket_s);
  const int64_t h = ((int64_t)at.group * 32 + lane) * VEC;
  const bool on = h < q.H && DLR_IN(at.b, q.B);
  const int64_t t0 = (int64_t)at.tile * kTile + warp * S;
  const int n = (int)max((int64_t)0, min((int64_t)S, q.L - t0));

  pack<T, VEC> xr[S] = {}, rr[S] = {}, ir[S] = {};
  if (on) {
    load_steps(rr, q.r.row(at.b, t0) + h, q.r.st, n);
    load_steps(ir, q.i.row(at.b, t0) + h, q.i.st, n);
    load_steps(xr, q.x.row(at.b, t0) + h, q.x.st, n);
  }
  float kz[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) kz[v] = on ? -q.c * softplus(q.p[h + v]) * kLog2e : 0.0f;
  const uint32_t cut = cuts(q.reset, at.b * q.L + t0, n);
  float a[S][VEC], b[S][VEC], A[VEC], e[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) A[v] = 1.0f, e[v] = 0.0f;
#pragma unroll
  for (int j = 0; j < S; ++j)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const gate g = make_gate(to_f(rr[j].v[v]), to_f(ir[j].v[v]), kz[v]);
      a[j][v] = g.a;
      b[j][v] = g.m * g.si * to_f(xr[j].v[v]);
      if (n < S && j >= n) a[j][v] = 1.0f, b[j][v] = 0.0f;
      e[v] = (cut >> j) & 1u ? b[j][v] : fmaf(a[j][v], e[v], b[j][v]);
      A[v] *= a[j][v];
    }
#pragma unroll
  for (int v = 0; v < VEC; ++v) map_s[warp][lane * VEC + v] = make_float2(A[v], e[v]);
  if (lane == 0) cut_s[warp] = cut;
  __syncthreads();

  if (warp == 0) {
    float s[VEC], end[VEC];
    bool any = false;
    const int64_t row = (at.b * q.tiles + at.tile) * q.H + h;
#pragma unroll
    for (int w = 1; w < W; ++w)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float2 m = map_s[w][lane * VEC + v];
        e[v] = cut_s[w] ? m.y : fmaf(m.x, e[v], m.y);
        A[v] *= m.x;
      }
#pragma unroll
    for (int w = 0; w < W; ++w) any |= cut_s[w] != 0;
    if (at.tile == 0)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        s[v] = h0 && on ? h0[at.b * q.H + h + v] : 0.0f;
        if (on) q.in[row + v] = s[v];
      }
    chain<kChain>(q, at, row, 1, on, A, e, any, s, end);
    if (at.tile == q.tiles - 1 && h_last && on)
#pragma unroll
      for (int v = 0; v < VEC; ++v) h_last[at.b * q.H + h + v] = end[v];
#pragma unroll
    for (int v = 0; v < VEC; ++v) in_s[lane * VEC + v] = s[v];
  }
  __syncthreads();

  float s[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) s[v] = in_s[lane * VEC + v];
  for (int w = 0; w < warp; ++w)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float2 m = map_s[w][lane * VEC + v];
      s[v] = cut_s[w] ? m.y : fmaf(m.x, s[v], m.y);
    }
  T* yp = y.row(at.b, t0) + h;
#pragma unroll
  for (int j = 0; j < S; ++j) {
    pack<T, VEC> o;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      s[v] = (cut >> j) & 1u ? b[j][v] : fmaf(a[j][v], s[v], b[j][v]);
      o.v[v] = from_f<T>(s[v]);
    }
    if (on && j < n && DLR_IN(t0 + j, q.L)) *reinterpret_cast<pack<T, VEC>*>(yp + j * y.st) = o;
  }
}

template <typename T, int VEC, int W, bool kChain>
__global__ void __launch_bounds__(W * 32, 16 / W)
back_kernel(Job<T> q, view<const T> dy, const float* __restrict__ states,
            const float* __restrict__ dh_last, view<T> dx, view<T> dr, view<T> di,
            float* __restrict__ dh0, float* __restrict__ part) {
  constexpr int S = kTile / W;
  __shared__ float2 map_s[W][32 * VEC];  // (A, e) of each warp's steps
  __shared__ float back_s[W][32 * VEC];  // and C; at the end the warps' sums for dp
  __shared__ float in_s[32 * VEC];
  __shared__ uint32_t cut_s[W], ticket_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Tile at = take_tile<kChain>(q, true, &ticket_s);
  const int64_t h = ((int64_t)at.group * 32 + lane) * VEC;
  const bool on = h < q.H && DLR_IN(at.b, q.B);
  const int64_t t0 = (int64_t)at.tile * kTile + warp * S;
  const int64_t row = (at.b * q.tiles + at.tile) * q.H + h;
  const int n = (int)max((int64_t)0, min((int64_t)S, q.L - t0));

  pack<T, VEC> xr[S] = {}, rr[S] = {}, ir[S] = {}, gr[S] = {};
  if (on) {
    load_steps(rr, q.r.row(at.b, t0) + h, q.r.st, n);
    load_steps(ir, q.i.row(at.b, t0) + h, q.i.st, n);
    load_steps(xr, q.x.row(at.b, t0) + h, q.x.st, n);
    load_steps(gr, dy.row(at.b, t0) + h, dy.st, n);
  }
  float k[VEC], s[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    k[v] = on ? q.c * softplus(q.p[h + v]) : 0.0f;
    s[v] = on ? states[row + v] : 0.0f;
  }
  const uint32_t cut = cuts(q.reset, at.b * q.L + t0, n);
  // the decay (see kept_decay), and b, in whose place the state before the step comes later
  float ka[S][VEC], hb[S][VEC], A[VEC], e[VEC], C[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) A[v] = 1.0f, e[v] = 0.0f, C[v] = 0.0f;
#pragma unroll
  for (int j = 0; j < S; ++j)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const gate g = make_gate(to_f(rr[j].v[v]), to_f(ir[j].v[v]), -k[v] * kLog2e);
      ka[j][v] = keep_decay(g);
      hb[j][v] = g.m * g.si * to_f(xr[j].v[v]);
      if (n < S && j >= n) ka[j][v] = -0.0f, hb[j][v] = 0.0f;
      const float a = kept_decay(ka[j][v]);
      e[v] = (cut >> j) & 1u ? hb[j][v] : fmaf(a, e[v], hb[j][v]);
      A[v] *= a;
    }
#pragma unroll
  for (int j = S - 1; j >= 0; --j)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float G = to_f(gr[j].v[v]) + C[v];
      C[v] = (cut >> j) & 1u ? 0.0f : kept_decay(ka[j][v]) * G;
    }
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    map_s[warp][lane * VEC + v] = make_float2(A[v], e[v]);
    back_s[warp][lane * VEC + v] = C[v];
  }
  if (lane == 0) cut_s[warp] = cut;
  __syncthreads();

  if (warp == 0) {
    float tA[VEC], tC[VEC], in[VEC], end[VEC];
    bool any = false;
#pragma unroll
    for (int v = 0; v < VEC; ++v) tA[v] = 1.0f, tC[v] = 0.0f;
#pragma unroll
    for (int w = W - 1; w >= 0; --w) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float m = map_s[w][lane * VEC + v].x, c = back_s[w][lane * VEC + v];
        tC[v] = cut_s[w] ? c : fmaf(m, tC[v], c);
        tA[v] *= m;
      }
      any |= cut_s[w] != 0;
    }
    if (at.tile == q.tiles - 1)
#pragma unroll
      for (int v = 0; v < VEC; ++v) in[v] = dh_last && on ? dh_last[at.b * q.H + h + v] : 0.0f;
    chain<kChain>(q, at, row, -1, on, tA, tC, any, in, end);
    if (at.tile == 0 && dh0 && on)
#pragma unroll
      for (int v = 0; v < VEC; ++v) dh0[at.b * q.H + h + v] = end[v];
#pragma unroll
    for (int v = 0; v < VEC; ++v) in_s[lane * VEC + v] = in[v];
  }
  // the states before the steps, while the first warp looks along the chain
  for (int w = 0; w < warp; ++w)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float2 m = map_s[w][lane * VEC + v];
      s[v] = cut_s[w] ? m.y : fmaf(m.x, s[v], m.y);
    }
#pragma unroll
  for (int j = 0; j < S; ++j)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float b = hb[j][v];
      if ((cut >> j) & 1u) s[v] = 0.0f;
      hb[j][v] = s[v];
      s[v] = fmaf(kept_decay(ka[j][v]), s[v], b);
    }
  __syncthreads();

  float sum[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) C[v] = in_s[lane * VEC + v], sum[v] = 0.0f;
  for (int w = W - 1; w > warp; --w)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float m = map_s[w][lane * VEC + v].x, c = back_s[w][lane * VEC + v];
      C[v] = cut_s[w] ? c : fmaf(m, C[v], c);
    }
  T* xp = dx.row(at.b, t0) + h;
  T* rp = dr.row(at.b, t0) + h;
  T* ip = di.row(at.b, t0) + h;
#pragma unroll
  for (int j = S - 1; j >= 0; --j) {
    pack<T, VEC> ox, orr, oi;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float sr = sigmoid(to_f(rr[j].v[v])), si = sigmoid(to_f(ir[j].v[v]));
      const float a = kept_decay(ka[j][v]), u = kept_rest(ka[j][v]);
      const float rm = rsqrt_approx(max_nan(u, 1e-36f));
      const float G = to_f(gr[j].v[v]) + C[v], sx = si * to_f(xr[j].v[v]);
      const float E = G * a * (hb[j][v] - a * rm * sx) * sr, Gm = G * (u * rm);
      if (j < n) sum[v] += E;
      ox.v[v] = from_f<T>(Gm * si);
      oi.v[v] = from_f<T>(Gm * sx * (1.0f - si));
      orr.v[v] = from_f<T>(-k[v] * E * (1.0f - sr));
      C[v] = (cut >> j) & 1u ? 0.0f : a * G;
    }
    if (on && j < n && DLR_IN(t0 + j, q.L)) {
      *reinterpret_cast<pack<T, VEC>*>(xp + j * dx.st) = ox;
      *reinterpret_cast<pack<T, VEC>*>(rp + j * dr.st) = orr;
      *reinterpret_cast<pack<T, VEC>*>(ip + j * di.st) = oi;
    }
  }
  __syncthreads();  // back_s has been read
#pragma unroll
  for (int v = 0; v < VEC; ++v) back_s[warp][lane * VEC + v] = sum[v];
  __syncthreads();
  if (warp == 0 && on)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) t += back_s[w][lane * VEC + v];
      part[row + v] = t;
    }
}

// dp = -c sigmoid(p) times the sum of a channel's parts, in a fixed order: a warp for each 32
// channels and 8 rows of warps that share the parts
__global__ void __launch_bounds__(256)
back_sum(const float* __restrict__ part, int64_t n, int64_t H, const float* __restrict__ p, float c,
         float* __restrict__ dp) {
  __shared__ float sums[8][32];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int64_t h = blockIdx.x * (int64_t)32 + lane;
  float s = 0.0f;
  if (h < H)
    for (int64_t k = row; k < n; k += 8) s += part[k * H + h];
  sums[row][lane] = s;
  __syncthreads();
  if (row == 0 && h < H) {
#pragma unroll
    for (int j = 1; j < 8; ++j) s += sums[j][lane];
    dp[h] = -c * sigmoid(p[h]) * s;
  }
}

constexpr int kThreads = 128;

// one token: a thread for each (batch entry, channel)
template <typename T>
__global__ void __launch_bounds__(kThreads)
step_kernel(view<const T> x, view<const T> r, view<const T> i, const float* __restrict__ p,
            const uint8_t* __restrict__ reset, int64_t B, int64_t H, float c, const float* h,
            view<T> y, float* h_out) {
  const int64_t k = blockIdx.x * (int64_t)kThreads + threadIdx.x;
  if (k >= B * H) return;
  const int64_t b = k / H, ch = k % H;
  const float kz = -c * softplus(p[ch]) * kLog2e;
  const gate g = make_gate(to_f(r.row(b, 0)[ch]), to_f(i.row(b, 0)[ch]), kz);
  const float bt = g.m * g.si * to_f(x.row(b, 0)[ch]);
  const float s = reset && reset[b] ? bt : fmaf(g.a, h[k], bt);
  if (!DLR_IN(k, B * H)) return;
  h_out[k] = s;
  y.row(b, 0)[ch] = from_f<T>(s);
}

template <typename T>
view<const T> in_view(const glr_view& v) {
  return {static_cast<const T*>(v.data), v.stride_b, v.stride_t};
}
template <typename T>
view<T> out_view(const glr_out& v) {
  return {static_cast<T*>(v.data), v.stride_b, v.stride_t};
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Bytes of the parts of a workspace: the chain's counter and flags, the maps, the entering values
// and (backwards) the parts of dp. Flags are counted for the narrowest groups, of 32 channels.
struct Space {
  size_t head, maps, in;
  Space(int64_t B, int64_t L, int64_t H) {
    const size_t rows = (size_t)B * (size_t)glr_states(L);
    head = align256(4 * (kHead + rows * (size_t)((H + 31) / 32)));
    maps = align256(sizeof(float2) * rows * (size_t)H);
    in = align256(sizeof(float) * rows * (size_t)H);
  }
};

// Two neighbouring 16-bit channels to a lane when every row begins on a 4-byte boundary and H is
// even: a warp then reads 128 bytes of a row at once, where single channels make 64.
template <typename V>
bool in_pairs(const V& v) {
  return ((reinterpret_cast<uintptr_t>(v.data) | (uintptr_t)(v.stride_b * 2) |
           (uintptr_t)(v.stride_t * 2)) & 3u) == 0;
}

template <typename T, int VEC, typename A>
Job<T> make_job(const A& a, float* in, const Space& sp) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const int64_t groups = (a.H + 32 * VEC - 1) / (32 * VEC);
  return {in_view<T>(a.x), in_view<T>(a.r), in_view<T>(a.i), a.p, a.reset, in,
          reinterpret_cast<float2*>(ws + sp.head), reinterpret_cast<uint32_t*>(ws),
          device_status_word(), a.B, a.L, a.H, a.B * groups, (int)groups, (int)glr_states(a.L),
          (float)a.c};
}
template <typename T>
cudaError_t clear_chain(const Job<T>& q, cudaStream_t s) {
  return cudaMemsetAsync(q.head, 0, 4 * (size_t)(kHead + q.chains * q.tiles), s);
}

template <typename T, int VEC, int W>
cudaError_t scan_v(const glr_scan_args& a, cudaStream_t s) {
  const Space sp(a.B, a.L, a.H);
  float* in = a.states ? a.states
                       : reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + sp.head +
                                                  sp.maps);
  const Job<T> q = make_job<T, VEC>(a, in, sp);
  const unsigned blocks = (unsigned)(q.chains * q.tiles);
  if (q.tiles == 1) {
    scan_kernel<T, VEC, W, false><<<blocks, W * 32, 0, s>>>(q, out_view<T>(a.y), a.h0, a.h_last);
  } else {
    const cudaError_t e = clear_chain(q, s);
    if (e != cudaSuccess) return e;
    scan_kernel<T, VEC, W, true><<<blocks, W * 32, 0, s>>>(q, out_view<T>(a.y), a.h0, a.h_last);
  }
  return cudaGetLastError();
}

template <typename T, int VEC, int W>
cudaError_t back_v(const glr_scan_backward_args& a, cudaStream_t s) {
  const Space sp(a.B, a.L, a.H);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  float* in = reinterpret_cast<float*>(ws + sp.head + sp.maps);
  float* part = reinterpret_cast<float*>(ws + sp.head + sp.maps + sp.in);
  const Job<T> q = make_job<T, VEC>(a, in, sp);
  const unsigned blocks = (unsigned)(q.chains * q.tiles);
  auto launch = [&](auto kernel) {
    kernel<<<blocks, W * 32, 0, s>>>(q, in_view<T>(a.dy), a.states, a.dh_last, out_view<T>(a.dx),
                                     out_view<T>(a.dr), out_view<T>(a.di), a.dh0, part);
  };
  if (q.tiles == 1) {
    launch(back_kernel<T, VEC, W, false>);
  } else {
    const cudaError_t e = clear_chain(q, s);
    if (e != cudaSuccess) return e;
    launch(back_kernel<T, VEC, W, true>);
  }
  back_sum<<<(unsigned)((a.H + 31) / 32), 256, 0, s>>>(part, a.B * q.tiles, a.H, a.p, (float)a.c,
                                                       a.dp);
  return cudaGetLastError();
}

template <typename T>
cudaError_t scan_t(const glr_scan_args& a, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (a.H % 2 == 0 && in_pairs(a.x) && in_pairs(a.r) && in_pairs(a.i) && in_pairs(a.y))
      return scan_v<T, 2, 4>(a, s);
  return scan_v<T, 1, 4>(a, s);
}
template <typename T>
cudaError_t back_t(const glr_scan_backward_args& a, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (a.H % 2 == 0 && in_pairs(a.x) && in_pairs(a.r) && in_pairs(a.i) && in_pairs(a.dy) &&
        in_pairs(a.dx) && in_pairs(a.dr) && in_pairs(a.di))
      return back_v<T, 2, 8>(a, s);
  return back_v<T, 1, 8>(a, s);
}

template <typename T>
cudaError_t step_t(const glr_step_args& a, cudaStream_t s) {
  const int64_t blocks = (a.B * a.H + kThreads - 1) / kThreads;
  step_kernel<T><<<(unsigned)blocks, kThreads, 0, s>>>(
      in_view<T>(a.x), in_view<T>(a.r), in_view<T>(a.i), a.p, a.reset, a.B, a.H, (float)a.c, a.h,
      out_view<T>(a.y), a.h_out);
  return cudaGetLastError();
}

}  // namespace

size_t scan_workspace_bytes(int64_t B, int64_t L, int64_t H) {
  const Space sp(B, L, H);
  return sp.head + sp.maps + sp.in;
}
size_t scan_backward_workspace_bytes(int64_t B, int64_t L, int64_t H) {
  const Space sp(B, L, H);
  return sp.head + sp.maps + 2 * sp.in;
}
// blocks of the largest grid that a call of this size launches
int64_t scan_blocks(int64_t B, int64_t L, int64_t H) {
  return B * glr_states(L) * ((H + 31) / 32);
}

cudaError_t launch_scan(const glr_scan_args& a, cudaStream_t s) {
  if (a.type == GLR_BF16) return scan_t<__nv_bfloat16>(a, s);
  if (a.type == GLR_F16) return scan_t<__half>(a, s);
  return scan_t<float>(a, s);
}
cudaError_t launch_scan_backward(const glr_scan_backward_args& a, cudaStream_t s) {
  if (a.type == GLR_BF16) return back_t<__nv_bfloat16>(a, s);
  if (a.type == GLR_F16) return back_t<__half>(a, s);
  return back_t<float>(a, s);
}
cudaError_t launch_step(const glr_step_args& a, cudaStream_t s) {
  if (a.type == GLR_BF16) return step_t<__nv_bfloat16>(a, s);
  if (a.type == GLR_F16) return step_t<__half>(a, s);
  return step_t<float>(a, s);
}

}  // namespace glr
}  // namespace dlr
