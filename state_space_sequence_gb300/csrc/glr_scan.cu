// glr_scan.cu -- the gated linear recurrence of include/glr.h: h_t = abar_t h_{t-1} + b_t per
// channel with a decay that the token chooses, its gradients, and one token from a carried state.
//
// A stretch of steps maps the state before it to the state after it by h -> A h + e, A the product
// of its decays and e its end state from zero; stretches compose in the same form. The gradients
// run backwards in time with G_t = dy_t + abar_{t+1} G_{t+1}: a stretch maps the gradient that
// enters behind it to the one that leaves before it by G -> A G + C with the same A.
//
// Each direction is one launch that reads every input once from memory. Blocks stay on the GPU and
// take tiles (some steps of a group of channels) in turn; while a block works on one tile, the next
// one's inputs come into shared memory by asynchronous copies. Each warp takes S of a tile's steps,
// its gates in registers; the warps' maps meet in shared memory, the tiles of a row in a chain
// through global memory: a tile publishes its map, looks back over the maps of the tiles before it
// to the nearest one whose end value is there, and publishes its own end value. End values are
// always formed in the same order (each from the one before it), so the results do not depend on
// which of them a tile found. A tile that begins a sequence knows its end from its own steps.
#include <algorithm>

#include "glr_common.cuh"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 16;

int* device_status_word();

namespace glr {
namespace {

constexpr int kHead = 64;  // words of the chain's workspace before its flags

// Flags of a tile: nothing yet, its map is there, its end value is there.
constexpr uint32_t kHasMap = 1, kHasEnd = 2;
constexpr uint64_t kWaitNs = 1000ull * 1000ull * 1000ull;  // a longer wait is a fault

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
  int b, group, tile;  // tile < 0: none left
};

// Tiles are handed out by a counter, the first tile of every chain before the second of any. A
// block takes its tiles in the order it got them and waits for tiles handed out earlier only, so
// the earliest unfinished one waits for nothing, whatever order the GPU runs blocks in.
template <typename J>
__device__ __forceinline__ Tile tile_of(const J& q, uint32_t k, bool backwards) {
  const uint32_t chains = (uint32_t)q.chains;
  Tile at{0, 0, -1};
  if (k >= chains * (uint32_t)q.tiles) return at;
  at.tile = (int)(k / chains);
  const uint32_t chain = k % chains;
  if (backwards) at.tile = q.tiles - 1 - at.tile;
  at.group = (int)(chain % (uint32_t)q.groups);
  at.b = (int)(chain / (uint32_t)q.groups);
  return at;
}

// Called by one warp whose lanes have stored what the flag announces.
__device__ __forceinline__ void publish(uint32_t* flag, uint32_t what) {
  __threadfence();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) store_release(flag, what);
}

// Called by one warp. Waits until one of the `back` tiles before this one has its end value and all
// those between have their maps; each lane looks at one tile at a time (`step` flags from one to
// the next). Returns how far back it is, or 0 when the wait ran out. The first tile of a chain always
// comes to its end value by itself.
__device__ __forceinline__ int look_back(const uint32_t* flag, int back, int step) {
  const int lane = threadIdx.x & 31;
  uint64_t t0 = 0;
  for (int first = 0;;) {
    const int k = first + lane + 1;
    const uint32_t f = k <= back ? load_acquire(flag - (int64_t)step * k) : 0u;
    const uint32_t ends = __ballot_sync(0xffffffffu, f == kHasEnd);
    const uint32_t none = __ballot_sync(0xffffffffu, f == 0u);
    const int l = ends ? __ffs(ends) - 1 : 32;
    if (!(none & (l == 32 ? 0xffffffffu : (1u << l) - 1u))) {
      if (l < 32) return first + l + 1;
      first += 32;  // 32 maps and no end among them
      continue;
    }
    const uint64_t t = timer_ns();
    if (t0 == 0) t0 = t;
    if (__any_sync(0xffffffffu, t - t0 > kWaitNs)) return 0;
  }
}

// Called by one warp: the value s that enters the tile, and `end`, the one that leaves it, from
// the tile's map (A, e); `cut`: the map does not depend on what enters. row: the lane's first
// element of in and maps, dir = 1 forwards, -1 backwards. The first tile of the chain has its s.
template <int VEC, typename J>
__device__ __forceinline__ void chain(const J& q, const Tile& at, int64_t row, int dir,
                                      const bool (&on)[VEC], const float (&A)[VEC],
                                      const float (&e)[VEC], bool cut, float (&s)[VEC],
                                      float (&end)[VEC]) {
  const int done = dir > 0 ? at.tile : q.tiles - 1 - at.tile;  // tiles of the chain before this
  const bool last = done == q.tiles - 1;
  const int64_t dH = dir * q.H;
  uint32_t* flag = q.head + kHead + ((int64_t)at.b * q.groups + at.group) * q.tiles + at.tile;
  if (done > 0) {
    if (!last) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        if (!on[v]) continue;
        if (cut)
          q.in[row + dH + v] = e[v];
        else
          q.maps[row + v] = make_float2(A[v], e[v]);
      }
      publish(flag, cut ? kHasEnd : kHasMap);
    }
    const int far = look_back(flag, done, dir);
    if (far == 0 && (threadIdx.x & 31) == 0) report_status(q.status, DLR_ERR_TIMEOUT);
#pragma unroll
    for (int v = 0; v < VEC; ++v)
      s[v] = on[v] && far ? __ldcg(&q.in[row - (far - 1) * dH + v]) : 0.0f;
#pragma unroll 4
    for (int k = far - 1; k >= 1; --k)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float2 m = on[v] ? __ldcg(&q.maps[row - k * dH + v]) : make_float2(0.0f, 0.0f);
        s[v] = fmaf(m.x, s[v], m.y);
      }
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) end[v] = cut ? e[v] : fmaf(A[v], s[v], e[v]);
  if (last || (done > 0 && cut)) return;
#pragma unroll
  for (int v = 0; v < VEC; ++v)
    if (on[v]) q.in[row + dH + v] = end[v];
  publish(flag, kHasEnd);
}

// bits of the n steps from t on that begin a sequence
__device__ __forceinline__ uint32_t cuts(const uint8_t* reset, int64_t first, int n) {
  if (!reset) return 0u;
  const int lane = threadIdx.x & 31;
  return __ballot_sync(0xffffffffu, lane < n && reset[first + lane] != 0);
}

// A decay in one register with its digits both next to 1 and next to 0: a - 1 (negative; -0 for
// a = 1) where a > 1/2, else a.
__device__ __forceinline__ float2 keep_decay(const gate2& g) {
  return make_float2(g.a.x > 0.5f ? -g.rest.x : g.a.x, g.a.y > 0.5f ? -g.rest.y : g.a.y);
}
__device__ __forceinline__ float2 sign_ones(float2 k) {
  return make_float2(__float_as_int(k.x) < 0 ? 1.0f : 0.0f, __float_as_int(k.y) < 0 ? 1.0f : 0.0f);
}
__device__ __forceinline__ float2 kept_decay(float2 k) { return add2(k, sign_ones(k)); }

// A warp's S steps of VEC channels a lane are S VEC / 2 pairs: the two channels of a step, or, with one
// channel to a lane, two steps. half(): step j of channel v.
template <int VEC, int N>
__device__ __forceinline__ float& half(float2 (&p)[N], int j, int v) {
  if constexpr (VEC == 2) return v ? p[j].y : p[j].x;
  return j & 1 ? p[j / 2].y : p[j / 2].x;
}
__device__ __forceinline__ float2 floats(pack<__nv_bfloat16, 2> k) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&k);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 floats(pack<__half, 2> k) {
  return __half22float2(*reinterpret_cast<const __half2*>(&k));
}
// pair m of the rows [.][C] at p
template <typename T, int VEC, int C>
__device__ __forceinline__ float2 get2(const T* p, int m) {
  if constexpr (VEC == 2) return floats(*reinterpret_cast<const pack<T, 2>*>(p + m * C));
  else return make_float2(p[2 * m * C], p[(2 * m + 1) * C]);
}

// s through the step j: abar s + b
template <int VEC, int N>
__device__ __forceinline__ void advance(float (&s)[VEC], float2 (&a)[N], float2 (&b)[N], int j) {
  if constexpr (VEC == 2) {
    const float2 t = fma2(a[j], make_float2(s[0], s[1]), b[j]);
    s[0] = t.x, s[1] = t.y;
  } else {
    s[0] = fmaf(half<VEC>(a, j, 0), s[0], half<VEC>(b, j, 0));
  }
}

// How a tile's inputs come into shared memory: by asynchronous copies of 16 bytes where every row
// begins on a 16-byte boundary and H is a whole number of them, of 4 bytes where the same holds for 4,
// else (16-bit types with odd strides) by loads of single elements.
template <int kBytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool on) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  const int n = on ? kBytes : 0;  // nothing is read and zeros are written where off
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void copies_end() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// `steps` rows of C channels of v into dst [steps][C]; rows past the end and channels past H are zero
template <typename T, int C, int kBytes, int kThreads>
__device__ __forceinline__ void stage(T* dst, const view<const T>& v, int64_t b, int64_t t0,
                                      int64_t h0, int steps, int64_t L, int64_t H) {
  constexpr int per = kBytes / (int)sizeof(T), cols = C / per;
  const int col = threadIdx.x % cols * per;
  const bool in = h0 + col < H;
  const T* src = v.row(b, t0) + h0 + col;
  if constexpr (kBytes == 2) {
#pragma unroll 4
    for (int j = threadIdx.x / cols; j < steps; j += kThreads / cols)
      dst[j * C + col] = in && t0 + j < L ? src[j * v.st] : from_f<T>(0.0f);
  } else {
    const int64_t dp = (kThreads / cols) * v.st;
    const T* p = src + (threadIdx.x / cols) * v.st;
#pragma unroll 4
    for (int j = threadIdx.x / cols; j < steps; j += kThreads / cols, p += dp) {
      const bool on = in && t0 + j < L;
      copy_async<kBytes>(dst + j * C + col, on ? p : v.p, on);
    }
  }
}

// VEC neighbouring values to memory: at once, or one by one where they are not aligned
template <typename T, int VEC, bool kOne>
__device__ __forceinline__ void put(T* p, const float (&f)[VEC], bool (&on)[VEC]) {
  if constexpr (kOne) {
#pragma unroll
    for (int v = 0; v < VEC; ++v)
      if (on[v]) p[v] = from_f<T>(f[v]);
  } else {
    pack<T, VEC> o;
#pragma unroll
    for (int v = 0; v < VEC; ++v) o.v[v] = from_f<T>(f[v]);
    if (on[0]) *reinterpret_cast<pack<T, VEC>*>(p) = o;
  }
}

// channels of a lane: a warp's row of a tile is 128 bytes
template <typename T>
constexpr int kVec = 4 / (int)sizeof(T);

constexpr int kScanSteps = 16;                       // of a warp
constexpr int kScanWarps = 8;
constexpr int kScanTile = kScanSteps * kScanWarps;   // steps
constexpr int kScanBlocks = 2;                       // blocks that an SM holds

template <typename T, int kBytes>
__global__ void __launch_bounds__(kScanWarps * 32, kScanBlocks)
scan_kernel(Job<T> q, view<T> y, const float* __restrict__ h0, float* __restrict__ h_last,
            float* __restrict__ states) {
  constexpr int VEC = kVec<T>, W = kScanWarps, S = kScanSteps, C = 32 * VEC, threads = W * 32;
  constexpr int NP = S * VEC / 2;
  constexpr bool kOne = kBytes == 2;
  extern __shared__ __align__(16) uint8_t smem[];
  T* const buf = reinterpret_cast<T*>(smem);  // [2][r i x][kScanTile][C]
  __shared__ float2 map_s[W][C];
  __shared__ float in_s[C];
  __shared__ uint32_t cut_s[W];
  __shared__ Tile tile_s[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  if (threadIdx.x == 0) tile_s[0] = tile_of(q, q.tiles > 1 ? atomicAdd(q.head, 1u) : blockIdx.x, false);
  __syncthreads();
  auto fetch = [&](const Tile& at, int k) {
    if (at.tile >= 0) {
      T* d = buf + k * 3 * kScanTile * C;
      const int64_t t0 = (int64_t)at.tile * kScanTile, c0 = (int64_t)at.group * C;
      const int steps = (int)min((int64_t)kScanTile, q.L - t0);
      stage<T, C, kBytes, threads>(d, q.r, at.b, t0, c0, steps, q.L, q.H);
      stage<T, C, kBytes, threads>(d + kScanTile * C, q.i, at.b, t0, c0, steps, q.L, q.H);
      stage<T, C, kBytes, threads>(d + 2 * kScanTile * C, q.x, at.b, t0, c0, steps, q.L, q.H);
    }
    copies_end();
  };
  fetch(tile_s[0], 0);
  for (int turn = 0;; turn ^= 1) {
    const Tile at = tile_s[turn];
    if (at.tile < 0) return;
    uint32_t ticket = 0;
    if (threadIdx.x == 0) {
      ticket = q.tiles > 1 ? atomicAdd(q.head, 1u) : 0xffffffffu;
      tile_s[turn ^ 1] = tile_of(q, ticket, false);
    }
    copies_wait();
    __syncthreads();
    fetch(tile_s[turn ^ 1], turn ^ 1);

    const int64_t h = ((int64_t)at.group * 32 + lane) * VEC;
    const int64_t t0 = (int64_t)at.tile * kScanTile + warp * S;
    const int n = (int)max((int64_t)0, min((int64_t)S, q.L - t0));
    const T* mine = buf + turn * 3 * kScanTile * C + warp * S * C + lane * VEC;
    bool on[VEC];
    float kz[VEC], A[VEC], e[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      on[v] = h + v < q.H && DLR_IN(at.b, q.B);
      kz[v] = on[v] ? -q.c * softplus(q.p[h + v]) * kLog2e : 0.0f;
      A[v] = 1.0f, e[v] = 0.0f;
    }
    const uint32_t cut = cuts(q.reset, at.b * q.L + t0, n);  // as n, the same for all of the warp
    float2 a[NP], b[NP];
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      const gate2 g = make_gate2(get2<T, VEC, C>(mine, m), get2<T, VEC, C>(mine + kScanTile * C, m),
                                 make_float2(kz[0], kz[VEC - 1]));
      a[m] = g.a;
      b[m] = mul2(g.m, mul2(g.si, get2<T, VEC, C>(mine + 2 * kScanTile * C, m)));
    }
    if (n < S) {
#pragma unroll
      for (int j = 0; j < S; ++j)
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          if (j >= n) half<VEC>(a, j, v) = 1.0f, half<VEC>(b, j, v) = 0.0f;
    }
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      if constexpr (VEC == 2) {
        A[0] *= a[m].x, A[1] *= a[m].y;
      } else {
        A[0] *= a[m].x * a[m].y;
      }
    }
    if (cut == 0) {
#pragma unroll
      for (int j = 0; j < S; ++j) advance<VEC>(e, a, b, j);
    } else {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        advance<VEC>(e, a, b, j);
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          if ((cut >> j) & 1u) e[v] = half<VEC>(b, j, v);
      }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) map_s[warp][lane * VEC + v] = make_float2(A[v], e[v]);
    if (lane == 0) cut_s[warp] = cut;
    __syncthreads();

    if (warp == 0) {
      float s[VEC], end[VEC];
      bool any = false;
      const int64_t row = ((int64_t)at.b * q.tiles + at.tile) * q.H + h;
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
        for (int v = 0; v < VEC; ++v) s[v] = h0 && on[v] ? h0[at.b * q.H + h + v] : 0.0f;
      chain(q, at, row, 1, on, A, e, any, s, end);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        if (at.tile == q.tiles - 1 && h_last && on[v]) h_last[at.b * q.H + h + v] = end[v];
        in_s[lane * VEC + v] = s[v];
      }
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
    if (states && t0 % GLR_STATE_STEPS == 0 && n > 0)
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        if (on[v])
          states[(at.b * ((q.L - 1) / GLR_STATE_STEPS + 1) + t0 / GLR_STATE_STEPS) * q.H + h + v] =
              s[v];
    T* yp = y.row(at.b, t0) + h;
    if (n == S && cut == 0) {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        advance<VEC>(s, a, b, j);
        put<T, VEC, kOne>(yp, s, on);
        yp += y.st;
      }
    } else {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        advance<VEC>(s, a, b, j);
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          if ((cut >> j) & 1u) s[v] = half<VEC>(b, j, v);
        if (j < n && DLR_IN(t0 + j, q.L)) put<T, VEC, kOne>(yp, s, on);
        yp += y.st;
      }
    }
  }
}

constexpr int kBackSteps = 8;
constexpr int kBackWarps = 8;
constexpr int kBackTile = kBackSteps * kBackWarps;
constexpr int kBackBlocks = 2;
static_assert(kBackTile == GLR_STATE_STEPS, "a tile begins at a kept state");

template <typename T, int kBytes>
__global__ void __launch_bounds__(kBackWarps * 32, kBackBlocks)
back_kernel(Job<T> q, view<const T> dy, const float* __restrict__ states,
            const float* __restrict__ dh_last, view<T> dx, view<T> dr, view<T> di,
            float* __restrict__ dh0, float* __restrict__ part) {
  constexpr int VEC = kVec<T>, W = kBackWarps, S = kBackSteps, C = 32 * VEC, threads = W * 32;
  constexpr int NP = S * VEC / 2;
  constexpr int kArray = kBackTile * C;
  constexpr bool kOne = kBytes == 2;
  extern __shared__ __align__(16) uint8_t smem[];
  T* const buf = reinterpret_cast<T*>(smem);  // [2][r i x dy][kBackTile][C]
  __shared__ float2 map_s[W][C];  // (A, e) of each warp's steps
  __shared__ float back_s[W][C];  // and C; at the end of a tile the warps' sums for dp
  __shared__ float in_s[C];
  __shared__ uint32_t cut_s[W];
  __shared__ Tile tile_s[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  if (threadIdx.x == 0) tile_s[0] = tile_of(q, q.tiles > 1 ? atomicAdd(q.head, 1u) : blockIdx.x, true);
  __syncthreads();
  auto fetch = [&](const Tile& at, int k) {
    if (at.tile >= 0) {
      T* d = buf + k * 4 * kArray;
      const int64_t t0 = (int64_t)at.tile * kBackTile, c0 = (int64_t)at.group * C;
      const int steps = (int)min((int64_t)kBackTile, q.L - t0);
      stage<T, C, kBytes, threads>(d, q.r, at.b, t0, c0, steps, q.L, q.H);
      stage<T, C, kBytes, threads>(d + kArray, q.i, at.b, t0, c0, steps, q.L, q.H);
      stage<T, C, kBytes, threads>(d + 2 * kArray, q.x, at.b, t0, c0, steps, q.L, q.H);
      stage<T, C, kBytes, threads>(d + 3 * kArray, dy, at.b, t0, c0, steps, q.L, q.H);
    }
    copies_end();
  };
  fetch(tile_s[0], 0);
  for (int turn = 0;; turn ^= 1) {
    const Tile at = tile_s[turn];
    if (at.tile < 0) return;
    if (threadIdx.x == 0)
      tile_s[turn ^ 1] = tile_of(q, q.tiles > 1 ? atomicAdd(q.head, 1u) : 0xffffffffu, true);
    copies_wait();
    __syncthreads();
    fetch(tile_s[turn ^ 1], turn ^ 1);

    const int64_t h = ((int64_t)at.group * 32 + lane) * VEC;
    const int64_t t0 = (int64_t)at.tile * kBackTile + warp * S;
    const int64_t row = ((int64_t)at.b * q.tiles + at.tile) * q.H + h;
    const int n = (int)max((int64_t)0, min((int64_t)S, q.L - t0));
    const T* mine = buf + turn * 4 * kArray + warp * S * C + lane * VEC;
    auto raw = [&](int array, int m) { return get2<T, VEC, C>(mine + array * kArray, m); };
    bool on[VEC];
    float k[VEC], s[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      on[v] = h + v < q.H && DLR_IN(at.b, q.B);
      k[v] = on[v] ? q.c * softplus(q.p[h + v]) : 0.0f;
      s[v] = on[v] ? states[row + v] : 0.0f;
    }
    const uint32_t cut = cuts(q.reset, at.b * q.L + t0, n);
    const float2 k2 = make_float2(k[0], k[VEC - 1]), kz = mul2(k2, two(-kLog2e));
    // the decay (see keep_decay), and b, in whose place the state before the step comes later
    float2 ka[NP], hb[NP];
    float A[VEC], e[VEC], G[VEC];
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      const gate2 g = make_gate2(raw(0, m), raw(1, m), kz);
      ka[m] = keep_decay(g);
      hb[m] = mul2(g.m, mul2(g.si, raw(2, m)));
    }
    if (n < S) {
#pragma unroll
      for (int j = 0; j < S; ++j)
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          if (j >= n) half<VEC>(ka, j, v) = -0.0f, half<VEC>(hb, j, v) = 0.0f;
    }
    // the warp's maps in both directions
    {
      float2 a[NP], t[NP];
#pragma unroll
      for (int m = 0; m < NP; ++m) a[m] = kept_decay(ka[m]), t[m] = raw(3, m);
#pragma unroll
      for (int v = 0; v < VEC; ++v) A[v] = 1.0f, e[v] = 0.0f, G[v] = 0.0f;
#pragma unroll
      for (int j = 0; j < S; ++j) {
        advance<VEC>(e, a, hb, j);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          A[v] *= half<VEC>(a, j, v);
          if ((cut >> j) & 1u) e[v] = half<VEC>(hb, j, v);
        }
      }
#pragma unroll
      for (int j = S - 1; j >= 0; --j)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          const float d = j < n ? half<VEC>(t, j, v) : 0.0f;
          G[v] = (cut >> j) & 1u ? 0.0f : half<VEC>(a, j, v) * (d + G[v]);
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      map_s[warp][lane * VEC + v] = make_float2(A[v], e[v]);
      back_s[warp][lane * VEC + v] = G[v];
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
        for (int v = 0; v < VEC; ++v)
          in[v] = dh_last && on[v] ? dh_last[at.b * q.H + h + v] : 0.0f;
      chain(q, at, row, -1, on, tA, tC, any, in, end);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        if (at.tile == 0 && dh0 && on[v]) dh0[at.b * q.H + h + v] = end[v];
        in_s[lane * VEC + v] = in[v];
      }
    }
    // the states before the steps, while the first warp looks along the chain
    for (int w = 0; w < warp; ++w)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float2 m = map_s[w][lane * VEC + v];
        s[v] = cut_s[w] ? m.y : fmaf(m.x, s[v], m.y);
      }
    {
      float2 a[NP];
#pragma unroll
      for (int m = 0; m < NP; ++m) a[m] = kept_decay(ka[m]);
#pragma unroll
      for (int j = 0; j < S; ++j) {
        float before[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          if ((cut >> j) & 1u) s[v] = 0.0f;
          before[v] = s[v];
        }
        advance<VEC>(s, a, hb, j);
#pragma unroll
        for (int v = 0; v < VEC; ++v) half<VEC>(hb, j, v) = before[v];
      }
    }
    __syncthreads();

    float sum[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) G[v] = in_s[lane * VEC + v], sum[v] = 0.0f;
    for (int w = W - 1; w > warp; --w)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float m = map_s[w][lane * VEC + v].x, c = back_s[w][lane * VEC + v];
        G[v] = cut_s[w] ? c : fmaf(m, G[v], c);
      }
    T* xp = dx.row(at.b, t0) + h;
    T* rp = dr.row(at.b, t0) + h;
    T* ip = di.row(at.b, t0) + h;
#pragma unroll
    for (int m = NP - 1; m >= 0; --m) {
      constexpr int per = VEC == 2 ? 1 : 2;  // steps of a pair
      const int j = m * per;
      if (j >= n) continue;
      const float2 sr = sigmoid2(raw(0, m)), si = sigmoid2(raw(1, m));
      // 1 - a^2 from what is kept: 1 - a^2, or -k (2 + k) with k = a - 1
      const float2 neg = sign_ones(ka[m]), a = add2(ka[m], neg);
      const float2 u = fma2(mul2(ka[m], two(-1.0f)), fma2(neg, two(2.0f), ka[m]),
                            fma2(neg, two(-1.0f), two(1.0f)));
      const float2 rm = rsqrt2(u), sx = mul2(si, raw(2, m)), dyv = raw(3, m);
      float2 t;  // G of the two
      if constexpr (VEC == 2) {
        t = add2(dyv, make_float2(G[0], G[1]));
        const float2 next = mul2(a, t);
        G[0] = (cut >> j) & 1u ? 0.0f : next.x;
        G[1] = (cut >> j) & 1u ? 0.0f : next.y;
      } else {
        t.y = G[0];
        if (j + 1 < n) {
          t.y += dyv.y;
          G[0] = (cut >> (j + 1)) & 1u ? 0.0f : a.y * t.y;
        }
        t.x = dyv.x + G[0];
        G[0] = (cut >> j) & 1u ? 0.0f : a.x * t.x;
      }
      const float2 arm = mul2(mul2(a, rm), two(-1.0f));
      const float2 E = mul2(mul2(mul2(t, a), sr), fma2(arm, sx, hb[m]));
      const float2 tm = mul2(t, mul2(u, rm));
      const float2 ox = mul2(tm, si);
      const float2 oi = mul2(mul2(tm, sx), fma2(si, two(-1.0f), two(1.0f)));
      const float2 orr = mul2(mul2(k2, E), fma2(sr, two(1.0f), two(-1.0f)));
      if constexpr (VEC == 2) {
        sum[0] += E.x, sum[1] += E.y;
      } else {
        sum[0] += E.x;
        if (j + 1 < n) sum[0] += E.y;
      }
#pragma unroll
      for (int d = 0; d < per; ++d) {
        float px[VEC], pr[VEC], pi[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          px[v] = d + v ? ox.y : ox.x;
          pr[v] = d + v ? orr.y : orr.x;
          pi[v] = d + v ? oi.y : oi.x;
        }
        if (j + d < n && DLR_IN(t0 + j + d, q.L)) {
          put<T, VEC, kOne>(xp + (j + d) * dx.st, px, on);
          put<T, VEC, kOne>(rp + (j + d) * dr.st, pr, on);
          put<T, VEC, kOne>(ip + (j + d) * di.st, pi, on);
        }
      }
    }
    __syncthreads();  // back_s has been read
#pragma unroll
    for (int v = 0; v < VEC; ++v) back_s[warp][lane * VEC + v] = sum[v];
    __syncthreads();
    if (warp == 0)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) t += back_s[w][lane * VEC + v];
        if (on[v]) part[row + v] = t;
      }
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
  const gate2 g = make_gate2(two(to_f(r.row(b, 0)[ch])), two(to_f(i.row(b, 0)[ch])), two(kz));
  const float bt = g.m.x * g.si.x * to_f(x.row(b, 0)[ch]);
  const float s = reset && reset[b] ? bt : fmaf(g.a.x, h[k], bt);
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

// Bytes of the parts of a workspace for tiles of `steps` steps: the chain's counter and flags (for
// the narrowest groups, of 32 channels), the maps and the entering values.
struct Space {
  int64_t tiles;
  size_t head, maps, in;
  Space(int64_t B, int64_t L, int64_t H, int64_t steps) : tiles(L < 1 ? 0 : (L - 1) / steps + 1) {
    const size_t rows = (size_t)B * (size_t)tiles;
    head = align256(4 * (kHead + rows * (size_t)((H + 31) / 32)));
    maps = align256(sizeof(float2) * rows * (size_t)H);
    in = align256(sizeof(float) * rows * (size_t)H);
  }
};

// the widest access of `n` bytes that a view's rows allow
template <typename V>
bool wide(const V& v, int64_t size, uintptr_t n) {
  return ((reinterpret_cast<uintptr_t>(v.data) | (uintptr_t)(v.stride_b * size) |
           (uintptr_t)(v.stride_t * size)) & (n - 1)) == 0;
}

template <typename T, typename A>
Job<T> make_job(const A& a, const Space& sp) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const int64_t groups = (a.H + 32 * kVec<T> - 1) / (32 * kVec<T>);
  return {in_view<T>(a.x), in_view<T>(a.r), in_view<T>(a.i), a.p, a.reset,
          reinterpret_cast<float*>(ws + sp.head + sp.maps), reinterpret_cast<float2*>(ws + sp.head),
          reinterpret_cast<uint32_t*>(ws), device_status_word(), a.B, a.L, a.H, a.B * groups,
          (int)groups, (int)sp.tiles, (float)a.c};
}

// Blocks for `tiles` tiles: what the GPU holds at once at most. A chain of one tile needs no
// counter and takes a block for each.
template <typename T>
cudaError_t prepare_chain(const Job<T>& q, int per_sm, unsigned* blocks, cudaStream_t s) {
  const int64_t all = q.chains * q.tiles;
  *blocks = (unsigned)all;
  if (q.tiles == 1) return cudaSuccess;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  *blocks = (unsigned)std::min<int64_t>(all, (int64_t)sms * per_sm);
  return cudaMemsetAsync(q.head, 0, 4 * (size_t)(kHead + all), s);
}

template <typename T, int kBytes>
cudaError_t scan_w(const glr_scan_args& a, cudaStream_t s) {
  constexpr size_t smem = 2 * 3 * kScanTile * 128;
  const Job<T> q = make_job<T>(a, Space(a.B, a.L, a.H, kScanTile));
  unsigned blocks;
  cudaError_t e = prepare_chain(q, kScanBlocks, &blocks, s);
  if (e == cudaSuccess) e = max_smem_once<scan_kernel<T, kBytes>>(smem);
  if (e != cudaSuccess) return e;
  scan_kernel<T, kBytes><<<blocks, kScanWarps * 32, smem, s>>>(q, out_view<T>(a.y), a.h0, a.h_last,
                                                               a.states);
  return cudaGetLastError();
}

template <typename T, int kBytes>
cudaError_t back_w(const glr_scan_backward_args& a, cudaStream_t s) {
  constexpr size_t smem = 2 * 4 * kBackTile * 128;
  const Space sp(a.B, a.L, a.H, kBackTile);
  const Job<T> q = make_job<T>(a, sp);
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + sp.head + sp.maps +
                                         sp.in);
  unsigned blocks;
  cudaError_t e = prepare_chain(q, kBackBlocks, &blocks, s);
  if (e == cudaSuccess) e = max_smem_once<back_kernel<T, kBytes>>(smem);
  if (e != cudaSuccess) return e;
  back_kernel<T, kBytes><<<blocks, kBackWarps * 32, smem, s>>>(
      q, in_view<T>(a.dy), a.states, a.dh_last, out_view<T>(a.dx), out_view<T>(a.dr),
      out_view<T>(a.di), a.dh0, part);
  back_sum<<<(unsigned)((a.H + 31) / 32), 256, 0, s>>>(part, a.B * q.tiles, a.H, a.p, (float)a.c,
                                                       a.dp);
  return cudaGetLastError();
}

template <typename T>
cudaError_t scan_t(const glr_scan_args& a, cudaStream_t s) {
  const int64_t z = sizeof(T);
  auto all = [&](int64_t n) {
    return a.H * z % n == 0 && wide(a.x, z, n) && wide(a.r, z, n) && wide(a.i, z, n) &&
           wide(a.y, z, n);
  };
  if (all(16)) return scan_w<T, 16>(a, s);
  if (sizeof(T) == 4 || all(4)) return scan_w<T, 4>(a, s);
  if constexpr (sizeof(T) == 2) return scan_w<T, 2>(a, s);
}
template <typename T>
cudaError_t back_t(const glr_scan_backward_args& a, cudaStream_t s) {
  const int64_t z = sizeof(T);
  auto all = [&](int64_t n) {
    return a.H * z % n == 0 && wide(a.x, z, n) && wide(a.r, z, n) && wide(a.i, z, n) &&
           wide(a.dy, z, n) && wide(a.dx, z, n) && wide(a.dr, z, n) && wide(a.di, z, n);
  };
  if (all(16)) return back_w<T, 16>(a, s);
  if (sizeof(T) == 4 || all(4)) return back_w<T, 4>(a, s);
  if constexpr (sizeof(T) == 2) return back_w<T, 2>(a, s);
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
  const Space sp(B, L, H, kScanTile);
  return sp.head + sp.maps + sp.in;
}
size_t scan_backward_workspace_bytes(int64_t B, int64_t L, int64_t H) {
  const Space sp(B, L, H, kBackTile);
  return sp.head + sp.maps + 2 * sp.in;
}
// tiles (which a 32-bit counter hands out) of the finest cut that a call of this size takes
int64_t scan_tiles(int64_t B, int64_t L, int64_t H) {
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
