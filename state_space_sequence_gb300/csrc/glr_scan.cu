// glr_scan.cu -- the gated linear recurrence of include/glr.h: h_t = abar_t h_{t-1} + b_t per
// channel with a decay that the token chooses, its gradients, and one token from a carried state.
//
// A stretch of steps maps the state before it to the state after it by h -> A h + e, A the product
// of its decays and e its end state from zero; stretches compose in the same form. The gradients
// run backwards in time with G_t = dy_t + abar_{t+1} G_{t+1}: a stretch maps the gradient that
// enters behind it to the one that leaves before it by G -> A G + C with the same A.
//
// Each direction is one kernel that reads every input once from memory; before it goes a clearing
// of the chains' workspace, where a row is more than one tile, and after the gradients' a small
// kernel that adds up the parts of dp. Blocks stay on the GPU and take tiles (some steps of a group of channels) in turn; while a block works on one tile, the next
// one's inputs come into shared memory by asynchronous copies. Each warp takes S of a tile's steps,
// its gates in registers; the warps' maps meet in shared memory, the tiles of a row in a chain
// through global memory: a tile publishes its map, looks back over the maps of the tiles before it
// to the nearest one whose end value is there, and publishes its own end value. End values are
// always formed in the same order (each from the one before it), so the results do not depend on
// which of them a tile found. A tile that begins a sequence knows its end from its own steps.
//
// What bounds it: four arrays go through memory forwards and seven backwards, but in 16 bits the 4
// and 7 special functions and some 41 and 72 instructions an element weigh as much. B4 L16384 H2048
// bfloat16 takes 231 us forwards (4.6 TB/s, 69% of a plain copy's bandwidth) and 412 us backwards
// (4.6 TB/s), and 3 and 1 us less with the chain left out; at L2048 the counters show half of the
// issue slots used, the special-function pipe at 21%, and the rest of the time waits between a
// tile's two phases, which all warps of the one block on an SM go through together. Two smaller
// blocks on an SM (6 computing warps each: 297 and 612 us), 12 warps (248 and 415 us) or one
// reciprocal for both gates (241 and 425 us) were slower than the 233 and 415 us of their time. In
// float32 memory bounds it: B1 L4096 H4096 52 and 81 us (75% and 85%). Where a row of tiles is long
// and there are few, a tile's turn on its chain does: B1 L65536 H256 float32 92 us (43%; 46 us with
// the chain left out).
#include <algorithm>

#include "glr_common.cuh"
#include "tc_ptx.cuh"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 16;

int* device_status_word();

namespace glr {
namespace {

// Words of the chain's workspace before the maps; the first counts tickets.
constexpr int kHead = 64;

// Every word of the chain's workspace begins with these bits, a NaN that no arithmetic makes: a
// float that reads otherwise has been published. One 32-bit store publishes one float, so readers
// need neither flags nor fences. With flags, a tile's two fences and the flag's own way made B4
// L2048 H2048 bfloat16 take 56 us where it took 48 us so.
constexpr uint32_t kEmpty = 0xffffffffu;
constexpr uint64_t kWaitNs = 1000ull * 1000ull * 1000ull;  // a longer wait is a fault

__device__ __forceinline__ bool empty(float v) { return __float_as_uint(v) == kEmpty; }
__device__ __forceinline__ float full(float v) {  // any NaN but that one
  return empty(v) ? __uint_as_float(0x7fffffffu) : v;
}
// N neighbouring floats (each a store or load of its own to other threads)
template <int N>
__device__ __forceinline__ void post(float* p, const float (&v)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "one access");
  if constexpr (N == 1)
    asm volatile("st.relaxed.gpu.global.f32 [%0], %1;" ::"l"(p), "f"(full(v[0])) : "memory");
  else if constexpr (N == 2)
    asm volatile("st.relaxed.gpu.global.v2.f32 [%0], {%1, %2};" ::"l"(p), "f"(full(v[0])),
                 "f"(full(v[1]))
                 : "memory");
  else
    asm volatile("st.relaxed.gpu.global.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(full(v[0])),
                 "f"(full(v[1])), "f"(full(v[2])), "f"(full(v[3]))
                 : "memory");
}
template <int N>
__device__ __forceinline__ void look(const float* p, float (&v)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "one access");
  if constexpr (N == 1)
    asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v[0]) : "l"(p) : "memory");
  else if constexpr (N == 2)
    asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v[0]), "=f"(v[1])
                 : "l"(p)
                 : "memory");
  else
    asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ uint64_t timer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// What the two directions share. A chain is the row of tiles of one batch entry and group of 32 VEC
// channels. The channels of `in` and `maps` are padded to whole groups.
template <typename T>
struct Job {
  view<const T> x, r, i;
  const float* p;
  const uint8_t* reset;
  float* in;    // [B, tiles, HP]: the value that enters each tile but the chain's first
  float* maps;  // [B, tiles, HP / VEC, 2, VEC]: each tile's map, VEC of A and VEC of e
  float* run_in;    // [B, runs, HP]: with runs, the value that enters each but the first
  float* run_maps;  // [B, runs, HP / VEC, 2, VEC]: and its map
  uint32_t* head;
  int* status;
  int64_t B, L, H, HP, chains;
  int groups, tiles;
  int runs;  // runs of a chain (0: none)
  int most;  // tiles that a block takes at most
  float c;

  // the k-th tile of this block; called by one thread
  __device__ __forceinline__ uint32_t ticket(int k) const {
    if (tiles == 1) return k == 0 ? blockIdx.x : 0xffffffffu;
    return k < most ? atomicAdd(head, 1u) + 1u : 0xffffffffu;
  }
};

// Descriptions of arrays [B, L, H] for the tensor copies.
template <int N>
struct Maps {
  CUtensorMap map[N];
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

// s through a map (A, e): A s + e
template <int VEC>
__device__ __forceinline__ void through(const float (&A)[VEC], const float (&e)[VEC],
                                        float (&s)[VEC]) {
  if constexpr (VEC == 2) {
    const float2 t = fma2(make_float2(A[0], A[1]), make_float2(s[0], s[1]),
                          make_float2(e[0], e[1]));
    s[0] = t.x, s[1] = t.y;
  } else {
    s[0] = fmaf(A[0], s[0], e[0]);
  }
}
template <int N>
__device__ __forceinline__ bool any_empty(const float (&v)[N]) {
  bool is = false;
#pragma unroll
  for (int k = 0; k < N; ++k) is |= empty(v[k]);
  return __any_sync(0xffffffffu, is);
}

// The limit of a chain's waits.
struct Patience {
  uint64_t t0 = 0;
  bool gone = false;
  __device__ __forceinline__ bool ends() {  // called by whole warps
    const uint64_t t = timer_ns();
    if (t0 == 0) t0 = t;
    gone = __any_sync(0xffffffffu, t - t0 > kWaitNs);
    return gone;
  }
};

// Called by one warp: the value s that enters the tile, and `end`, the one that leaves it, from the
// tile's map (A, e); `cut`: the map does not depend on what enters. row: the lane's first element
// of `in`; dir = 1 forwards, -1 backwards. The first tile of the chain has its s.
//
// Each lane looks at one of the 32 tiles before this one, at the group's first channel, for the
// nearest whose end value is there with all maps between there too; the first tile of a chain
// always comes to its end value by itself. With the same loads comes the end value of the tile just
// before for the lane's own channels, which many chains side by side mostly find; else that end
// value and the maps are read then.
template <int VEC, typename J>
__device__ __forceinline__ void chain(const J& q, const Tile& at, int64_t row, int dir,
                                      const float (&A)[VEC], const float (&e)[VEC], bool cut,
                                      float (&s)[VEC], float (&end)[VEC]) {
  // maps read at a time: 8 against 4 is 90 against 94 us at B1 L65536 H256 f32; 8 pairs of
  // channels want too many registers (B8 L4096 H256 bf16: 24.3 against 23.6 us)
  constexpr int U = VEC == 1 ? 8 : 4;
  const int lane = threadIdx.x & 31;
  const int done = dir > 0 ? at.tile : q.tiles - 1 - at.tile;  // tiles of the chain before this
  const bool last = done == q.tiles - 1;
  const int64_t step = dir * q.HP;
  if (done > 0) {
    float m[2 * VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) m[v] = A[v], m[VEC + v] = e[v];
    const int64_t all = q.B * q.tiles * q.HP;
    if (!last && cut && DLR_IN(row + step + VEC - 1, all)) post(q.in + row + step, e);
    if (!last && !cut && DLR_IN(row + VEC - 1, all)) post(q.maps + 2 * row, m);
    const float* in = q.in + row;                   // the end of the tile before
    const float* maps = q.maps + 2 * (row - step);  // of the one before
    Patience wait;
    int far = 0;           // maps between the nearest end and this tile
    bool at_hand = false;  // none, and s has been read
    for (bool found = false; !found;) {
      const int k = far + lane;
      float has_end[1] = {0.0f}, has_map[1] = {0.0f};
      if (k < done) {
        look(in - lane * VEC - k * step, has_end);
        look(maps - 2 * (lane * VEC + k * step), has_map);
      }
      if (far == 0) look(in, s);
      const uint32_t ends = __ballot_sync(0xffffffffu, k < done && !empty(has_end[0]));
      const uint32_t there = __ballot_sync(0xffffffffu, k < done && !empty(has_map[0]));
      const int l = ends ? __ffs(ends) - 1 : 32;
      const uint32_t before = l == 32 ? 0xffffffffu : (1u << l) - 1u;
      if ((there & before) != before) {
        if (wait.ends()) break;
        continue;
      }
      far += l;
      found = l < 32;
      if (far == 0) at_hand = !any_empty(s);
    }
    // the end value with the first maps, then the others
    for (int k = far - 1; !at_hand; k -= U) {
      float t[U][2 * VEC], first[VEC];
      bool is;
      do {
        is = false;
        if (k == far - 1) look(in - far * step, first);
#pragma unroll
        for (int u = 0; u < U; ++u)
          look(maps - 2 * max(k - u, 0) * step, t[u]);
        if (k == far - 1)
#pragma unroll
          for (int v = 0; v < VEC; ++v) is |= empty(first[v]);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (k >= u)
#pragma unroll
            for (int v = 0; v < 2 * VEC; ++v) is |= empty(t[u][v]);
      } while (__any_sync(0xffffffffu, is) && !wait.ends());
      if (k == far - 1)
#pragma unroll
        for (int v = 0; v < VEC; ++v) s[v] = first[v];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k < u) continue;
        float a[VEC], b[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) a[v] = t[u][v], b[v] = t[u][VEC + v];
        through<VEC>(a, b, s);
      }
      at_hand = k < U;
    }
    if (wait.gone && lane == 0) report_status(q.status, DLR_ERR_TIMEOUT);
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) end[v] = s[v];
  through<VEC>(A, e, end);
  if (cut)
#pragma unroll
    for (int v = 0; v < VEC; ++v) end[v] = e[v];
  if (!last && !(done > 0 && cut) && DLR_IN(row + step, q.B * q.tiles * q.HP))
    post(q.in + row + step, end);
}

// The warps' maps of a tile, (A, e) of all its channels each, folded in shared memory's order by
// the chain's warp: the tile's map, and the value that enters each warp's steps.
template <int W, int VEC>
struct Fold {
  float A[W][VEC], e[W][VEC];
  uint32_t cut;
  template <int C>
  __device__ __forceinline__ void read(const float (&map)[W][2][C], uint32_t cuts) {
    const int lane = threadIdx.x & 31;
    cut = cuts;
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        A[w][v] = map[w][0][lane * VEC + v];
        e[w][v] = map[w][1][lane * VEC + v];
      }
  }
  __device__ __forceinline__ void advance(int w, float (&s)[VEC]) const {
    through<VEC>(A[w], e[w], s);
    if (cut && (cut >> w) & 1u)
#pragma unroll
      for (int v = 0; v < VEC; ++v) s[v] = e[w][v];
  }
  // the whole tile's map, from the first warp on or from the last
  __device__ __forceinline__ void all(bool backwards, float (&a)[VEC], float (&b)[VEC]) const {
#pragma unroll
    for (int v = 0; v < VEC; ++v) a[v] = 1.0f, b[v] = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      advance(backwards ? W - 1 - k : k, b);
      if constexpr (VEC == 2) {
        const float2 t = mul2(make_float2(a[0], a[1]), make_float2(A[k][0], A[k][1]));
        a[0] = t.x, a[1] = t.y;
      } else {
        a[0] *= A[k][0];
      }
    }
  }
};

// As chain(), for few chains, of which many tiles are at work at a time, in runs of kRun tiles: the
// last tile of a run publishes the map of the whole run, and later the value that enters the next
// run. A tile takes the value that enters its own run, looking back over runs, through the maps of
// its run's tiles before it. A map that does not depend on what enters has kCut for its A.
constexpr uint32_t kCut = 0xfffffffeu;
constexpr int kRun = 8;
template <int VEC>
__device__ __forceinline__ void through_cut(const float (&m)[2 * VEC], float (&s)[VEC]) {
  float a[VEC], b[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) a[v] = m[v], b[v] = m[VEC + v];
  through<VEC>(a, b, s);
  if (__float_as_uint(m[0]) == kCut)  // the same for all channels
#pragma unroll
    for (int v = 0; v < VEC; ++v) s[v] = m[VEC + v];
}
template <int VEC, typename J>
__device__ __forceinline__ void chain_runs(const J& q, const Tile& at, int64_t row, int dir,
                                           const float (&A)[VEC], const float (&e)[VEC], bool cut,
                                           float (&s)[VEC], float (&end)[VEC]) {
  constexpr int U = 4;
  const int lane = threadIdx.x & 31;
  const int done = dir > 0 ? at.tile : q.tiles - 1 - at.tile;  // tiles of the chain before this
  const bool last = done == q.tiles - 1;
  const int run = done / kRun, j = done % kRun;
  const bool closes = j == kRun - 1 && !last;
  const int64_t step = dir * q.HP, all = q.B * q.tiles * q.HP;
  // runs in the chain's order: their maps, and the values that enter them
  const int64_t h = row - ((int64_t)at.b * q.tiles + at.tile) * q.HP;
  const int64_t mine = ((int64_t)at.b * q.runs + run) * q.HP + h;
  float m[2 * VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) m[v] = cut ? __uint_as_float(kCut) : A[v], m[VEC + v] = e[v];
  if (!last && !closes && DLR_IN(row + VEC - 1, all)) post(q.maps + 2 * row, m);
  Patience wait;
  // the maps of the run's tiles before this one, the first of them first
  float t[kRun - 1][2 * VEC];
  const float* from = q.maps + 2 * (row - j * step);
  uint32_t top;
  do {
    top = 0;
#pragma unroll
    for (int u = 0; u < kRun - 1; ++u)
      if (u < j) {
        look(from + 2 * u * step, t[u]);
      }
#pragma unroll
    for (int u = 0; u < kRun - 1; ++u)
      if (u < j)
#pragma unroll
        for (int v = 0; v < 2 * VEC; ++v) top = max(top, __float_as_uint(t[u][v]));
  } while (__any_sync(0xffffffffu, top == kEmpty) && !wait.ends());
  float whole[2 * VEC];
  if (closes) {
    float a[VEC], b[VEC];
    bool any = cut;
#pragma unroll
    for (int v = 0; v < VEC; ++v) a[v] = 1.0f, b[v] = 0.0f;
#pragma unroll
    for (int u = 0; u < kRun - 1; ++u)
      if (u < j) {
        through_cut<VEC>(t[u], b);
        any |= __float_as_uint(t[u][0]) == kCut;
#pragma unroll
        for (int v = 0; v < VEC; ++v) a[v] *= t[u][v];
      }
    through_cut<VEC>(m, b);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      whole[v] = any ? __uint_as_float(kCut) : a[v] * m[v];
      whole[VEC + v] = b[v];
    }
    if (DLR_IN(mine + VEC - 1, q.B * q.runs * q.HP)) post(q.run_maps + 2 * mine, whole);
  }
  if (run > 0) {
    const float* in = q.run_in + mine;                    // the value that enters this run
    const float* maps = q.run_maps + 2 * (mine - q.HP);   // the run before
    int far = 0;
    bool at_hand = false;
    for (bool found = false; !found;) {
      const int k = far + lane;
      float has_in[1] = {0.0f}, has_map[1] = {0.0f};
      if (k < run) {
        look(in - lane * VEC - k * q.HP, has_in);
        look(maps - 2 * (lane * VEC + k * q.HP), has_map);
      }
      if (far == 0) look(in, s);
      const uint32_t ins = __ballot_sync(0xffffffffu, k < run && !empty(has_in[0]));
      // what leaves the first run is waited for, not its map, so that the look stops there
      const uint32_t there = __ballot_sync(0xffffffffu, k < run - 1 && !empty(has_map[0]));
      const int l = ins ? __ffs(ins) - 1 : 32;
      const uint32_t before = l == 32 ? 0xffffffffu : (1u << l) - 1u;
      if ((there & before) != before) {
        if (wait.ends()) break;
        continue;
      }
      far += l;
      found = l < 32;
      if (far == 0) at_hand = !any_empty(s);
    }
    for (int k = far - 1; !at_hand; k -= U) {
      float g[U][2 * VEC], first[VEC];
      do {
        top = 0;
        if (k == far - 1) {
          look(in - far * q.HP, first);
#pragma unroll
          for (int v = 0; v < VEC; ++v) top = max(top, __float_as_uint(first[v]));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) look(maps - 2 * max(k - u, 0) * q.HP, g[u]);
        if (k >= 0)
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int v = 0; v < 2 * VEC; ++v) top = max(top, __float_as_uint(g[u][v]));
      } while (__any_sync(0xffffffffu, top == kEmpty) && !wait.ends());
      if (k == far - 1)
#pragma unroll
        for (int v = 0; v < VEC; ++v) s[v] = first[v];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (k >= u) through_cut<VEC>(g[u], s);
      at_hand = k < U;
    }
  }
  if (closes) {
    float next[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) next[v] = s[v];
    through_cut<VEC>(whole, next);
    if (DLR_IN(mine + q.HP + VEC - 1, q.B * q.runs * q.HP)) post(q.run_in + mine + q.HP, next);
  }
#pragma unroll
  for (int u = 0; u < kRun - 1; ++u)
    if (u < j) through_cut<VEC>(t[u], s);
  if (wait.gone && lane == 0) report_status(q.status, DLR_ERR_TIMEOUT);
#pragma unroll
  for (int v = 0; v < VEC; ++v) end[v] = s[v];
  through_cut<VEC>(m, end);
}

// How many steps each of a tile's W warps has: S, or what the row's end leaves of them. The
// supplying warp writes the counts beside the tile's place and the computing warps read them there.
// A warp's padding, its maps, its sums and its stores all go by that one number, which a compiler
// cannot form again from the tile's place at one of them. In a draft each warp formed its own in
// 32-bit arithmetic; its padding went by the right count and its stores by S, past the row's end.
// Reading the source did not show why.
template <int W, int S, typename J>
__device__ __forceinline__ void write_steps(const J& q, const Tile& at, int (&steps)[W]) {
  const int lane = threadIdx.x & 31;
  if (lane >= W) return;
  const int64_t left = q.L - ((int64_t)at.tile * W + lane) * S;
  steps[lane] = at.tile < 0 ? 0 : (int)max((int64_t)0, min((int64_t)S, left));
}

// bits of the n steps from t on that begin a sequence
__device__ __forceinline__ uint32_t cuts(const uint8_t* reset, int64_t first, int n) {
  if (!reset) return 0u;
  const int lane = threadIdx.x & 31;
  return __ballot_sync(0xffffffffu, lane < n && reset[first + lane] != 0);
}

// A decay in one register with its digits both next to 1 and next to 0: a - 1 (negative; -0 for
// a = 1) where a > 1/2, else a.
__device__ __forceinline__ float2 keep_decay(float2 a, float2 rest) {
  return make_float2(a.x > 0.5f ? -rest.x : a.x, a.y > 0.5f ? -rest.y : a.y);
}
__device__ __forceinline__ float2 sign_ones(float2 k) {
  return make_float2(__float_as_int(k.x) < 0 ? 1.0f : 0.0f, __float_as_int(k.y) < 0 ? 1.0f : 0.0f);
}
__device__ __forceinline__ float2 kept_decay(float2 k) { return add2(k, sign_ones(k)); }

// A warp's S steps of VEC channels a lane are S VEC / 2 pairs: the two channels of a step, or, with
// one channel to a lane, two steps. half(): step j of channel v.
template <int VEC, int N>
__device__ __forceinline__ float& half(float2 (&p)[N], int j, int v) {
  if constexpr (VEC == 2) return v ? p[j].y : p[j].x;
  return j & 1 ? p[j / 2].y : p[j / 2].x;
}
// pair m of the rows [.][C] at p
template <typename T, int VEC, int C>
__device__ __forceinline__ float2 get2(const T* p, int m) {
  if constexpr (VEC == 2) return unpack2<T>(*reinterpret_cast<const uint32_t*>(p + m * C));
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

// How a tile's inputs come into shared memory and its outputs leave it. Where every row begins on a
// 16-byte boundary and H is a whole number of 16 bytes, one thread has a whole tile moved by a
// tensor copy (kTma), which also fills what a tile has past the ends with zeros and leaves it out
// on the way back; describing an array to it costs the host some 0.1 us. Else the computing warps
// copy 4 bytes at a time, or single elements where not even 4-byte boundaries hold (16-bit types
// with odd strides), and store for themselves.
constexpr int kTma = 16;

__device__ __forceinline__ void copy_async(void* dst, const void* src, bool on) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  const int n = on ? 4 : 0;  // nothing is read and zeros are written where off
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void copies_end() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// kSteps rows of C channels of v into dst [kSteps][C], by kThreads threads; rows past the end and
// channels past H are zero
template <typename T, int C, int kSteps, int kBytes, int kThreads>
__device__ __forceinline__ void stage(T* dst, const view<const T>& v, int64_t b, int64_t t0,
                                      int64_t h0, int64_t L, int64_t H) {
  constexpr int per = kBytes / (int)sizeof(T), cols = C / per, rows = kThreads / cols;
  static_assert(kSteps % rows == 0, "whole turns");
  const int col = threadIdx.x % cols * per, first = threadIdx.x / cols;
  const T* p = v.row(b, t0 + first) + h0 + col;
  const int64_t dp = rows * v.st;
  dst += first * C + col;
  if (kBytes != 2 && t0 + kSteps <= L && h0 + C <= H) {
#pragma unroll
    for (int j = 0; j < kSteps; j += rows, p += dp) copy_async(dst + j * C, p, true);
    return;
  }
  const bool in = h0 + col < H;
#pragma unroll 4
  for (int j = 0; j < kSteps; j += rows, p += dp) {
    const bool on = in && t0 + first + j < L;
    if constexpr (kBytes == 2)
      dst[j * C] = on ? *p : from_f<T>(0.0f);
    else
      copy_async(dst + j * C, on ? p : v.p, on);
  }
}

// Named barriers: a warp that only arrives does not wait.
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// VEC neighbouring values to memory: at once, or one by one where they are not aligned
template <typename T, int VEC, bool kOne>
__device__ __forceinline__ void put(T* p, const float (&f)[VEC], bool (&on)[VEC]) {
  if constexpr (kOne) {
#pragma unroll
    for (int v = 0; v < VEC; ++v)
      if (on[v]) p[v] = from_f<T>(f[v]);
  } else {
    words<T, VEC> o;
    o.from(f);
    if (on[0]) o.put(p);
  }
}

// Channels of a lane: a warp's row of a tile is 128 bytes.
template <typename T>
constexpr int kVec = 4 / (int)sizeof(T);

constexpr int kScanSteps = 8;                        // of a warp
constexpr int kScanWarps = 14;                       // that compute; two more serve them
constexpr int kScanTile = kScanSteps * kScanWarps;   // steps
constexpr int kScanThreads = 32 * (kScanWarps + 2);
constexpr int kRing = 8;                             // tiles whose places a block remembers

// Named barriers of a block, two of each kind for even and odd tiles: the maps of a tile are in
// shared memory (the computing warps arrive, the chain's warp waits); the values that enter its
// warps are there (the chain's warp arrives, all others wait); and two for the beginning.
constexpr int kMapsBar = 1, kEnterBar = 3, kWarpsBar = 5;

template <typename T>
struct ScanShared {
  static constexpr int C = 32 * kVec<T>;
  T buf[2][3][kScanTile][C];        // r, i, x of two tiles
  T out[kScanTile][C];
  float map[3][kScanWarps][2][C];   // A and e of each warp's steps
  float enter[2][kScanWarps][C];    // the state that enters them
  float kz[kRing][C];
  int steps[kRing][kScanWarps];     // that there are of each warp's
  uint32_t cut[3][kScanWarps];
  Tile tile[kRing];
  uint64_t here[2];                 // barriers of the buffers' copies
};

// One warp keeps the chain and one supplies the tiles; the others compute, one tile ahead of the
// chain: they have the gates of tile k + 1 done before they need the state that enters tile k, so a
// tile's way along the chain (stores and loads through L2) passes while they work. A tile is 14
// warps of 8 steps: with the gates of two tiles in registers (64 of them) 16 warps fill the
// register file.
template <typename T, int kBytes, bool kRuns>
__global__ void __launch_bounds__(kScanThreads, 1)
scan_kernel(Job<T> q, const __grid_constant__ Maps<3> in, const __grid_constant__ Maps<1> out,
            view<T> y, const float* __restrict__ h0, float* __restrict__ h_last,
            float* __restrict__ states) {
  constexpr int VEC = kVec<T>, W = kScanWarps, S = kScanSteps, C = 32 * VEC, NP = S * VEC / 2;
  constexpr int kWork = 32 * W;
  constexpr bool kOne = kBytes == 2, kBulk = kBytes == kTma;
  extern __shared__ __align__(128) uint8_t smem[];
  ScanShared<T>& sh = *reinterpret_cast<ScanShared<T>*>(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  if (warp == W + 1) {
    auto take = [&](int k) {  // the place of the block's k-th tile
      const uint32_t t = lane == 0 ? q.ticket(k) : 0u;
      const Tile at = tile_of(q, __shfl_sync(0xffffffffu, t, 0), false);
      if (lane == 0) sh.tile[k % kRing] = at;
      __syncwarp();
    };
    auto params = [&](int k) {  // its steps and decay parameters
      const Tile at = sh.tile[k % kRing];
      write_steps<W, S>(q, at, sh.steps[k % kRing]);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const int64_t h = ((int64_t)at.group * 32 + lane) * VEC + v;
        sh.kz[k % kRing][lane * VEC + v] =
            at.tile >= 0 && h < q.H ? -q.c * softplus(q.p[h]) * kLog2e : 0.0f;
      }
    };
    auto copy = [&](int k) {
      const Tile at = sh.tile[k % kRing];
      if (!kBulk || at.tile < 0 || lane != 0) return;
      tc::mbar_arrive_expect_tx(&sh.here[k & 1], sizeof(sh.buf[0]));
#pragma unroll
      for (int a = 0; a < 3; ++a)
        tc::tma_load_3d(&sh.buf[k & 1][a][0][0], &in.map[a], at.group * C, at.tile * kScanTile,
                        at.b, &sh.here[k & 1]);
    };
    if (lane == 0) {
      tc::mbar_init(&sh.here[0], 1);
      tc::mbar_init(&sh.here[1], 1);
      tc::mbar_fence_init();
    }
    for (int k = 0; k < 3; ++k) {
      take(k);
      if (k < 2) copy(k);
      params(k);
    }
    __syncthreads();
    bar_sync(kWarpsBar, kWork + 32);
    copy(2);
    for (int k = 0; sh.tile[k % kRing].tile >= 0; ++k) {
      take(k + 3);
      params(k + 3);
      bar_sync(kEnterBar + (k & 1), kScanThreads);
      copy(k + 3);
    }
    return;
  }
  if (warp == W) {
    __syncthreads();
    for (int k = 0;; ++k) {
      bar_sync(kMapsBar + (k & 1), kWork + 32);
      const Tile at = sh.tile[k % kRing];
      if (at.tile < 0) return;
      const int64_t h = ((int64_t)at.group * 32 + lane) * VEC;
      const int64_t row = ((int64_t)at.b * q.tiles + at.tile) * q.HP + h;
      const uint32_t cut = __ballot_sync(0xffffffffu, lane < W && sh.cut[k % 3][lane % W] != 0);
      bool on[VEC];
      float A[VEC], e[VEC], s[VEC], end[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) on[v] = h + v < q.H && DLR_IN(at.b, q.B);
      Fold<W, VEC> fold;
      fold.read(sh.map[k % 3], cut);
      fold.all(false, A, e);
      if (at.tile < (kRuns ? kRun : 1))  // what enters the first tile, or the first run
#pragma unroll
        for (int v = 0; v < VEC; ++v) s[v] = h0 && on[v] ? h0[at.b * q.H + h + v] : 0.0f;
      if constexpr (kRuns)
        chain_runs(q, at, row, 1, A, e, cut != 0, s, end);
      else
        chain(q, at, row, 1, A, e, cut != 0, s, end);
#pragma unroll
      for (int w = 0; w < W; ++w) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) sh.enter[k & 1][w][lane * VEC + v] = s[v];
        fold.advance(w, s);
      }
      bar_arrive(kEnterBar + (k & 1), kScanThreads);
      if (at.tile == q.tiles - 1 && h_last)
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          if (on[v]) h_last[at.b * q.H + h + v] = end[v];
    }
  }

  auto fetch = [&](int k) {
    if constexpr (!kBulk) {
      const Tile at = sh.tile[k % kRing];
      if (at.tile >= 0) {
        const int64_t t0 = (int64_t)at.tile * kScanTile, c0 = (int64_t)at.group * C;
        auto& d = sh.buf[k & 1];
        stage<T, C, kScanTile, kBytes, kWork>(&d[0][0][0], q.r, at.b, t0, c0, q.L, q.H);
        stage<T, C, kScanTile, kBytes, kWork>(&d[1][0][0], q.i, at.b, t0, c0, q.L, q.H);
        stage<T, C, kScanTile, kBytes, kWork>(&d[2][0][0], q.x, at.b, t0, c0, q.L, q.H);
      }
      copies_end();
    }
  };
  struct Part {  // what a warp has of a tile: its steps, how many there are, which begin a sequence
    float2 a[NP] = {}, b[NP] = {};
    int n = 0;
    uint32_t cut = 0;
  };
  auto gates = [&](int k, Part& z) {
    const Tile at = sh.tile[k % kRing];
    z.n = sh.steps[k % kRing][warp];
    z.cut = 0;
    if (at.tile < 0) {
      bar_arrive(kMapsBar + (k & 1), kWork + 32);
      return;
    }
    const int64_t t0 = (int64_t)at.tile * kScanTile + warp * S;
    z.cut = cuts(q.reset, at.b * q.L + t0, z.n);
    const float* own = &sh.kz[k % kRing][lane * VEC];
    const float2 kz = make_float2(own[0], own[VEC - 1]);
    const T* r = &sh.buf[k & 1][0][warp * S][lane * VEC];
    if (kBulk && !tc::mbar_wait_sleep(&sh.here[k & 1], (k >> 1) & 1) && lane == 0)
      report_status(q.status, DLR_ERR_TIMEOUT);
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      gates2(get2<T, VEC, C>(r, m), get2<T, VEC, C>(r + kScanTile * C, m),
             get2<T, VEC, C>(r + 2 * kScanTile * C, m), kz, z.a[m], z.b[m]);
    }
    if (z.n < S) {
#pragma unroll
      for (int j = 0; j < S; ++j)
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          if (j >= z.n) half<VEC>(z.a, j, v) = 1.0f, half<VEC>(z.b, j, v) = 0.0f;
    }
    float A[VEC], e[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) A[v] = 1.0f, e[v] = 0.0f;
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      if constexpr (VEC == 2) {
        const float2 t = mul2(make_float2(A[0], A[1]), z.a[m]);
        A[0] = t.x, A[1] = t.y;
      } else {
        A[0] *= z.a[m].x * z.a[m].y;
      }
    }
    if (z.cut == 0) {
#pragma unroll
      for (int j = 0; j < S; ++j) advance<VEC>(e, z.a, z.b, j);
    } else {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        advance<VEC>(e, z.a, z.b, j);
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          if ((z.cut >> j) & 1u) e[v] = half<VEC>(z.b, j, v);
      }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      sh.map[k % 3][warp][0][lane * VEC + v] = A[v];
      sh.map[k % 3][warp][1][lane * VEC + v] = e[v];
    }
    if (lane == 0) sh.cut[k % 3][warp] = z.cut;
    bar_arrive(kMapsBar + (k & 1), kWork + 32);
  };
  auto finish = [&](int k, Part& z) {
    const Tile at = sh.tile[k % kRing];
    const int64_t h = ((int64_t)at.group * 32 + lane) * VEC;
    const int64_t t0 = (int64_t)at.tile * kScanTile + warp * S;
    bool on[VEC];
    float s[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      on[v] = h + v < q.H && DLR_IN(at.b, q.B);
      s[v] = sh.enter[k & 1][warp][lane * VEC + v];
    }
    if (states && z.n > 0) {
      const int64_t runs = (q.L - 1) / S + 1;
      float* to = states + (at.b * runs + t0 / S) * q.H + h;
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        if (on[v] && DLR_IN((at.b * runs + t0 / S) * q.H + h + v, q.B * runs * q.H)) to[v] = s[v];
    }
    T* yp = kBulk ? &sh.out[warp * S][lane * VEC] : y.row(at.b, t0) + h;
    const int64_t st = kBulk ? C : y.st;
    if (kBulk) {
      if (lane == 0) tc::bulk_wait_group_read0();  // the last tile's have left
      __syncwarp();
#pragma unroll
      for (int v = 0; v < VEC; ++v) on[v] = true;
    }
    if (z.cut == 0 && (kBulk || z.n == S)) {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        advance<VEC>(s, z.a, z.b, j);
        put<T, VEC, kOne>(yp + j * st, s, on);
      }
    } else {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        advance<VEC>(s, z.a, z.b, j);
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          if ((z.cut >> j) & 1u) s[v] = half<VEC>(z.b, j, v);
        if (j < z.n && DLR_IN(t0 + j, q.L)) put<T, VEC, kOne>(yp + j * st, s, on);
      }
    }
    if (kBulk && z.n > 0) {
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tc::tma_store_3d(&out.map[0], &sh.out[warp * S][0], at.group * C, (int)t0, at.b);
        tc::bulk_commit_group();
      }
    }
  };
  // tile k's gates are in `now`; true when it was the last
  auto turn = [&](int k, Part& now, Part& next) {
    gates(k + 1, next);
    if (!kBulk) copies_wait();
    bar_sync(kEnterBar + (k & 1), kScanThreads);
    fetch(k + 3);
    finish(k, now);
    const bool last = sh.tile[(k + 1) % kRing].tile < 0;
    if (kBulk && last && lane == 0) tc::bulk_wait_group0();
    return last;
  };
  Part z0, z1;
  __syncthreads();
  fetch(0);
  if (!kBulk) {
    copies_wait();
    bar_sync(kWarpsBar + 1, kWork);
  }
  fetch(1);
  gates(0, z0);
  if (!kBulk) copies_wait();
  bar_sync(kWarpsBar, kWork + 32);
  if (sh.tile[0].tile < 0) return;
  fetch(2);
  for (int k = 0;; k += 2) {
    if (turn(k, z0, z1)) return;
    if (turn(k + 1, z1, z0)) return;
  }
}

constexpr int kBackSteps = 8;
constexpr int kBackWarps = 14;
constexpr int kBackTile = kBackSteps * kBackWarps;
constexpr int kBackThreads = 32 * (kBackWarps + 2);
static_assert(kBackSteps == GLR_STATE_STEPS && kScanSteps == GLR_STATE_STEPS,
              "the forward pass keeps the state that enters a warp's steps");

template <typename T>
struct BackShared {
  static constexpr int C = 32 * kVec<T>;
  T rd[4][2][kBackTile][C];         // r, dy of four tiles; r's place takes dr
  T ix[2][2][kBackTile][C];         // i, x of two; they take di, dx
  float map[3][kBackWarps][2][C];   // A and C of each warp's steps
  float enter[2][kBackWarps][C];    // the gradient that enters behind them
  float sum[2][kBackWarps][C];      // their parts of dp
  float k[kRing][C];                // c softplus(p)
  int steps[kRing][kBackWarps];     // that there are of each warp's
  uint32_t cut[3][kBackWarps];
  Tile tile[kRing];
  uint64_t rd_here[4], ix_here[2];  // barriers of the buffers' copies
};

// As scan_kernel, backwards. One tile ahead of the chain the computing warps need r and dy only (a
// tile's map is made of the decays and dy), which come three tiles ahead; i and x come one ahead.
// With what enters known, a warp first goes back over its steps for G, then forwards from the
// kept state, so that each step's state is at hand when its gradients are formed: nothing is
// computed twice but sigmoid(r), and only the decays and G stay in registers.
template <typename T, int kBytes, bool kRuns>
__global__ void __launch_bounds__(kBackThreads, 1)
back_kernel(Job<T> q, const __grid_constant__ Maps<4> in, const __grid_constant__ Maps<3> out,
            view<const T> dy, const float* __restrict__ states, const float* __restrict__ dh_last,
            view<T> dx, view<T> dr, view<T> di, float* __restrict__ dh0, float* __restrict__ part) {
  constexpr int VEC = kVec<T>, W = kBackWarps, S = kBackSteps, C = 32 * VEC, NP = S * VEC / 2;
  constexpr int kWork = 32 * W;
  constexpr bool kOne = kBytes == 2, kBulk = kBytes == kTma;
  extern __shared__ __align__(128) uint8_t smem[];
  BackShared<T>& sh = *reinterpret_cast<BackShared<T>*>(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  if (warp == W + 1) {
    auto take = [&](int k) {  // the place of the block's k-th tile
      const uint32_t t = lane == 0 ? q.ticket(k) : 0u;
      const Tile at = tile_of(q, __shfl_sync(0xffffffffu, t, 0), true);
      if (lane == 0) sh.tile[k % kRing] = at;
      __syncwarp();
    };
    auto params = [&](int k) {  // its steps and decay parameters
      const Tile at = sh.tile[k % kRing];
      write_steps<W, S>(q, at, sh.steps[k % kRing]);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const int64_t h = ((int64_t)at.group * 32 + lane) * VEC + v;
        sh.k[k % kRing][lane * VEC + v] = at.tile >= 0 && h < q.H ? q.c * softplus(q.p[h]) : 0.0f;
      }
    };
    auto copy = [&](T* dst, uint64_t* here, int first, int k) {
      const Tile at = sh.tile[k % kRing];
      if (!kBulk || at.tile < 0 || lane != 0) return;
      tc::mbar_arrive_expect_tx(here, 2 * kBackTile * 128);
#pragma unroll
      for (int a = 0; a < 2; ++a)
        tc::tma_load_3d(dst + a * kBackTile * C, &in.map[first + a], at.group * C,
                        at.tile * kBackTile, at.b, here);
    };
    auto copy_rd = [&](int k) { copy(&sh.rd[k & 3][0][0][0], &sh.rd_here[k & 3], 0, k); };
    auto copy_ix = [&](int k) { copy(&sh.ix[k & 1][0][0][0], &sh.ix_here[k & 1], 2, k); };
    // the parts of dp of the block's k-th tile
    auto sums = [&](int k) {
      const Tile at = sh.tile[k % kRing];
      const int64_t h = ((int64_t)at.group * 32 + lane) * VEC;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) t += sh.sum[k & 1][w][lane * VEC + v];
        const int64_t to = ((int64_t)at.b * q.tiles + at.tile) * q.H + h + v;
        if (h + v < q.H && DLR_IN(to, q.B * q.tiles * q.H)) part[to] = t;
      }
    };
    if (lane == 0) {
      for (int k = 0; k < 4; ++k) tc::mbar_init(&sh.rd_here[k], 1);
      for (int k = 0; k < 2; ++k) tc::mbar_init(&sh.ix_here[k], 1);
      tc::mbar_fence_init();
    }
    for (int k = 0; k < 3; ++k) {
      take(k);
      copy_rd(k);
      if (k == 0) copy_ix(0);
      params(k);
    }
    __syncthreads();
    int k = 0;
    for (; sh.tile[k % kRing].tile >= 0; ++k) {
      take(k + 3);
      params(k + 3);
      bar_sync(kEnterBar + (k & 1), kBackThreads);  // all warps are done with tile k - 1
      copy_rd(k + 3);
      copy_ix(k + 1);
      if (k > 0) sums(k - 1);
    }
    bar_sync(kWarpsBar, kWork + 32);
    if (k > 0) sums(k - 1);
    return;
  }
  if (warp == W) {
    __syncthreads();
    for (int k = 0;; ++k) {
      bar_sync(kMapsBar + (k & 1), kWork + 32);
      const Tile at = sh.tile[k % kRing];
      if (at.tile < 0) return;
      const int64_t h = ((int64_t)at.group * 32 + lane) * VEC;
      const int64_t row = ((int64_t)at.b * q.tiles + at.tile) * q.HP + h;
      const uint32_t cut = __ballot_sync(0xffffffffu, lane < W && sh.cut[k % 3][lane % W] != 0);
      bool on[VEC];
      float A[VEC], e[VEC], s[VEC], end[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) on[v] = h + v < q.H && DLR_IN(at.b, q.B);
      Fold<W, VEC> fold;
      fold.read(sh.map[k % 3], cut);
      fold.all(true, A, e);
      if (q.tiles - 1 - at.tile < (kRuns ? kRun : 1))
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          s[v] = dh_last && on[v] ? dh_last[at.b * q.H + h + v] : 0.0f;
      if constexpr (kRuns)
        chain_runs(q, at, row, -1, A, e, cut != 0, s, end);
      else
        chain(q, at, row, -1, A, e, cut != 0, s, end);
#pragma unroll
      for (int w = W - 1; w >= 0; --w) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) sh.enter[k & 1][w][lane * VEC + v] = s[v];
        fold.advance(w, s);
      }
      bar_arrive(kEnterBar + (k & 1), kBackThreads);
      if (at.tile == 0 && dh0)
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          if (on[v]) dh0[at.b * q.H + h + v] = end[v];
    }
  }

  auto fetch = [&](T* dst, const view<const T>& v0, const view<const T>& v1, int k) {
    if constexpr (!kBulk) {
      const Tile at = sh.tile[k % kRing];
      if (at.tile < 0) return;
      const int64_t t0 = (int64_t)at.tile * kBackTile, c0 = (int64_t)at.group * C;
      stage<T, C, kBackTile, kBytes, kWork>(dst, v0, at.b, t0, c0, q.L, q.H);
      stage<T, C, kBackTile, kBytes, kWork>(dst + kBackTile * C, v1, at.b, t0, c0, q.L, q.H);
    }
  };
  auto fetch_rd = [&](int k) { fetch(&sh.rd[k & 3][0][0][0], q.r, dy, k); };
  auto fetch_ix = [&](int k) { fetch(&sh.ix[k & 1][0][0][0], q.i, q.x, k); };
  auto wait = [&](uint64_t* here, int parity) {
    if (kBulk && !tc::mbar_wait_sleep(here, parity) && lane == 0)
      report_status(q.status, DLR_ERR_TIMEOUT);
  };
  struct Part {  // what a warp has of a tile: its decays, its steps, which begin a sequence
    float2 ka[NP] = {};
    int n = 0;
    uint32_t cut = 0;
  };
  auto decays = [&](int k, Part& z) {
    const Tile at = sh.tile[k % kRing];
    z.n = sh.steps[k % kRing][warp];
    z.cut = 0;
    if (at.tile < 0) {
      bar_arrive(kMapsBar + (k & 1), kWork + 32);
      return;
    }
    const int64_t t0 = (int64_t)at.tile * kBackTile + warp * S;
    z.cut = cuts(q.reset, at.b * q.L + t0, z.n);
    const float* own = &sh.k[k % kRing][lane * VEC];
    const float2 kz = mul2(make_float2(own[0], own[VEC - 1]), two(-kLog2e));
    const T* r = &sh.rd[k & 3][0][warp * S][lane * VEC];
    wait(&sh.rd_here[k & 3], (k >> 2) & 1);
    float2 a[NP];
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      float2 rest;
      decay2(mul2(kz, sigmoid2(get2<T, VEC, C>(r, m))), rest, a[m]);
      z.ka[m] = keep_decay(a[m], rest);
    }
    if (z.n < S) {  // steps past the end pass the gradient through; their dy is zero
#pragma unroll
      for (int j = 0; j < S; ++j)
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          if (j >= z.n) half<VEC>(a, j, v) = 1.0f, half<VEC>(z.ka, j, v) = -0.0f;
    }
    float A[VEC], G[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) A[v] = 1.0f, G[v] = 0.0f;
    float2 d[NP];
#pragma unroll
    for (int m = 0; m < NP; ++m) d[m] = get2<T, VEC, C>(r + kBackTile * C, m);
#pragma unroll
    for (int j = S - 1; j >= 0; --j) {
      if constexpr (VEC == 2) {
        const float2 t = mul2(a[j], add2(d[j], make_float2(G[0], G[1])));
        G[0] = t.x, G[1] = t.y;
      } else {
        G[0] = half<VEC>(a, j, 0) * (half<VEC>(d, j, 0) + G[0]);
      }
      if (z.cut)
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          if ((z.cut >> j) & 1u) G[v] = 0.0f;
    }
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      if constexpr (VEC == 2) {
        const float2 t = mul2(make_float2(A[0], A[1]), a[m]);
        A[0] = t.x, A[1] = t.y;
      } else {
        A[0] *= a[m].x * a[m].y;
      }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      sh.map[k % 3][warp][0][lane * VEC + v] = A[v];
      sh.map[k % 3][warp][1][lane * VEC + v] = G[v];
    }
    if (lane == 0) sh.cut[k % 3][warp] = z.cut;
    bar_arrive(kMapsBar + (k & 1), kWork + 32);
  };
  // the state that enters the warp's steps of a tile
  auto kept = [&](int k, const Part& z, float (&s)[VEC]) {
    const Tile at = sh.tile[k % kRing];
    const int64_t h = ((int64_t)at.group * 32 + lane) * VEC;
    const int64_t t0 = (int64_t)at.tile * kBackTile + warp * S;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const int64_t runs = (q.L - 1) / S + 1, from = (at.b * runs + t0 / S) * q.H + h + v;
      s[v] = z.n > 0 && h + v < q.H && DLR_IN(from, q.B * runs * q.H) ? states[from] : 0.0f;
    }
  };
  // plain (a constant in each call): all S steps are there and none begins a sequence
  auto finish = [&](int k, Part& z, float (&s)[VEC], const bool plain) {
    const Tile at = sh.tile[k % kRing];
    const int64_t h = ((int64_t)at.group * 32 + lane) * VEC;
    const int64_t t0 = (int64_t)at.tile * kBackTile + warp * S;
    bool on[VEC];
    float G[VEC], sum[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      on[v] = kBulk || (h + v < q.H && DLR_IN(at.b, q.B));
      G[v] = sh.enter[k & 1][warp][lane * VEC + v];
      sum[v] = 0.0f;
    }
    const float* own = &sh.k[k % kRing][lane * VEC];
    const float2 k2 = make_float2(own[0], own[VEC - 1]);
    T* r = &sh.rd[k & 3][0][warp * S][lane * VEC];
    T* i = &sh.ix[k & 1][0][warp * S][lane * VEC];
    T* x = i + kBackTile * C;
    float2 t[NP];  // G of each step
#pragma unroll
    for (int m = 0; m < NP; ++m) t[m] = get2<T, VEC, C>(r + kBackTile * C, m);
#pragma unroll
    for (int m = NP - 1; m >= 0; --m) {
      float2 a = kept_decay(z.ka[m]);
      if constexpr (VEC == 2) {
        t[m] = add2(t[m], make_float2(G[0], G[1]));
        const float2 g = mul2(a, t[m]);
        G[0] = g.x, G[1] = g.y;
        if (!plain && (z.cut >> m) & 1u) G[0] = G[1] = 0.0f;
      } else {
        t[m].y += G[0];
        G[0] = a.y * t[m].y;
        if (!plain && (z.cut >> (2 * m + 1)) & 1u) G[0] = 0.0f;
        t[m].x += G[0];
        G[0] = a.x * t[m].x;
        if (!plain && (z.cut >> (2 * m)) & 1u) G[0] = 0.0f;
      }
    }
    wait(&sh.ix_here[k & 1], (k >> 1) & 1);
#pragma unroll
    for (int m = 0; m < NP; ++m) {
      constexpr int per = VEC == 2 ? 1 : 2;  // steps of a pair
      const int j = m * per;
      const float2 sr = sigmoid2(get2<T, VEC, C>(r, m)), si = sigmoid2(get2<T, VEC, C>(i, m));
      const float2 sx = mul2(si, get2<T, VEC, C>(x, m));
      // 1 - a^2 from what is kept: 1 - k^2, or -k (2 + k) where k = a - 1
      const float2 neg = sign_ones(z.ka[m]), a = add2(z.ka[m], neg);
      const float2 u = fma2(mul2(z.ka[m], two(-1.0f)), fma2(neg, two(2.0f), z.ka[m]),
                            fma2(neg, two(-1.0f), two(1.0f)));
      const float2 rm = rsqrt2(u), mm = mul2(u, rm), b = mul2(mm, sx);
      float2 before;  // the state before the step
      if constexpr (VEC == 2) {
        if (!plain && (z.cut >> m) & 1u) s[0] = s[1] = 0.0f;
        before = make_float2(s[0], s[1]);
        const float2 n = fma2(a, before, b);
        s[0] = n.x, s[1] = n.y;
      } else {
        if (!plain && (z.cut >> j) & 1u) s[0] = 0.0f;
        before.x = s[0];
        s[0] = fmaf(a.x, s[0], b.x);
        if (!plain && (z.cut >> (j + 1)) & 1u) s[0] = 0.0f;
        before.y = s[0];
        s[0] = fmaf(a.y, s[0], b.y);
      }
      const float2 arm = mul2(mul2(a, two(-1.0f)), rm);
      const float2 E = mul2(mul2(mul2(t[m], a), sr), fma2(arm, sx, before));
      const float2 tm = mul2(t[m], mm);
      const float2 ox = mul2(tm, si);
      const float2 oi = mul2(mul2(tm, sx), fma2(si, two(-1.0f), two(1.0f)));
      const float2 orr = mul2(mul2(k2, E), add2(sr, two(-1.0f)));
      if constexpr (VEC == 2) {
        if (plain || j < z.n) {
          const float2 n = add2(make_float2(sum[0], sum[1]), E);
          sum[0] = n.x, sum[1] = n.y;
        }
      } else {
        if (plain || j < z.n) sum[0] += E.x;
        if (plain || j + 1 < z.n) sum[0] += E.y;
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
        if constexpr (kBulk) {
          put<T, VEC, kOne>(x + (j + d) * C, px, on);
          put<T, VEC, kOne>(r + (j + d) * C, pr, on);
          put<T, VEC, kOne>(i + (j + d) * C, pi, on);
        } else if (j + d < z.n && DLR_IN(t0 + j + d, q.L)) {
          put<T, VEC, kOne>(dx.row(at.b, t0 + j + d) + h, px, on);
          put<T, VEC, kOne>(dr.row(at.b, t0 + j + d) + h, pr, on);
          put<T, VEC, kOne>(di.row(at.b, t0 + j + d) + h, pi, on);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) sh.sum[k & 1][warp][lane * VEC + v] = sum[v];
    if (kBulk && z.n > 0) {
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tc::tma_store_3d(&out.map[0], &sh.ix[k & 1][1][warp * S][0], at.group * C, (int)t0, at.b);
        tc::tma_store_3d(&out.map[1], &sh.rd[k & 3][0][warp * S][0], at.group * C, (int)t0, at.b);
        tc::tma_store_3d(&out.map[2], &sh.ix[k & 1][0][warp * S][0], at.group * C, (int)t0, at.b);
        tc::bulk_commit_group();
      }
    }
  };
  // tile k's decays are in `now`; true when it was the last
  auto turn = [&](int k, Part& now, Part& next) {
    float s[VEC];
    kept(k, now, s);
    decays(k + 1, next);
    if (kBulk) {
      if (lane == 0) tc::bulk_wait_group_read0();  // the outputs of tile k - 1 have left
      __syncwarp();
    } else {
      copies_wait();
    }
    bar_sync(kEnterBar + (k & 1), kBackThreads);
    fetch_rd(k + 3);
    fetch_ix(k + 1);
    if (!kBulk) copies_end();
    if (now.n == S && now.cut == 0)
      finish(k, now, s, true);
    else
      finish(k, now, s, false);
    return sh.tile[(k + 1) % kRing].tile < 0;
  };
  Part z0, z1;
  __syncthreads();
  for (int k = 0; k < 3; ++k) fetch_rd(k);
  fetch_ix(0);
  if (!kBulk) {
    copies_end();
    copies_wait();
    bar_sync(kWarpsBar + 1, kWork);
  }
  decays(0, z0);
  const bool any = sh.tile[0].tile >= 0;  // read now: its place in the ring is used again
  for (int k = 0; any; k += 2) {
    if (turn(k, z0, z1)) break;
    if (turn(k + 1, z1, z0)) break;
  }
  bar_sync(kWarpsBar, kWork + 32);  // the supplying warp has the last tile's sums to add
  if (kBulk && lane == 0) tc::bulk_wait_group0();
}

// dp = -c sigmoid(p) times the sum of a channel's parts, in a fixed order: a warp for each 32
// channels and 8 rows of warps that share the parts. Bound by latency: a warp adds its parts one
// after another, and few channels make few blocks. B8 L4096 H256 (296 parts, 8 blocks): 11 us by
// itself with cold caches, beside back_kernel's 39.
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
constexpr int kStepRows = 4;

// One token. A thread has VEC channels (two neighbouring 16-bit or 32-bit ones where the rows allow
// an access of both) of kStepRows batch entries, whose loads go out together and share the decay
// parameter. Two channels and four entries to a thread: 256 x 4096 bf16 in 3.8 us, against 6.9 us
// with one element.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads)
step_kernel(view<const T> x, view<const T> r, view<const T> i, const float* __restrict__ p,
            const uint8_t* __restrict__ reset, int64_t B, int64_t H, float c, const float* h,
            view<T> y, float* h_out) {
  const int64_t ch = (blockIdx.x * (int64_t)kThreads + threadIdx.x) * VEC;
  const int64_t b0 = blockIdx.y * (int64_t)kStepRows;
  if (ch >= H) return;
  const int n = (int)min((int64_t)kStepRows, B - b0);
  float xv[kStepRows][VEC], rv[kStepRows][VEC], iv[kStepRows][VEC], hv[kStepRows][VEC];
  bool cut[kStepRows];
  auto read = [&](const T* from, float* to) {
    words<T, VEC> k;
    k.get(from);
    k.to(to);
  };
#pragma unroll
  for (int j = 0; j < kStepRows; ++j) {
    if (j >= n) break;
    read(r.row(b0 + j, 0) + ch, rv[j]);
    read(i.row(b0 + j, 0) + ch, iv[j]);
    read(x.row(b0 + j, 0) + ch, xv[j]);
    words<float, VEC> k;
    k.get(h + (b0 + j) * H + ch);
    k.to(hv[j]);
    cut[j] = reset && reset[b0 + j];
  }
  float kz[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) kz[v] = -c * softplus(p[ch + v]) * kLog2e;
#pragma unroll
  for (int j = 0; j < kStepRows; ++j) {
    if (j >= n) break;
    float2 a, b;
    gates2(make_float2(rv[j][0], rv[j][VEC - 1]), make_float2(iv[j][0], iv[j][VEC - 1]),
           make_float2(xv[j][0], xv[j][VEC - 1]), make_float2(kz[0], kz[VEC - 1]), a, b);
    float2 s = fma2(a, make_float2(hv[j][0], hv[j][VEC - 1]), b);
    if (cut[j]) s = b;
    if (!DLR_IN((b0 + j) * H + ch + VEC - 1, B * H)) continue;
    const float out[2] = {s.x, s.y};
    words<float, VEC> k;
    k.from(out);
    k.put(h_out + (b0 + j) * H + ch);
    words<T, VEC> t;
    t.from(out);
    t.put(y.row(b0 + j, 0) + ch);
  }
}

template <typename T>
view<const T> in_view(const glr_view& v) {
  return {static_cast<const T*>(v.data), v.stride_b, v.stride_t};
}
template <typename T>
view<T> out_view(const glr_out& v) {
  return {static_cast<T*>(v.data), v.stride_b, v.stride_t};
}

// Bytes of the parts of a workspace for tiles of `steps` steps, laid out one behind the other: the
// head, the maps, the entering values, and those of the runs.
struct Space {
  int64_t tiles, HP;
  size_t head, maps, in, runs;
  Space(int64_t B, int64_t L, int64_t H, int64_t steps)
      : tiles(L < 1 ? 0 : (L - 1) / steps + 1), HP((H + 63) / 64 * 64), head(4 * kHead) {
    in = sizeof(float) * (size_t)B * (size_t)tiles * (size_t)HP;
    maps = 2 * in;
    runs = 3 * sizeof(float) * (size_t)B * (size_t)((tiles + kRun - 1) / kRun) * (size_t)HP;
  }
  size_t all() const { return head + maps + in + runs; }
};

// A tensor map over an array [B, L, H] whose boxes are `rows` rows of 128 bytes.
template <typename T, typename V>
bool describe(CUtensorMap* m, const V& v, int64_t B, int64_t L, int64_t H, int rows) {
  auto fn = tc::tensor_map_encoder();
  if (!fn) return false;
  const CUtensorMapDataType type = sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : is_half<T>   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t dims[3] = {(cuuint64_t)H, (cuuint64_t)L, (cuuint64_t)B};
  // the stride of a dimension of one is never used
  const cuuint64_t st = (cuuint64_t)(L > 1 ? v.stride_t : H) * sizeof(T);
  const cuuint64_t strides[2] = {st, B > 1 ? (cuuint64_t)v.stride_b * sizeof(T) : st};
  const cuuint32_t box[3] = {128 / sizeof(T), (cuuint32_t)rows, 1}, one[3] = {1, 1, 1};
  return fn(m, type, 3, const_cast<void*>(static_cast<const void*>(v.data)), dims, strides, box,
            one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// whether it can be: strides that are positive, a multiple of 16 bytes and below 2^40 of them
template <typename V>
bool can_describe(const V& v, int64_t size, int64_t B, int64_t L) {
  auto ok = [&](int64_t s) { return s > 0 && s * size % 16 == 0 && s * size < (int64_t(1) << 40); };
  return (reinterpret_cast<uintptr_t>(v.data) & 15u) == 0 && (L <= 1 || ok(v.stride_t)) &&
         (B <= 1 || ok(v.stride_b));
}

// whether accesses of `n` bytes fit a view's rows
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
          reinterpret_cast<float*>(ws + sp.head + sp.maps), reinterpret_cast<float*>(ws + sp.head),
          nullptr, nullptr, reinterpret_cast<uint32_t*>(ws), device_status_word(), a.B, a.L, a.H,
          sp.HP, a.B * groups,
          (int)groups, (int)sp.tiles, 0, 1, (float)a.c};
}

// Blocks for all tiles, one to an SM at most; the chain's workspace becomes empty. A chain of one
// tile needs neither that nor the counter: each has a block.
template <typename T>
cudaError_t prepare_chain(Job<T>& q, const Space& sp, unsigned* blocks, cudaStream_t s) {
  const int64_t all = q.chains * q.tiles;
  *blocks = (unsigned)all;
  if (q.tiles == 1) return cudaSuccess;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  *blocks = (unsigned)std::min<int64_t>(all, sms);
  q.most = (int)((all - 1) / *blocks + 1);  // all blocks get as many, however early they come
  // Runs, where many tiles of a chain are at work at a time. B1 L65536, us with and without runs:
  // float32 H64 (2 chains) 28 and 41, H128 (4) 63 and 57, H256 (8) 115 and 89; bfloat16 H64 (1) 21
  // and 65, H256 (4) 68 and 89, but B2 H256 (8) 128 and 112.
  if (*blocks / q.chains * kVec<T> >= 64) q.runs = (q.tiles - 1) / kRun + 1;
  q.run_in = q.in + sp.in / sizeof(float);
  q.run_maps = q.run_in + q.B * q.runs * q.HP;
  return cudaMemsetAsync(q.head, 0xff, q.runs ? sp.all() : sp.head + sp.maps + sp.in, s);
}

template <typename T, int kBytes>
cudaError_t scan_w(const glr_scan_args& a, cudaStream_t s) {
  constexpr size_t smem = sizeof(ScanShared<T>);
  const Space sp(a.B, a.L, a.H, kScanTile);
  Job<T> q = make_job<T>(a, sp);
  unsigned blocks;
  cudaError_t e = prepare_chain(q, sp, &blocks, s);
  if (e != cudaSuccess) return e;
  Maps<3> in{};
  Maps<1> out{};
  if (kBytes == kTma && !(describe<T>(&in.map[0], a.r, a.B, a.L, a.H, kScanTile) &&
                          describe<T>(&in.map[1], a.i, a.B, a.L, a.H, kScanTile) &&
                          describe<T>(&in.map[2], a.x, a.B, a.L, a.H, kScanTile) &&
                          describe<T>(&out.map[0], a.y, a.B, a.L, a.H, kScanSteps)))
    return cudaErrorInvalidValue;
  auto launch = [&](auto kernel, cudaError_t ready) {
    if (ready != cudaSuccess) return ready;
    kernel<<<blocks, kScanThreads, smem, s>>>(q, in, out, out_view<T>(a.y), a.h0, a.h_last,
                                              a.states);
    return cudaGetLastError();
  };
  return q.runs ? launch(scan_kernel<T, kBytes, true>,
                         max_smem_once<scan_kernel<T, kBytes, true>>(smem))
                : launch(scan_kernel<T, kBytes, false>,
                         max_smem_once<scan_kernel<T, kBytes, false>>(smem));
}

template <typename T, int kBytes>
cudaError_t back_w(const glr_scan_backward_args& a, cudaStream_t s) {
  constexpr size_t smem = sizeof(BackShared<T>);
  const Space sp(a.B, a.L, a.H, kBackTile);
  Job<T> q = make_job<T>(a, sp);
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + sp.all());
  unsigned blocks;
  cudaError_t e = prepare_chain(q, sp, &blocks, s);
  if (e != cudaSuccess) return e;
  Maps<4> in{};
  Maps<3> out{};
  if (kBytes == kTma && !(describe<T>(&in.map[0], a.r, a.B, a.L, a.H, kBackTile) &&
                          describe<T>(&in.map[1], a.dy, a.B, a.L, a.H, kBackTile) &&
                          describe<T>(&in.map[2], a.i, a.B, a.L, a.H, kBackTile) &&
                          describe<T>(&in.map[3], a.x, a.B, a.L, a.H, kBackTile) &&
                          describe<T>(&out.map[0], a.dx, a.B, a.L, a.H, kBackSteps) &&
                          describe<T>(&out.map[1], a.dr, a.B, a.L, a.H, kBackSteps) &&
                          describe<T>(&out.map[2], a.di, a.B, a.L, a.H, kBackSteps)))
    return cudaErrorInvalidValue;
  auto launch = [&](auto kernel, cudaError_t ready) {
    if (ready == cudaSuccess)
      kernel<<<blocks, kBackThreads, smem, s>>>(q, in, out, in_view<T>(a.dy), a.states, a.dh_last,
                                                out_view<T>(a.dx), out_view<T>(a.dr),
                                                out_view<T>(a.di), a.dh0, part);
    return ready;
  };
  e = q.runs ? launch(back_kernel<T, kBytes, true>,
                      max_smem_once<back_kernel<T, kBytes, true>>(smem))
             : launch(back_kernel<T, kBytes, false>,
                      max_smem_once<back_kernel<T, kBytes, false>>(smem));
  if (e != cudaSuccess) return e;
  back_sum<<<(unsigned)((a.H + 31) / 32), 256, 0, s>>>(part, a.B * q.tiles, a.H, a.p, (float)a.c,
                                                       a.dp);
  return cudaGetLastError();
}

template <typename T>
cudaError_t scan_t(const glr_scan_args& a, cudaStream_t s) {
  const int64_t z = sizeof(T);
  auto tma = [&](const auto& v) { return can_describe(v, z, a.B, a.L); };
  auto all = [&](int64_t n) {
    return a.H * z % n == 0 && wide(a.x, z, n) && wide(a.r, z, n) && wide(a.i, z, n) &&
           wide(a.y, z, n);
  };
  if (a.H * z % 16 == 0 && tma(a.x) && tma(a.r) && tma(a.i) && tma(a.y))
    return scan_w<T, kTma>(a, s);
  if (all(4)) return scan_w<T, 4>(a, s);
  if constexpr (sizeof(T) == 2) return scan_w<T, 2>(a, s);
  return cudaErrorInvalidValue;  // not reached: float rows begin on 4-byte boundaries
}
template <typename T>
cudaError_t back_t(const glr_scan_backward_args& a, cudaStream_t s) {
  const int64_t z = sizeof(T);
  auto tma = [&](const auto& v) { return can_describe(v, z, a.B, a.L); };
  auto all = [&](int64_t n) {
    return a.H * z % n == 0 && wide(a.x, z, n) && wide(a.r, z, n) && wide(a.i, z, n) &&
           wide(a.dy, z, n) && wide(a.dx, z, n) && wide(a.dr, z, n) && wide(a.di, z, n);
  };
  if (a.H * z % 16 == 0 && tma(a.x) && tma(a.r) && tma(a.i) && tma(a.dy) && tma(a.dx) &&
      tma(a.dr) && tma(a.di))
    return back_w<T, kTma>(a, s);
  if (all(4)) return back_w<T, 4>(a, s);
  if constexpr (sizeof(T) == 2) return back_w<T, 2>(a, s);
  return cudaErrorInvalidValue;  // not reached, as above
}

template <typename T, int VEC>
cudaError_t step_v(const glr_step_args& a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.H + kThreads * VEC - 1) / (kThreads * VEC)),
                  (unsigned)((a.B + kStepRows - 1) / kStepRows));
  step_kernel<T, VEC><<<grid, kThreads, 0, s>>>(in_view<T>(a.x), in_view<T>(a.r), in_view<T>(a.i),
                                                a.p, a.reset, a.B, a.H, (float)a.c, a.h,
                                                out_view<T>(a.y), a.h_out);
  return cudaGetLastError();
}
template <typename T>
cudaError_t step_t(const glr_step_args& a, cudaStream_t s) {
  const int64_t z = sizeof(T);
  auto rows = [&](const auto& v) {  // stride_t is not used
    return ((reinterpret_cast<uintptr_t>(v.data) | (uintptr_t)(v.stride_b * z)) & (2 * z - 1)) == 0;
  };
  if (a.H % 2 == 0 && rows(a.x) && rows(a.r) && rows(a.i) && rows(a.y) &&
      ((reinterpret_cast<uintptr_t>(a.h) | reinterpret_cast<uintptr_t>(a.h_out)) & 7u) == 0)
    return step_v<T, 2>(a, s);
  return step_v<T, 1>(a, s);
}

}  // namespace

size_t scan_workspace_bytes(int64_t B, int64_t L, int64_t H) {
  const Space sp(B, L, H, kScanTile);
  return sp.tiles <= 1 ? 0 : sp.all();
}
size_t scan_backward_workspace_bytes(int64_t B, int64_t L, int64_t H) {
  const Space sp(B, L, H, kBackTile);
  return sp.all() + sp.in;  // and the parts of dp
}
// tiles, which a 32-bit counter hands out, of the finest cut that a call of this size takes
int64_t scan_tiles(int64_t B, int64_t L, int64_t H) {
  return B * ((L + kScanTile - 1) / kScanTile) * ((H + 31) / 32);
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
