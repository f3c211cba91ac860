// xent.cu -- the softmax cross entropy of include/xent.h: a projection onto the vocabulary whose
// logits live in tensor memory, and its gradients.
//
// Four products on the 5th-generation tensor cores, one kernel (xgemm) with four ends:
//   the loss        z = h W^T, a tile's rows reduced to their maximum and sum of exponentials (the target's
//                   logit apart);
//   the gradients   z again for a piece of the vocabulary, d = (softmax - onehot) dloss rounded to
//                   the inputs' type and stored; then dh += d W and dW = d^T h over that piece.
// The gradients form the logits a second time, a third of their work, for never holding more of d
// than a piece (256 MB of it, or 256 columns where they take more). W and h are read as they lie: the operands of the last two products
// have their rows along the sum, which the tensor core takes as they are (MN-major).
//
// float32 goes through the same kernel: x = x0 + x1 + x2 with bfloat16 parts, exact to 2^-24, and
// the six products of parts whose orders of magnitude add up to no less than 2^-16, the small ones
// first. Products of parts are exact and accumulated in float32, as those of 16-bit inputs; but the
// tensor core cuts off where it adds, a step of 16 of the sum at a time, and what that leaves out adds
// up (5e-6 of dh at V = 4099), so float32's, few rows' and long sums are added to a second accumulator
// piece by piece (`product`).
//
// 8192 x 50257 x 2048 bfloat16, tensor products at the rate of the power limit: z with the loss 950 us
// (1.78 PFLOP/s), d 1100, dh 1114, dW 1152 (1.46); with the rows laid out and the sums' ends the gradients
// take 3430. 16 rows of it: 40 us, W read at 5.1 TB/s.
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "dlr_common.cuh"
#include "glr_common.cuh"
#include "tc_ptx.cuh"
#include "xent.h"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 26;

int* device_status_word();

namespace xent {
namespace {

using glr::ex2;
using glr::from_f;
using glr::kLog2e;
using glr::to_f;

constexpr int kBM = 128, kBN = 256, kBK = 64;  // a tile, and the sum's extent of a stage
constexpr uint32_t kABytes = kBM * kBK * 2, kBBytes = kBN * kBK * 2;
constexpr uint32_t kStage = kABytes + kBBytes;
constexpr int kStages = 4;
constexpr uint32_t kBox = 32 * 128;                // a warp's staging: 32 rows x 128 bytes
constexpr uint32_t kBoxes = 2;
constexpr uint32_t kEpiOff = kStages * kStage;
constexpr uint32_t kBarOff = kEpiOff + 4 * kBoxes * kBox;
constexpr size_t kSmem = 1024 + kBarOff + 256;
constexpr uint32_t kTmemCols = 512;
constexpr int kThreads = 256;
constexpr int kGroup = 16;  // rows of tiles that go through the columns together
static_assert(kSmem <= 232448, "shared memory");

enum Mode { kLoss, kGrad, kRows, kColumns };

// The parts whose products are formed, the small ones first.
__device__ __constant__ const int8_t kPartA[6] = {0, 2, 1, 0, 1, 0};
__device__ __constant__ const int8_t kPartB[6] = {2, 0, 1, 1, 0, 0};

struct gemm_args {
  int M, N, K;
  int bn;              // columns of a tile, at most kBN (kLoss, kGrad)
  int splits, k_split; // kRows: parts of the sum, each of k_split, that go to float32 sums of their own
  int products;        // 1, or 6 for float32
  int chunk;           // KEEPS: stages between additions to the second accumulator (kSmall times as many of the
                       // small products' stages)
  int a_rows;          // of A's box: all kBM, or those of the only tile (not kColumns)
  int a_along, b_along;  // rows along the sum have their 64s as a dimension of the map
  int b_row;           // where the piece begins among W's rows
  int v0;              // first column's place in the vocabulary (kLoss, kGrad)
  const int64_t* target;
  int V;
  const float* lse;    // kGrad
  const float* dloss;
  const float* scale;  // of d in 16 bits and its inverse, or null
  float2* stats;       // kLoss: [column of tiles, M] maximum and sum
  float* hit;          // [M] the target's logit: kLoss writes it, kGrad takes it (null: its own)
  int keep;            // kRows: 1 store the sums (float32, at tmC), 2 add them to those there
  void* out;
  int64_t out_stride;
  int* status;
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, tc::mbar_wait_sleep(bar, parity)) != 0;
}

constexpr int kSmall = 8;
// KEEPS: where the piece of a sum ends that begins at stage k of `steps`, and how many pieces there are. Of
// float32's six products all but the last are 2^-8 of the sum or less, and so is what they lose.
__device__ __forceinline__ int small_stages(const gemm_args& g, int steps) {
  return g.products == 1 ? 0 : steps / g.products * (g.products - 1);
}
__device__ __forceinline__ int piece_end(const gemm_args& g, int k, int steps) {
  const int small = small_stages(g, steps);
  return k < small ? min(small, k + kSmall * g.chunk) : min(steps, k + g.chunk);
}
__device__ __forceinline__ int pieces(const gemm_args& g, int steps) {
  const int small = small_stages(g, steps), most = kSmall * g.chunk;
  return (small + most - 1) / most + (steps - small + g.chunk - 1) / g.chunk;
}

// Tile t in an order that keeps kGroup rows of tiles on one column's operand at a time.
__device__ __forceinline__ void tile_at(int64_t t, int mt, int nt, int& mi, int& ni) {
  const int64_t per = (int64_t)kGroup * nt;
  const int g = (int)(t / per), first = g * kGroup, rows = min(kGroup, mt - first);
  const int64_t r = t - g * per;
  mi = first + (int)(r % rows);
  ni = (int)(r / rows);
}

// bf16 parts of a float32: x = b[0] + b[1] + b[2] to 2^-24 of x.
__device__ __forceinline__ void split3(float x, __nv_bfloat16 (&b)[3]) {
  b[0] = __float2bfloat16_rn(x);
  float r = x - __bfloat162float(b[0]);
  if (!isfinite(r)) {  // x is not finite, or rounds to an infinity: its parts are cut off instead
    b[0] = __ushort_as_bfloat16((unsigned short)(__float_as_uint(x) >> 16));
    if (x != x) b[0] = __float2bfloat16_rn(x);
    r = isfinite(x) ? x - __bfloat162float(b[0]) : 0.0f;
  }
  b[1] = __float2bfloat16_rn(r);
  b[2] = __float2bfloat16_rn(r - __bfloat162float(b[1]));
}

// T: the operands' type (bfloat16 also for float32's parts); O: the inputs' own, float for parts, in
// three of which kGrad then stores d. Warp 0 loads, warp 1 issues the products, warp 2 has the tensor
// memory, warps 4-7 read the accumulators; two accumulators take turns.
template <Mode MODE, typename T, typename O, bool KEEPS>
__global__ void __launch_bounds__(kThreads, 1)
xgemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
      const __grid_constant__ CUtensorMap tmC, const gemm_args g) {
  constexpr bool kAmn = MODE == kColumns, kBmn = MODE == kRows || MODE == kColumns;
  // KEEPS: accumulator 0 works, 1 keeps; otherwise they take turns
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + kBarOff);
  uint64_t* full = bars;
  uint64_t* empty = bars + kStages;
  uint64_t* acc_full = bars + 2 * kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // all tiles have kBN columns and the whole sum, but where a few would leave SMs without one
  const int bn = MODE == kLoss || MODE == kGrad ? g.bn : kBN;
  const int mt = (g.M + kBM - 1) / kBM, nt = (g.N + bn - 1) / bn;
  const int64_t tiles = (int64_t)mt * nt, work = MODE == kRows ? tiles * g.splits : tiles;
  // stages of a tile's sum: nk(t) for each product, from k_from(t) on
  auto k_from = [&](int64_t t) { return MODE == kRows ? (int)(t / tiles) * g.k_split : 0; };
  auto stages = [&](int64_t t) {
    const int k = MODE == kRows ? min(g.k_split, g.K - k_from(t)) : g.K;
    return (k + kBK - 1) / kBK;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&full[s], 2);
      tc::mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      tc::mbar_init(&acc_full[a], 1);
      tc::mbar_init(&acc_empty[a], 4);
    }
    tc::mbar_fence_init();
  }
  if (warp == 2) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;

  if ((warp == 0 || warp == 3) && lane == 0) {
    // warp 0 loads A's rows, warp 3 B's: with one thread for both the six copies of a stage took
    // longer to issue than its products
    const bool is_a = warp == 0;
    const uint32_t bytes = (is_a ? (kAmn ? kBM : g.a_rows) : bn) * kBK * 2;
    const CUtensorMap* map = is_a ? &tmA : &tmB;
    // rows along the sum: a box of 64 x 64 for each 64 of them, by one copy where the map has them as
    // a dimension
    const bool mn = is_a ? kAmn : kBmn, along = mn && (is_a ? g.a_along : g.b_along);
    const int shift = is_a ? 0 : g.b_row;
    uint32_t it = 0;
    for (int64_t t = blockIdx.x; t < work && ok; t += gridDim.x) {
      int mi, ni;
      tile_at(t % tiles, mt, nt, mi, ni);
      const int row = is_a ? mi * kBM : ni * bn, nk = stages(t), from = k_from(t);
      for (int p = 0; p < g.products && ok; ++p) {
        const int product = g.products == 1 ? 5 : p;
        const int part = is_a ? kPartA[product] : kPartB[product];
        for (int k = 0, k0 = from; k < nk; ++k, k0 += kBK, ++it) {
          const uint32_t s = it % kStages;
          if (it >= kStages && !(ok = tc::mbar_wait(&empty[s], ((it / kStages) - 1) & 1))) break;
          uint8_t* to = base + (DLR_IN(s, kStages) ? s : 0) * kStage + (is_a ? 0 : kABytes);
          tc::mbar_arrive_expect_tx(&full[s], bytes);
          if (along) {
            tc::tma_load_4d(to, map, 0, shift + k0, row / 64, part, &full[s]);
          } else if (mn) {
            for (uint32_t i = 0; i < bytes / 8192; ++i)
              tc::tma_load_3d(to + i * 8192, map, row + 64 * i, shift + k0, part, &full[s]);
          } else {
            tc::tma_load_3d(to, map, k0, shift + row, part, &full[s]);
          }
        }
      }
    }
    // before the CTA may exit, every copy it issued has landed (normally long since consumed)
    for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
      ok &= tc::mbar_wait(&full[j % kStages], (j / kStages) & 1);
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc =
        (glr::is_half<T> ? tc::idesc_f16_f32(kBM, bn) : tc::idesc_bf16_f32(kBM, bn)) |
        (kAmn ? 1u << 15 : 0u) | (kBmn ? 1u << 16 : 0u);
    uint32_t it = 0, local = 0;  // stages, accumulators handed over
    for (int64_t t = blockIdx.x; t < work && ok; t += gridDim.x) {
      const int steps = stages(t) * g.products;
      for (int k = 0; k < steps && ok;) {
        const uint32_t acc = KEEPS ? 0 : local & 1, turns = KEEPS ? 1 : 2;
        if (local >= turns && !(ok = tc::mbar_wait(&acc_empty[acc], (local / turns - 1) & 1))) break;
        tc::fence_after_sync();
        const uint32_t d = tmem + acc * kBN;
        const int stop = KEEPS ? piece_end(g, k, steps) : steps;
        for (int first = k; k < stop; ++k, ++it) {
          const int s = it % kStages;
          if (!(ok = tc::mbar_wait(&full[s], (it / kStages) & 1))) break;
          tc::fence_after_sync();
          const uint8_t* a = base + s * kStage;
          const uint8_t* b = a + kABytes;
          const uint64_t ad =
              kAmn ? tc::smem_desc_mn_sw128(a, 8192, 1024) : tc::smem_desc_k_sw128(a);
          const uint64_t bd =
              kBmn ? tc::smem_desc_mn_sw128(b, 8192, 1024) : tc::smem_desc_k_sw128(b);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)  // 16 of the sum: 32 bytes of a row, or 16 rows
            tc::mma_kind_f16(d, ad + (kAmn ? 128 : 2) * kk, bd + (kBmn ? 128 : 2) * kk, idesc,
                             k != first || kk != 0);
          tc::mma_commit(&empty[s]);
        }
        if (!ok) break;
        tc::mma_commit(&acc_full[acc]);
        ++local;
      }
    }
  } else if (warp >= 4) {
    const int q = warp - 4;
    uint8_t* boxes = base + kEpiOff + q * kBoxes * kBox;
    uint32_t local = 0, boxed = 0;
    float scale = 1.0f, unscale = 1.0f;
    if (g.scale) scale = g.scale[0], unscale = g.scale[1];
    for (int64_t t = blockIdx.x; t < work && ok; t += gridDim.x) {
      int mi, ni;
      tile_at(t % tiles, mt, nt, mi, ni);
      const int m0 = mi * kBM + q * 32, n0 = ni * bn, row = m0 + lane;
      const int cols = min(bn, g.N - n0);
      // what a row brings, fetched before the accumulator is waited for
      int64_t target = -1;
      float lse = 0.0f, weight = 0.0f, exact = 0.0f;
      if constexpr (MODE == kLoss || MODE == kGrad) {
        if (row < g.M) {
          target = g.target[row];
          if constexpr (MODE == kGrad) {
            lse = g.lse[row];
            weight = g.dloss[row] * scale;
            if (g.hit) exact = g.hit[row];
          }
        }
      }
      const bool counts = target >= 0 && target < g.V;
      // its column, if it is one of the tile's (slices of columns may reach past a narrow tile)
      const int64_t in_tile = target - g.v0 - n0;
      const int64_t at = counts && in_tile < bn ? in_tile : -1;
      const uint32_t lanes = uint32_t(q * 32) << 16;
      // all but the last chunk to the second accumulator
      const int chunks = KEEPS ? pieces(g, stages(t) * g.products) : 1;
      if constexpr (KEEPS) {
        for (int c = 0; c + 1 < chunks && ok; ++c, ++local) {
          if (!(ok = warp_wait(&acc_full[0], local & 1))) break;
          tc::fence_after_sync();
          for (int i = 0; i < bn; i += 16) {
            uint32_t v[16], w[16];
            tc::tmem_ld16_issue(tmem + lanes + i, v);
            if (c) tc::tmem_ld16_issue(tmem + lanes + kBN + i, w);
            tc::tmem_wait_ld16(v);
            if (c) {
              tc::tmem_wait_ld16(w);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(w[e]));
            }
            tc::tmem_st16(tmem + lanes + kBN + i, v);
          }
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&acc_empty[0]);
        }
        if (!ok) break;
      }
      const uint32_t acc = KEEPS ? 0 : local & 1;
      const uint32_t tcol = tmem + acc * kBN + lanes;
      auto load = [&](int c, float (&v)[32]) {
        tc::tmem_ld32(tcol + c, v);
        if constexpr (KEEPS) {
          if (chunks > 1) {
            float w[32];
            tc::tmem_ld32(tcol + kBN + c, w);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] += w[i];
          }
        }
      };
      if (!(ok = warp_wait(&acc_full[acc], KEEPS ? local & 1 : (local >> 1) & 1))) break;
      ++local;
      tc::fence_after_sync();
      if constexpr (MODE == kLoss) {
        float top = -INFINITY, sum = 0.0f;
        for (int c = 0; c < cols; c += 32) {
          float v[32];
          load(c, v);
          if (cols - c < 32)
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = i < cols - c ? v[i] : -INFINITY;
          if (at >= c && at < c + 32)  // the target's stays by itself: a sure row's loss hangs on the others
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (at == c + i) {
                if (DLR_IN(row, g.M)) g.hit[row] = v[i];
                v[i] = -INFINITY;
              }
          float most = v[0];
#pragma unroll
          for (int i = 1; i < 32; ++i) most = fmaxf(most, v[i]);
          const float next = fmaxf(top, most), from = next == -INFINITY ? 0.0f : next;
          float part = 0.0f;
#pragma unroll
          for (int i = 0; i < 32; ++i) part += ex2((v[i] - from) * kLog2e);
          sum = fmaf(sum, ex2((top - from) * kLog2e), part);
          top = next;
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&acc_empty[acc]);
        if (row < g.M && DLR_IN(ni, nt)) g.stats[(int64_t)ni * g.M + row] = make_float2(top, sum);
      } else if constexpr (MODE == kGrad) {
        constexpr int kParts = sizeof(O) == 4 ? 3 : 1;
        const uint32_t sw = uint32_t(lane & 7);
        const int n_slices = (cols + 63) / 64;
        for (int c = 0; c < n_slices; ++c) {
          float v[64];
          {
            float lo[32], hi[32];
            load(c * 64, lo);
            load(c * 64 + 32, hi);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = lo[i], v[32 + i] = hi[i];
          }
          if (g.hit && at >> 6 == c)
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (at == c * 64 + i) v[i] = exact;
          if (c == n_slices - 1) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&acc_empty[acc]);
          }
          // z - lse first, which is exact next to the top: lse log2(e) has a rounding that grows with lse
          // and would be the whole row's
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            const float2 t = glr::mul2(
                glr::add2(make_float2(v[i], v[i + 1]), glr::two(-lse)), glr::two(kLog2e));
            const float p0 = ex2(t.x) - (at == c * 64 + i ? 1.0f : 0.0f);
            const float p1 = ex2(t.y) - (at == c * 64 + i + 1 ? 1.0f : 0.0f);
            v[i] = counts ? p0 * weight : 0.0f;
            v[i + 1] = counts ? p1 * weight : 0.0f;
          }
#pragma unroll
          for (int part = 0; part < kParts; ++part, ++boxed) {
            uint8_t* box = boxes + (boxed % kBoxes) * kBox;
            if (lane == 0) tc::bulk_wait_group_read<kBoxes - 1>();  // its last store has read it
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float a = v[8 * k + 2 * i], b = v[8 * k + 2 * i + 1];
                w[i] = glr::pack2<T>(make_float2(a, b));
                if constexpr (kParts == 3) {  // what this part leaves
                  const float2 f = glr::unpack2<T>(w[i]);
                  v[8 * k + 2 * i] = a - f.x;
                  v[8 * k + 2 * i + 1] = b - f.y;
                }
              }
              if (DLR_IN(box - base + lane * 128 + 127, kBarOff))
                *reinterpret_cast<uint4*>(box + lane * 128 + ((uint32_t(k) ^ sw) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (m0 < g.M) tc::tma_store_3d(&tmC, box, n0 + c * 64, m0, part);
              tc::bulk_commit_group();
            }
          }
        }
      } else {
        const uint32_t sw = uint32_t(lane & 7);
        for (int c = 0; c < cols; c += 32, ++boxed) {
          float v[32];
          load(c, v);
          if (c + 32 >= cols) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&acc_empty[acc]);
          }
          if (MODE == kRows && g.keep) {  // float32 sums, to be added up over the pieces
            uint8_t* box = boxes + (boxed % kBoxes) * kBox;
            if (lane == 0) tc::bulk_wait_group_read<kBoxes - 1>();  // its last store has read it
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (DLR_IN(box - base + lane * 128 + 127, kBarOff))
                *reinterpret_cast<float4*>(box + lane * 128 + ((uint32_t(k) ^ sw) << 4)) =
                  make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (m0 < g.M) {
                const int split = (int)(t / tiles);
                if (g.keep == 1)
                  tc::tma_store_3d(&tmC, box, n0 + c, m0, split);
                else
                  tc::tma_reduce_add_3d(&tmC, box, n0 + c, m0, split);
              }
              tc::bulk_commit_group();
            }
            continue;
          }
          // to rows of out, through shared memory so that a row's 32 go together
          float* box = reinterpret_cast<float*>(boxes);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 32; ++i) box[lane * 33 + i] = v[i];
          __syncwarp();
          const int col = n0 + c + lane;
          if (col < g.N) {
            O* to = static_cast<O*>(g.out) + (int64_t)m0 * g.out_stride + col;
#pragma unroll 8
            for (int r = 0; r < 32; ++r) {
              if (m0 + r >= g.M) break;
              to[r * g.out_stride] = from_f<O>(box[r * 33 + lane] * unscale);
            }
          }
        }
      }
    }
    if ((MODE == kGrad || MODE == kRows) && lane == 0) tc::bulk_wait_group0();
  }
  if (!ok) report_status(g.status, DLR_ERR_TIMEOUT);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 2) tc::tmem_dealloc(tmem, kTmemCols);
}

// The logit of one row and one of the vocabulary's, by a warp: 16 terms one after the other for 4096, rounded
// to nearest.
template <typename T>
__device__ __forceinline__ float row_logit(const T* h, const T* w, int64_t D, int lane) {
  float2 sum[4] = {};
  for (int64_t d = lane * 8; d < D; d += 256) {
    glr::words<T, 8> a, b;
    if (d + 8 <= D) {
      a.get(h + d);
      b.get(w + d);
    } else {
      float u[8], v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[i] = d + i < D ? to_f(h[d + i]) : 0.0f;
        v[i] = d + i < D ? to_f(w[d + i]) : 0.0f;
      }
      a.from(u);
      b.from(v);
    }
    float x[8], y[8];
    a.to(x);
    b.to(y);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sum[i] = glr::fma2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(y[2 * i], y[2 * i + 1]), sum[i]);
  }
  const float2 s = glr::add2(glr::add2(sum[0], sum[1]), glr::add2(sum[2], sum[3]));
  float z = s.x + s.y;
#pragma unroll
  for (int k = 16; k; k >>= 1) z += __shfl_xor_sync(0xffffffffu, z, k);
  return z;
}

// lse and loss of 32 rows to a block from the tiles' maxima and sums, which are those of the other logits
// than the target's; the block's WARPS warps share the tiles of a row and meet in order (many of them where
// there are few rows). EXACT: the targets' logits are formed here again: a sure row's is a long sum of one
// sign, of which a single accumulator cuts off 3e-6, and its loss is small beside it. (8192 x 50257 x 2048:
// losses 1.7e-6 -> 2.8e-7 off, 10 -> 21 of 960 us, in the gradients 9 more; with eight warps 29.)
template <int WARPS, typename T, bool EXACT>
__global__ void __launch_bounds__(32 * WARPS)
finish_loss(const float2* stats, const float* hit, const int64_t* target, float* loss, float* lse,
            int64_t M, int nt, int64_t V, const T* h, int64_t h_pitch, const T* W, int64_t w_pitch,
            int64_t D) {
  __shared__ float2 part[WARPS][32];
  __shared__ float exact[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t m = (int64_t)blockIdx.x * 32 + lane;
  float top = -INFINITY, sum = 0.0f;
  auto add = [&](float2 s) {
    const float next = fmaxf(top, s.x), from = next == -INFINITY ? 0.0f : next;
    sum = sum * expf(top - from) + s.y * expf(s.x - from);
    top = next;
  };
  if constexpr (EXACT)
    for (int r = warp; r < 32; r += WARPS) {
      const int64_t row = (int64_t)blockIdx.x * 32 + r, t = row < M ? target[row] : -1;
      if (t < 0 || t >= V) continue;
      const float z = row_logit(h + row * h_pitch, W + t * w_pitch, D, lane);
      if (lane == 0) exact[r] = z;
    }
  if (m < M)
#pragma unroll 4
    for (int k = warp; k < nt; k += WARPS) add(stats[(int64_t)k * M + m]);
  part[warp][lane] = make_float2(top, sum);
  __syncthreads();
  if (warp || m >= M) return;
  for (int u = 1; u < WARPS; ++u) add(part[u][lane]);
  const float rest = logf(sum), others = top + rest;
  const int64_t t = target[m];
  if (t < 0 || t >= V) {
    lse[m] = others;
    loss[m] = 0.0f;
    return;
  }
  // log(1 + e^x) for what the others are beyond the target: neither is a difference of large numbers
  const float z = EXACT ? exact[lane] : hit[m], x = (top - z) + rest, little = log1pf(expf(-fabsf(x)));
  loss[m] = fmaxf(x, 0.0f) + little;
  lse[m] = z == -INFINITY && others == -INFINITY ? z : fmaxf(z, others) + little;
}

// The sums over the pieces, and over the parts of each, in the inputs' type.
template <typename O>
__global__ void __launch_bounds__(256)
finish_rows(const float* acc, int64_t pitch, int splits, O* out, int64_t stride, int64_t M, int64_t D,
            const float* scale) {
  const int64_t per = (D + 3) / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = i / per, c = (i - m * per) * 4;
  if (m >= M) return;
  const float k = scale ? scale[1] : 1.0f;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int k = 0; k < splits; ++k) {
    const float4 p = *reinterpret_cast<const float4*>(acc + (k * M + m) * pitch + c);
    v = make_float4(v.x + p.x, v.y + p.y, v.z + p.z, v.w + p.w);
  }
  const float o[4] = {v.x * k, v.y * k, v.z * k, v.w * k};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (c + j < D) out[m * stride + c + j] = from_f<O>(o[j]);
}

// What d is divided by before it is rounded to 16 bits, and its inverse: the largest |dloss| of a row that
// counts. Under a mean all weights are then 1, and d of the many targets that are hardly expected, next to -1,
// is exact; by dloss itself all of them had the same rounding, up to 2^-8 (dh 2.5e-3 off at 8192 x 50257 x
// 2048, now 1.8e-3, of which the result's own rounding is 1.7e-3). float16 adds a factor 2^14 for its range.
//
// The first block does that. The others form the targets' logits of 32 rows each again, which kGrad then takes:
// lse is that of these.
template <typename T>
__global__ void __launch_bounds__(1024)
before_back(const float* dloss, const int64_t* target, int64_t M, int64_t V, float most, float* scale,
            const T* h, int64_t h_pitch, const T* W, int64_t w_pitch, int64_t D, float* hit) {
  __shared__ float part[32];
  if (blockIdx.x) {
    const int64_t row = (int64_t)(blockIdx.x - 1) * 32 + (threadIdx.x >> 5), t = row < M ? target[row] : -1;
    if (t < 0 || t >= V) return;
    const float z = row_logit(h + row * h_pitch, W + t * w_pitch, D, threadIdx.x & 31);
    if ((threadIdx.x & 31) == 0) hit[row] = z;
    return;
  }
  float top = 0.0f;
#pragma unroll 8
  for (int64_t m = threadIdx.x; m < M; m += 1024) {
    const float w = fabsf(dloss[m]);
    top = fmaxf(top, target[m] >= 0 && target[m] < V ? w : 0.0f);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  top = part[threadIdx.x];
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (threadIdx.x) return;
  if (top == 0.0f || top > 3.4e38f) top = most;  // nothing to scale, or an infinity
  top = fminf(fmaxf(top, 0x1p-100f), 0x1p100f);
  scale[0] = most / top;
  scale[1] = top / most;
}

// Rows as the products take them: [parts, rows, pitch] with zeros between `cols` and the pitch. Rows
// whose target does not count are zeros (target NULL: all count).
template <typename T, typename S>
__global__ void __launch_bounds__(256)
stage_rows(const S* src, int64_t stride, T* dst, int64_t rows, int64_t cols, int64_t pitch,
           const int64_t* target, int64_t V) {
  const int64_t per = pitch / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t r = i / per, c = (i - r * per) * 8;
  if (r >= rows) return;
  const bool counts = !target || (target[r] >= 0 && target[r] < V);
  const S* p = src + r * stride + c;
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = counts && c + k < cols ? to_f(p[k]) : 0.0f;
  if constexpr (sizeof(S) == 4) {
    __nv_bfloat16 b[8][3];
#pragma unroll
    for (int k = 0; k < 8; ++k) split3(v[k], b[k]);
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = __bfloat16_as_ushort(b[2 * k][part]) |
               (uint32_t)__bfloat16_as_ushort(b[2 * k + 1][part]) << 16;
      *reinterpret_cast<uint4*>(dst + (part * rows + r) * pitch + c) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = glr::pack2<T>(make_float2(v[2 * k], v[2 * k + 1]));
    *reinterpret_cast<uint4*>(dst + r * pitch + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__global__ void clear_rows(void* dst, int64_t rows, int64_t bytes, int64_t stride) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, r = i / bytes;
  if (r < rows) static_cast<uint8_t*>(dst)[r * stride + (i - r * bytes)] = 0;
}

// ---- host ---------------------------------------------------------------------------------

// [parts, rows, cols], rows `pitch` elements apart, in boxes of box_rows x 128 bytes (swizzled).
// `blocks` > 0: columns in 64s as a dimension of their own, `blocks` of them to a box of box_rows rows
// each; then cols is a multiple of 64 or the rows are followed by as many elements as are missing.
bool make_map(CUtensorMap* m, const void* p, CUtensorMapDataType type, uint64_t parts, uint64_t rows,
              uint64_t cols, uint64_t pitch, uint32_t box_rows, uint32_t blocks = 0) {
  auto fn = tc::tensor_map_encoder();
  if (!fn) return false;
  const uint64_t size = type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
  if (blocks) {
    cuuint64_t dims[4] = {64, rows, (cols + 63) / 64, parts};
    cuuint64_t strides[3] = {pitch * 2, 128, rows * pitch * 2};
    cuuint32_t box[4] = {64, box_rows, blocks, 1}, one[4] = {1, 1, 1, 1};
    return fn(m, type, 4, const_cast<void*>(p), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  cuuint64_t dims[3] = {cols, rows, parts};
  cuuint64_t strides[2] = {pitch * size, rows * pitch * size};
  cuuint32_t box[3] = {uint32_t(128 / size), box_rows, 1}, one[3] = {1, 1, 1};
  return fn(m, type, 3,
            const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
    n = 1;
  return n;
}

// Rows that the products read: the caller's own, or staged ones.
struct operand {
  const void* p;
  uint64_t parts, rows, cols, pitch;
  bool ours = false;  // rows are a multiple of 64 elements apart, in the workspace
  bool blocks() const { return cols % 64 == 0 || ours; }
};

template <Mode MODE, typename T, typename O, bool KEEPS>
cudaError_t launch(const operand& a, const operand& b, const operand* c, gemm_args g,
                    cudaStream_t s) {
  constexpr auto kType = glr::is_half<T> ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                         : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  constexpr bool kAmn = MODE == kColumns, kBmn = MODE == kRows || MODE == kColumns;
  CUtensorMap ma, mb, mc;
  // Few rows are copied alone: the tile's others are what lies there, and so are their sums, which no
  // one reads. Filling them with zeros cost 16 x 50257 x 2048 8 of 54 us.
  g.a_rows = (int)std::min<int64_t>(kBM, up(g.M, 16));
  g.a_along = kAmn && a.blocks(), g.b_along = kBmn && b.blocks();
  if (!make_map(&ma, a.p, kType, a.parts, a.rows, a.cols, a.pitch, kAmn ? kBK : g.a_rows,
                g.a_along ? kBM / 64 : 0) ||
      !make_map(&mb, b.p, kType, b.parts, b.rows, b.cols, b.pitch, kBmn ? kBK : g.bn,
                g.b_along ? kBN / 64 : 0))
    return cudaErrorInvalidValue;
  if (!c)
    mc = ma;  // not used
  else if (!make_map(&mc, c->p, MODE == kRows ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : kType, c->parts,
                     c->rows, c->cols, c->pitch, 32))
    return cudaErrorInvalidValue;
  g.status = device_status_word();
  const cudaError_t e = max_smem_once<xgemm<MODE, T, O, KEEPS>>(kSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)((g.M + kBM - 1) / kBM) * ((g.N + g.bn - 1) / g.bn) * g.splits;
  xgemm<MODE, T, O, KEEPS><<<(unsigned)std::min<int64_t>(tiles, sm_count()), kThreads, kSmem, s>>>(
      ma, mb, mc, g);
  return cudaGetLastError();
}

// A product, and how often its sums go to the second accumulator. The tensor core cuts off some 2^-24 of what
// it has at each step of 16 terms, always towards zero, so that a sum of one sign loses 6e-8 of itself a step
// (measured: 3e-3 of 524288 terms, 5e-4 of 131072). float32's add up every 8 stages of 64 terms. In 16 bits:
// logits of few rows, which wait for W's memory anyway, every 4 (4e-7 of z left out instead of 3e-6 at 1690
// terms); logits of more than 64 stages every 32, dh and dW of more than 256 every 64, so that no more than
// 2e-5 is lost; shorter sums stay in one accumulator, and the two take turns. Both directions' logits go by
// one rule: d of a sure row is a small difference of z and lse.
template <Mode MODE, typename T, typename S>
cudaError_t product(const operand& a, const operand& b, const operand* c, gemm_args g,
                    cudaStream_t s) {
  if constexpr (sizeof(S) == 4) {
    g.chunk = 8;
    return launch<MODE, T, S, true>(a, b, c, g, s);
  } else {
    constexpr bool kLogits = MODE == kLoss || MODE == kGrad;
    const int stages = ((MODE == kRows ? g.k_split : g.K) + kBK - 1) / kBK;
    g.chunk = !kLogits ? 64 : g.M <= kBM ? 4 : 32;
    if ((kLogits && g.M <= kBM) || stages > (kLogits ? 64 : 256))
      return launch<MODE, T, S, true>(a, b, c, g, s);
    return launch<MODE, T, S, false>(a, b, c, g, s);
  }
}

constexpr int64_t kSMs = 152;
// Rounds of tiles of bn columns over the SMs.
int64_t rounds(int64_t rows, int64_t cols, int64_t bn, int64_t splits = 1) {
  return (((rows + kBM - 1) / kBM) * ((cols + bn - 1) / bn) * splits + kSMs - 1) / kSMs;
}
// Columns of a tile, a multiple of `step`: kBN, unless a last round would leave many SMs without one.
// A narrow tile reads its rows of A as often as a wide one.
int columns_of(int64_t rows, int64_t cols, int step) {
  int best = kBN;
  for (int bn = kBN; bn >= 128; bn -= step)
    if (rounds(rows, cols, bn) * (bn + 32) < rounds(rows, cols, best) * (best + 32)) best = bn;
  return best;
}
// Parts of the sum over K of the product for dh, where its tiles are few or would leave many SMs
// without one in the last round. Each part ends with the sums' way out, some eight stages.
int splits_of(int64_t rows, int64_t cols, int64_t K) {
  const int64_t nk = (K + kBK - 1) / kBK;
  int best = 1;
  auto cost = [&](int64_t s) { return rounds(rows, cols, kBN, s) * ((nk + s - 1) / s + 8); };
  for (int s = 2; s <= std::min<int64_t>(kSMs, nk); ++s)
    if (cost(s) < cost(best)) best = s;
  return (int)((nk + (nk + best - 1) / best - 1) / ((nk + best - 1) / best));  // none is empty
}

// Whether the products read a caller's rows as they lie: 16-bit values whose rows begin on multiples
// of 16 bytes, one after the other.
bool direct(int64_t type, const glr_view& v, int64_t rows, int64_t cols) {
  return type != GLR_F32 && (reinterpret_cast<uintptr_t>(v.data) & 15) == 0 &&
         (rows <= 1 || (v.stride_t % 8 == 0 && v.stride_t >= cols));
}

bool direct_h(const xent_loss_args& a) { return direct(a.type, a.h, a.M, a.D); }
template <typename ARGS>
bool direct_w(const ARGS& a) {
  return direct(a.type, a.W, a.V, a.D);
}

// Bytes of staged rows.
int64_t staged(int64_t type, int64_t rows, int64_t cols) {
  return up((type == GLR_F32 ? 3 : 1) * rows * up(cols, 64) * 2, 256);
}

template <typename T, typename S>
cudaError_t stage(const glr_view& v, void* to, int64_t rows, int64_t cols, const int64_t* target,
                  int64_t V, operand* out, cudaStream_t s) {
  const int64_t pitch = up(cols, 64), n = rows * (pitch / 8);
  stage_rows<T, S><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(
      static_cast<const S*>(v.data), v.stride_t, static_cast<T*>(to), rows, cols, pitch, target, V);
  *out = operand{to, sizeof(S) == 4 ? 3u : 1u, (uint64_t)rows, (uint64_t)cols, (uint64_t)pitch, true};
  return cudaGetLastError();
}

// The rows of h or W for the products: as they lie, or staged at `to`.
template <typename T, typename S>
cudaError_t rows_of(int64_t type, const glr_view& v, void* to, int64_t rows, int64_t cols,
                    operand* out, cudaStream_t s) {
  if (direct(type, v, rows, cols)) {
    *out = operand{v.data, 1, (uint64_t)rows, (uint64_t)cols,
                   (uint64_t)(rows > 1 ? v.stride_t : up(cols, 8))};
    return cudaSuccess;
  }
  return stage<T, S>(v, to, rows, cols, nullptr, 0, out, s);
}

// Whether the targets' logits are formed again: where all of a logit goes through one accumulator.
bool exact_targets(int64_t type, int64_t M) { return type != GLR_F32 && M > kBM; }

// How the gradients' vocabulary is cut, and where things lie in their workspace.
struct back_plan {
  int64_t piece, pieces;         // columns of a piece
  int64_t splits;                // parts of its sum for dh
  int64_t d, h, w, acc, scale, hit;  // offsets
  int64_t bytes;
  bool sums() const { return pieces > 1 || splits > 1; }  // dh goes through float32 sums
};
constexpr int64_t kPieceBytes = int64_t(256) << 20;
back_plan plan(int64_t type, int64_t M, int64_t V, int64_t D, bool w_there) {
  const int64_t parts = type == GLR_F32 ? 3 : 1;
  back_plan p;
  // A piece's d takes at most kPieceBytes, but for pieces of kBN columns, the narrowest. Of the piece counts from the least to twice as many, the
  // one whose three products take the fewest stages (a launch costs some forty).
  const int64_t most = std::max<int64_t>(kBN, kPieceBytes / (M * 2 * parts) / kBN * kBN);
  const int64_t least = (V + most - 1) / most;
  int64_t best = -1;
  for (int64_t n = least; n <= 2 * least; ++n) {
    const int64_t piece = up((V + n - 1) / n, kBN), pieces = (V + piece - 1) / piece;
    const int64_t s = splits_of(M, D, std::min(piece, V));
    const int64_t cost = pieces * (rounds(M, piece, kBN) * (D + kBK - 1) / kBK +
                                   rounds(M, D, kBN, s) * ((piece + kBK - 1) / kBK + s - 1) / s +
                                   rounds(piece, D, kBN) * (M + kBK - 1) / kBK + 3 * 40);
    if (best < 0 || cost < best) best = cost, p.piece = piece, p.pieces = pieces, p.splits = s;
  }
  p.d = 0;
  p.h = p.d + up(parts * M * std::min(p.piece, up(V, 64)) * 2, 256);
  p.w = p.h + staged(type, M, D);
  p.acc = p.w + (w_there ? 0 : staged(type, V, D));
  p.scale = p.acc + (p.sums() ? up(p.splits * M * up(D, 4) * 4, 256) : 0);
  p.hit = p.scale + 256;
  p.bytes = p.hit + (exact_targets(type, M) ? up(M * 4, 256) : 0);
  return p;
}

template <typename T, typename S>
cudaError_t loss_of(const xent_loss_args& a, cudaStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const int bn = columns_of(a.M, a.V, 16), nt = (int)((a.V + bn - 1) / bn);
  gemm_args g{};
  g.bn = bn, g.splits = 1;
  g.M = (int)a.M, g.N = (int)a.V, g.K = (int)a.D, g.V = (int)a.V;
  g.products = sizeof(S) == 4 ? 6 : 1;
  g.target = a.target;
  g.stats = reinterpret_cast<float2*>(ws), ws += up((int64_t)nt * a.M * 8, 256);
  g.hit = reinterpret_cast<float*>(ws), ws += up(a.M * 4, 256);
  operand h, w;
  cudaError_t e = rows_of<T, S>(a.type, a.h, ws, a.M, a.D, &h, s);
  if (e != cudaSuccess) return e;
  if (!direct_h(a)) ws += staged(a.type, a.M, a.D);
  e = rows_of<T, S>(a.type, a.W, ws, a.V, a.D, &w, s);
  if (e != cudaSuccess) return e;
  if ((e = product<kLoss, T, S>(h, w, nullptr, g, s)) != cudaSuccess) return e;
  const unsigned blocks = (unsigned)((a.M + 31) / 32);
  auto finish = [&](auto warps, auto exact) {
    finish_loss<warps.value, T, exact.value><<<blocks, 32 * warps.value, 0, s>>>(
        g.stats, g.hit, a.target, a.loss, a.lse, a.M, nt, a.V, static_cast<const T*>(h.p), (int64_t)h.pitch,
        static_cast<const T*>(w.p), (int64_t)w.pitch, a.D);
  };
  auto by_rows = [&](auto exact) {
    if (blocks < 152 || exact.value)
      finish(std::integral_constant<int, 32>{}, exact);
    else
      finish(std::integral_constant<int, 8>{}, exact);
  };
  if constexpr (sizeof(S) == 2)
    if (exact_targets(a.type, a.M)) {
      by_rows(std::true_type{});
      return cudaGetLastError();
    }
  by_rows(std::false_type{});
  return cudaGetLastError();
}

template <typename T, typename S>
cudaError_t back_of(const xent_loss_backward_args& a, cudaStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const back_plan p = plan(a.type, a.M, a.V, a.D, direct_w(a));
  const uint64_t parts = sizeof(S) == 4 ? 3 : 1;
  cudaError_t e;
  operand h, hz, w;
  // the rows of h that count, for dW; the logits take them too
  if ((e = stage<T, S>(a.h, ws + p.h, a.M, a.D, a.target, a.V, &hz, s)) != cudaSuccess) return e;
  h = hz;
  if ((e = rows_of<T, S>(a.type, a.W, ws + p.w, a.V, a.D, &w, s)) != cudaSuccess) return e;
  float *scale = nullptr, *hit = nullptr;
  if constexpr (sizeof(S) == 2) {
    const bool exact = exact_targets(a.type, a.M);
    scale = reinterpret_cast<float*>(ws + p.scale);
    if (exact) hit = reinterpret_cast<float*>(ws + p.hit);
    before_back<T><<<1 + (exact ? (unsigned)((a.M + 31) / 32) : 0), 1024, 0, s>>>(
        a.dloss, a.target, a.M, a.V, glr::is_half<S> ? 0x1p14f : 1.0f, scale, static_cast<const T*>(hz.p),
        (int64_t)hz.pitch, static_cast<const T*>(w.p), (int64_t)w.pitch, a.D, hit);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  for (int64_t k = 0; k < p.pieces; ++k) {
    const int64_t v0 = k * p.piece, cols = std::min(p.piece, a.V - v0);
    const operand d{ws + p.d, parts, (uint64_t)a.M, (uint64_t)cols, (uint64_t)up(cols, 64), true};
    gemm_args g{};
    g.bn = columns_of(a.M, cols, 64), g.splits = 1;
    g.M = (int)a.M, g.N = (int)cols, g.K = (int)a.D, g.V = (int)a.V;
    g.products = sizeof(S) == 4 ? 6 : 1;
    g.b_row = g.v0 = (int)v0;
    g.target = a.target, g.lse = a.lse, g.dloss = a.dloss, g.scale = scale, g.hit = hit;
    if ((e = product<kGrad, T, S>(h, w, &d, g, s)) != cudaSuccess) return e;
    if (a.dh.data) {
      gemm_args r{};
      r.M = (int)a.M, r.N = (int)a.D, r.K = (int)cols, r.products = g.products, r.b_row = (int)v0;
      r.scale = scale;
      r.out = a.dh.data, r.out_stride = a.dh.stride_t;
      // a short last piece may have fewer parts, and leaves the sums of the others as they are
      r.bn = kBN, r.k_split = (int)up((cols + p.splits - 1) / p.splits, kBK);
      r.splits = (int)((cols + r.k_split - 1) / r.k_split);
      r.keep = !p.sums() ? 0 : k == 0 ? 1 : 2;
      const operand acc{ws + p.acc, (uint64_t)p.splits, (uint64_t)a.M, (uint64_t)a.D, (uint64_t)up(a.D, 4)};
      if ((e = product<kRows, T, S>(d, w, r.keep ? &acc : nullptr, r, s)) != cudaSuccess) return e;
    }
    if (a.dW.data) {
      gemm_args c{};
      c.bn = kBN, c.splits = 1;
      c.M = (int)cols, c.N = (int)a.D, c.K = (int)a.M, c.products = g.products;
      c.scale = scale;
      c.out = static_cast<S*>(a.dW.data) + v0 * a.dW.stride_t, c.out_stride = a.dW.stride_t;
      if ((e = product<kColumns, T, S>(d, hz, nullptr, c, s)) != cudaSuccess) return e;
    }
  }
  if (a.dh.data && p.sums()) {
    const int64_t n = a.M * ((a.D + 3) / 4);
    finish_rows<S><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(
        reinterpret_cast<const float*>(ws + p.acc), up(a.D, 4), (int)p.splits,
        static_cast<S*>(a.dh.data), a.dh.stride_t, a.M, a.D, scale);
    return cudaGetLastError();
  }
  return cudaSuccess;
}

}  // namespace

// h_there, w_there: the products read those rows as they lie.
size_t loss_workspace_bytes(int64_t type, int64_t M, int64_t V, int64_t D, bool h_there,
                            bool w_there) {
  const int64_t bn = columns_of(M, V, 16), nt = (V + bn - 1) / bn;
  return (size_t)(up(nt * M * 8, 256) + up(M * 4, 256) + (h_there ? 0 : staged(type, M, D)) +
                  (w_there ? 0 : staged(type, V, D)));
}
size_t loss_workspace_bytes(const xent_loss_args& a) {
  return loss_workspace_bytes(a.type, a.M, a.V, a.D, direct_h(a), direct_w(a));
}

size_t loss_backward_workspace_bytes(int64_t type, int64_t M, int64_t V, int64_t D, bool w_there) {
  return (size_t)plan(type, M, V, D, w_there).bytes;
}
size_t loss_backward_workspace_bytes(const xent_loss_backward_args& a) {
  return loss_backward_workspace_bytes(a.type, a.M, a.V, a.D, direct_w(a));
}

cudaError_t launch_loss(const xent_loss_args& a, cudaStream_t s) {
  if (a.type == GLR_F32) return loss_of<__nv_bfloat16, float>(a, s);
  return a.type == GLR_BF16 ? loss_of<__nv_bfloat16, __nv_bfloat16>(a, s)
                            : loss_of<__half, __half>(a, s);
}

cudaError_t launch_loss_backward(const xent_loss_backward_args& a, cudaStream_t s) {
  if (a.type == GLR_F32) return back_of<__nv_bfloat16, float>(a, s);
  return a.type == GLR_BF16 ? back_of<__nv_bfloat16, __nv_bfloat16>(a, s)
                            : back_of<__half, __half>(a, s);
}

cudaError_t clear_gradient(const glr_out& dW, int64_t type, int64_t V, int64_t D, cudaStream_t s) {
  const int64_t size = type == GLR_F32 ? 4 : 2;
  clear_rows<<<(unsigned)((V * D * size + 255) / 256), 256, 0, s>>>(dW.data, V, D * size,
                                                                    dW.stride_t * size);
  return cudaGetLastError();
}

}  // namespace xent
}  // namespace dlr
