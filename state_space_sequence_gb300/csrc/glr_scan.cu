// glr_scan.cu -- the gated linear recurrence of include/glr.h: h_t = abar_t h_{t-1} + b_t per
// channel with a decay that the token chooses, its gradients, and one token from a carried state.
//
// A run of GLR_STATE_STEPS steps maps the state before it to the state after it by
// h -> A h + e, A the product of its decays and e its end state from zero. The forward pass forms
// (A, e) of every run, carries the state through the runs, and goes over each run again from the
// state before it. The gradients do the same backwards in time with G_t = dy_t + abar_{t+1}
// G_{t+1}: a run maps the gradient that enters behind it to the one that leaves before it by
// G -> A G + C with the same A.
#include "glr_common.cuh"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 16;

namespace glr {
namespace {

constexpr int kRun = GLR_STATE_STEPS;
constexpr int kThreads = 128;

template <typename T>
struct ScanIn {
  view<const T> x, r, i;
  const float* p;
  const uint8_t* reset;
  int64_t B, L, H;
  int64_t runs;  // runs of kRun steps in a row
  float c;
};

// where a block works: batch entry, run of steps, channel
struct Place {
  int64_t b, run, t0, h;
  int steps;
  bool on;
};
template <typename T>
__device__ __forceinline__ Place place(const ScanIn<T>& in) {
  const int64_t groups = (in.H + kThreads - 1) / kThreads;
  Place q;
  int64_t k = blockIdx.x;
  q.h = (k % groups) * kThreads + threadIdx.x;
  k /= groups;
  q.run = k % in.runs;
  q.b = k / in.runs;
  q.t0 = q.run * kRun;
  q.steps = (int)min((int64_t)kRun, in.L - q.t0);
  q.on = q.h < in.H;
  return q;
}

// (A, e) of each run
template <typename T>
__global__ void __launch_bounds__(kThreads) scan_runs(ScanIn<T> in, float2* __restrict__ agg) {
  const Place q = place(in);
  if (!q.on) return;
  const float kz = -in.c * softplus(in.p[q.h]) * kLog2e;
  float A = 1.0f, e = 0.0f;
  for (int j = 0; j < q.steps; ++j) {
    const int64_t t = q.t0 + j;
    const gate g = make_gate(to_f(in.r.row(q.b, t)[q.h]), to_f(in.i.row(q.b, t)[q.h]), kz);
    const bool cut = in.reset && in.reset[q.b * in.L + t];
    const float b = g.m * g.si * to_f(in.x.row(q.b, t)[q.h]);
    e = cut ? b : fmaf(g.a, e, b);
    A = cut ? 0.0f : A * g.a;
  }
  const int64_t at = (q.b * in.runs + q.run) * in.H + q.h;
  if (DLR_IN(at, in.B * in.runs * in.H)) agg[at] = make_float2(A, e);
}

// whether any step of the run begins a sequence
__device__ bool run_cut(const uint8_t* reset, int64_t b, int64_t L, int64_t t0, int steps) {
  bool cut = false;
  if (reset)
    for (int j = 0; j < steps; ++j) cut |= reset[b * L + t0 + j] != 0;
  return cut;
}

// the state before each run, and the last one
__global__ void __launch_bounds__(kThreads)
scan_carry(const float2* __restrict__ agg, const float* __restrict__ h0,
           const uint8_t* __restrict__ reset, int64_t B, int64_t L, int64_t H, int64_t runs,
           float* __restrict__ states, float* __restrict__ h_last) {
  const int64_t k = blockIdx.x * (int64_t)kThreads + threadIdx.x;
  if (k >= B * H) return;
  const int64_t b = k / H, h = k % H;
  float s = h0 ? h0[k] : 0.0f;
  for (int64_t run = 0; run < runs; ++run) {
    const int64_t at = (b * runs + run) * H + h;
    if (!DLR_IN(at, B * runs * H)) break;
    states[at] = s;
    const float2 g = agg[at];
    const bool cut = run_cut(reset, b, L, run * kRun, (int)min((int64_t)kRun, L - run * kRun));
    s = cut ? g.y : fmaf(g.x, s, g.y);
  }
  if (h_last) h_last[k] = s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
scan_apply(ScanIn<T> in, const float* __restrict__ states, view<T> y) {
  const Place q = place(in);
  if (!q.on) return;
  const float kz = -in.c * softplus(in.p[q.h]) * kLog2e;
  float s = states[(q.b * in.runs + q.run) * in.H + q.h];
  for (int j = 0; j < q.steps; ++j) {
    const int64_t t = q.t0 + j;
    const gate g = make_gate(to_f(in.r.row(q.b, t)[q.h]), to_f(in.i.row(q.b, t)[q.h]), kz);
    const bool cut = in.reset && in.reset[q.b * in.L + t];
    const float b = g.m * g.si * to_f(in.x.row(q.b, t)[q.h]);
    s = cut ? b : fmaf(g.a, s, b);
    y.row(q.b, t)[q.h] = from_f<T>(s);
  }
}

// (A, C) of each run, backwards
template <typename T>
__global__ void __launch_bounds__(kThreads)
back_runs(ScanIn<T> in, view<const T> dy, float2* __restrict__ agg) {
  const Place q = place(in);
  if (!q.on) return;
  const float kz = -in.c * softplus(in.p[q.h]) * kLog2e;
  float A = 1.0f, C = 0.0f;
  for (int j = q.steps - 1; j >= 0; --j) {
    const int64_t t = q.t0 + j;
    const float sr = sigmoid(to_f(in.r.row(q.b, t)[q.h]));
    float w, a;
    decay(kz * sr, w, a);
    const bool cut = in.reset && in.reset[q.b * in.L + t];
    const float G = to_f(dy.row(q.b, t)[q.h]) + C;
    C = cut ? 0.0f : a * G;
    A = cut ? 0.0f : A * a;
  }
  const int64_t at = (q.b * in.runs + q.run) * in.H + q.h;
  if (DLR_IN(at, in.B * in.runs * in.H)) agg[at] = make_float2(A, C);
}

// the gradient that enters behind each run, and that of the initial state
__global__ void __launch_bounds__(kThreads)
back_carry(const float2* __restrict__ agg, const float* __restrict__ dh_last,
           const uint8_t* __restrict__ reset, int64_t B, int64_t L, int64_t H, int64_t runs,
           float* __restrict__ behind, float* __restrict__ dh0) {
  const int64_t k = blockIdx.x * (int64_t)kThreads + threadIdx.x;
  if (k >= B * H) return;
  const int64_t b = k / H, h = k % H;
  float G = dh_last ? dh_last[k] : 0.0f;
  for (int64_t run = runs - 1; run >= 0; --run) {
    const int64_t at = (b * runs + run) * H + h;
    if (!DLR_IN(at, B * runs * H)) break;
    behind[at] = G;
    const float2 g = agg[at];
    const bool cut = run_cut(reset, b, L, run * kRun, (int)min((int64_t)kRun, L - run * kRun));
    G = cut ? g.y : fmaf(g.x, G, g.y);
  }
  if (dh0) dh0[k] = G;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
back_apply(ScanIn<T> in, view<const T> dy, const float* __restrict__ states,
           const float* __restrict__ behind, view<T> dx, view<T> dr, view<T> di,
           float* __restrict__ part) {
  __shared__ float before[kRun][kThreads];  // the state before each step
  const Place q = place(in);
  if (!q.on) return;
  const float k = in.c * softplus(in.p[q.h]), kz = -k * kLog2e;
  const int64_t at = (q.b * in.runs + q.run) * in.H + q.h;
  float s = states[at];
  for (int j = 0; j < q.steps; ++j) {
    const int64_t t = q.t0 + j;
    const gate g = make_gate(to_f(in.r.row(q.b, t)[q.h]), to_f(in.i.row(q.b, t)[q.h]), kz);
    if (in.reset && in.reset[q.b * in.L + t]) s = 0.0f;
    before[j][threadIdx.x] = s;
    s = fmaf(g.a, s, g.m * g.si * to_f(in.x.row(q.b, t)[q.h]));
  }
  float C = behind[at], sum = 0.0f;
  for (int j = q.steps - 1; j >= 0; --j) {
    const int64_t t = q.t0 + j;
    const gate g = make_gate(to_f(in.r.row(q.b, t)[q.h]), to_f(in.i.row(q.b, t)[q.h]), kz);
    const bool cut = in.reset && in.reset[q.b * in.L + t];
    const float G = to_f(dy.row(q.b, t)[q.h]) + C;
    const float x = to_f(in.x.row(q.b, t)[q.h]), sx = g.si * x;
    const float E = G * g.a * (before[j][threadIdx.x] - g.a * g.rm * sx) * g.sr;
    sum += E;
    const float Gm = G * g.m;
    dx.row(q.b, t)[q.h] = from_f<T>(Gm * g.si);
    di.row(q.b, t)[q.h] = from_f<T>(Gm * sx * (1.0f - g.si));
    dr.row(q.b, t)[q.h] = from_f<T>(-k * E * (1.0f - g.sr));
    C = cut ? 0.0f : g.a * G;
  }
  part[at] = sum;
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

template <typename T>
__global__ void __launch_bounds__(kThreads)
step_kernel(ScanIn<T> in, const float* h, view<T> y, float* h_out) {
  const int64_t k = blockIdx.x * (int64_t)kThreads + threadIdx.x;
  if (k >= in.B * in.H) return;
  const int64_t b = k / in.H, ch = k % in.H;
  const float kz = -in.c * softplus(in.p[ch]) * kLog2e;
  const gate g = make_gate(to_f(in.r.row(b, 0)[ch]), to_f(in.i.row(b, 0)[ch]), kz);
  const float bt = g.m * g.si * to_f(in.x.row(b, 0)[ch]);
  const float s = in.reset && in.reset[b] ? bt : fmaf(g.a, h[k], bt);
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

template <typename T>
cudaError_t scan_t(const glr_scan_args& a, cudaStream_t s) {
  const int64_t runs = glr_states(a.L), n = a.B * runs * a.H;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  float2* agg = reinterpret_cast<float2*>(ws);
  float* states = a.states ? a.states
                           : reinterpret_cast<float*>(ws + align256(sizeof(float2) * (size_t)n));
  ScanIn<T> in{in_view<T>(a.x), in_view<T>(a.r), in_view<T>(a.i), a.p, a.reset, a.B, a.L, a.H,
               runs, (float)a.c};
  const int64_t blocks = a.B * runs * ((a.H + kThreads - 1) / kThreads);
  scan_runs<T><<<(unsigned)blocks, kThreads, 0, s>>>(in, agg);
  const int64_t rows = (a.B * a.H + kThreads - 1) / kThreads;
  scan_carry<<<(unsigned)rows, kThreads, 0, s>>>(agg, a.h0, a.reset, a.B, a.L, a.H, runs, states,
                                                 a.h_last);
  scan_apply<T><<<(unsigned)blocks, kThreads, 0, s>>>(in, states, out_view<T>(a.y));
  return cudaGetLastError();
}

template <typename T>
cudaError_t back_t(const glr_scan_backward_args& a, cudaStream_t s) {
  const int64_t runs = glr_states(a.L), n = a.B * runs * a.H;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  float2* agg = reinterpret_cast<float2*>(ws);
  float* behind = reinterpret_cast<float*>(ws + align256(sizeof(float2) * (size_t)n));
  float* part = reinterpret_cast<float*>(ws + align256(sizeof(float2) * (size_t)n) +
                                         align256(sizeof(float) * (size_t)n));
  ScanIn<T> in{in_view<T>(a.x), in_view<T>(a.r), in_view<T>(a.i), a.p, a.reset, a.B, a.L, a.H,
               runs, (float)a.c};
  const int64_t blocks = a.B * runs * ((a.H + kThreads - 1) / kThreads);
  back_runs<T><<<(unsigned)blocks, kThreads, 0, s>>>(in, in_view<T>(a.dy), agg);
  const int64_t rows = (a.B * a.H + kThreads - 1) / kThreads;
  back_carry<<<(unsigned)rows, kThreads, 0, s>>>(agg, a.dh_last, a.reset, a.B, a.L, a.H, runs,
                                                 behind, a.dh0);
  back_apply<T><<<(unsigned)blocks, kThreads, 0, s>>>(in, in_view<T>(a.dy), a.states, behind,
                                                      out_view<T>(a.dx), out_view<T>(a.dr),
                                                      out_view<T>(a.di), part);
  back_sum<<<(unsigned)((a.H + 31) / 32), 256, 0, s>>>(part, a.B * runs, a.H, a.p, (float)a.c,
                                                       a.dp);
  return cudaGetLastError();
}

template <typename T>
cudaError_t step_t(const glr_step_args& a, cudaStream_t s) {
  ScanIn<T> in{in_view<T>(a.x), in_view<T>(a.r), in_view<T>(a.i), a.p, a.reset, a.B, 1, a.H, 1,
               (float)a.c};
  const int64_t blocks = (a.B * a.H + kThreads - 1) / kThreads;
  step_kernel<T><<<(unsigned)blocks, kThreads, 0, s>>>(in, a.h, out_view<T>(a.y), a.h_out);
  return cudaGetLastError();
}

}  // namespace

size_t scan_workspace_bytes(int64_t B, int64_t L, int64_t H) {
  const size_t n = (size_t)B * (size_t)glr_states(L) * (size_t)H;
  return align256(sizeof(float2) * n) + align256(sizeof(float) * n);
}
size_t scan_backward_workspace_bytes(int64_t B, int64_t L, int64_t H) {
  const size_t n = (size_t)B * (size_t)glr_states(L) * (size_t)H;
  return align256(sizeof(float2) * n) + 2 * align256(sizeof(float) * n);
}
// blocks of the largest grid that a call of this size launches
int64_t scan_blocks(int64_t B, int64_t L, int64_t H) {
  return B * glr_states(L) * ((H + kThreads - 1) / kThreads);
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
