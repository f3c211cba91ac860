// ssm_api.cu -- the extern "C" entry points declared in include/ssm.h: argument validation and
// kernel dispatch on the caller's stream.
#include <cuda_runtime.h>

#include "call_args.cuh"
#include "ssm.h"

namespace dlr {
dlr_status status_from_cuda(cudaError_t e);

namespace ssm {
int64_t conv_blocks(int64_t B, int64_t L, int64_t H);
size_t conv_backward_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t K);
cudaError_t launch_conv(const ssm_conv_args& a, cudaStream_t s);
cudaError_t launch_conv_backward(const ssm_conv_backward_args& a, cudaStream_t s);
cudaError_t launch_conv_step(const ssm_conv_step_args& a, cudaStream_t s);
size_t scan_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t N, int64_t G);
size_t scan_backward_workspace_bytes(int64_t B, int64_t L, int64_t H, int64_t N, int64_t G);
cudaError_t launch_scan(const ssm_scan_args& a, cudaStream_t s);
cudaError_t launch_scan_backward(const ssm_scan_backward_args& a, cudaStream_t s);
cudaError_t launch_step(const ssm_step_args& a, cudaStream_t s);
}  // namespace ssm
}  // namespace dlr

namespace {

using namespace dlr::args;

constexpr int64_t kMaxH = int64_t(1) << 24;
// elements that one call's activations, and items that one launch's threads, may count
constexpr int64_t kMaxItems = int64_t(1) << 38;

// B, L >= 1 steps of H channels
bool too_many(int64_t B, int64_t L, int64_t H) {
  return B > kMaxGrid || L > kMaxGrid || H > kMaxH || B > kMaxItems / (L < 1 ? 1 : L) ||
         B * (L < 1 ? 1 : L) > kMaxItems / H;
}

dlr_status conv_sizes(int64_t type, int64_t B, int64_t L, int64_t H, int64_t K, int64_t act) {
  if (bad_type(type) || B < 1 || L < 0 || H < 1 || K < 1) return DLR_ERR_INVALID_ARG;
  if (act != SSM_ACT_SILU && act != SSM_ACT_NONE) return DLR_ERR_INVALID_ARG;
  if (K > SSM_MAX_TAPS || too_many(B, L, H)) return DLR_ERR_UNSUPPORTED;
  if (dlr::ssm::conv_blocks(B, L < 1 ? 1 : L, H) > kMaxGrid) return DLR_ERR_UNSUPPORTED;
  return DLR_OK;
}

dlr_status scan_sizes(int64_t type, int64_t B, int64_t L, int64_t H, int64_t N, int64_t G,
                      int64_t softplus) {
  if (bad_type(type) || B < 1 || L < 0 || H < 1 || N < 1 || G < 1 || H % G)
    return DLR_ERR_INVALID_ARG;
  if (softplus != 0 && softplus != 1) return DLR_ERR_INVALID_ARG;
  if (N > SSM_MAX_STATES || too_many(B, L, H)) return DLR_ERR_UNSUPPORTED;
  // blocks of a launch, and threads: a lane for each state of a group and step at most
  if (B * H > kMaxGrid || B * (L + 1) > kMaxItems / (128 * G)) return DLR_ERR_UNSUPPORTED;
  return DLR_OK;
}

bool bad_data(const void* p, int64_t type) { return p && !aligned(p, type_bytes(type)); }

dlr_status copy_or_clear(void* to, const void* from, int64_t bytes, cudaStream_t s) {
  if (!to || to == from || bytes == 0) return DLR_OK;
  return dlr::status_from_cuda(
      from ? cudaMemcpyAsync(to, from, (size_t)bytes, cudaMemcpyDeviceToDevice, s)
           : cudaMemsetAsync(to, 0, (size_t)bytes, s));
}

}  // namespace

extern "C" {

int ssm_abi_version(void) { return 1; }

dlr_status ssm_conv(const ssm_conv_args* args, dlr_stream_t stream) {
  if (!args) return DLR_ERR_INVALID_ARG;
  const ssm_conv_args& a = *args;
  const dlr_status st = conv_sizes(a.type, a.B, a.L, a.H, a.K, a.act);
  if (st != DLR_OK) return st;
  if (bad_data(a.state, a.type) || bad_data(a.last, a.type)) return DLR_ERR_INVALID_ARG;
  if (a.K == 1 && (a.state || a.last)) return DLR_ERR_INVALID_ARG;
  const int64_t rows = a.B * (a.K - 1) * a.H * type_bytes(a.type);
  if (a.L == 0) {
    if (a.state != a.last && may_overlap(flat(a.state, rows), flat(a.last, rows)))
      return DLR_ERR_INVALID_ARG;
    return copy_or_clear(a.last, a.state, rows, (cudaStream_t)stream);
  }
  if (bad_view(a.x, a.type, a.B, a.L) || bad_view(a.y, a.type, a.B, a.L) || bad_f32(a.w) ||
      bad_f32_or_null(a.bias))
    return DLR_ERR_INVALID_ARG;
  const Area in[] = {strided(a.x, a.type, a.B, a.L, a.H), flat(a.w, 4 * a.H * a.K),
                     flat(a.bias, 4 * a.H), flat(a.state, rows), flat(a.reset, a.B * a.L)};
  const Area out[] = {strided(a.y, a.type, a.B, a.L, a.H), flat(a.last, rows)};
  if (!distinct(out[0]) || meet(in, out)) return DLR_ERR_INVALID_ARG;
  return dlr::status_from_cuda(dlr::ssm::launch_conv(a, (cudaStream_t)stream));
}

size_t ssm_conv_backward_workspace_size(int64_t B, int64_t L, int64_t H, int64_t K) {
  if (L < 1 || conv_sizes(GLR_F32, B, L, H, K, SSM_ACT_SILU) != DLR_OK) return 0;
  return dlr::ssm::conv_backward_workspace_bytes(B, L, H, K);
}

dlr_status ssm_conv_backward(const ssm_conv_backward_args* args, dlr_stream_t stream) {
  if (!args) return DLR_ERR_INVALID_ARG;
  const ssm_conv_backward_args& a = *args;
  dlr_status st = conv_sizes(a.type, a.B, a.L, a.H, a.K, a.act);
  if (st != DLR_OK) return st;
  if (bad_data(a.state, a.type) || bad_data(a.dlast, a.type) || bad_data(a.dstate, a.type) ||
      bad_f32(a.dw) || bad_f32_or_null(a.dbias))
    return DLR_ERR_INVALID_ARG;
  if (a.K == 1 && (a.state || a.dlast || a.dstate)) return DLR_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t rows = a.B * (a.K - 1) * a.H * type_bytes(a.type);
  if (a.L == 0) {
    const Area in[] = {flat(a.dlast == a.dstate ? nullptr : a.dlast, rows)};
    const Area out[] = {flat(a.dstate, rows), flat(a.dw, 4 * a.H * a.K), flat(a.dbias, 4 * a.H)};
    if (meet(in, out)) return DLR_ERR_INVALID_ARG;
    st = copy_or_clear(a.dw, nullptr, 4 * a.H * a.K, s);
    if (st == DLR_OK) st = copy_or_clear(a.dbias, nullptr, 4 * a.H, s);
    return st == DLR_OK ? copy_or_clear(a.dstate, a.dlast, rows, s) : st;
  }
  if (bad_view(a.x, a.type, a.B, a.L) || bad_view(a.dy, a.type, a.B, a.L) ||
      bad_view(a.dx, a.type, a.B, a.L) || bad_f32(a.w) || bad_f32_or_null(a.bias))
    return DLR_ERR_INVALID_ARG;
  const size_t need = dlr::ssm::conv_backward_workspace_bytes(a.B, a.L, a.H, a.K);
  if ((st = bad_workspace(a.workspace, a.workspace_bytes, need)) != DLR_OK) return st;
  const Area in[] = {strided(a.x, a.type, a.B, a.L, a.H), strided(a.dy, a.type, a.B, a.L, a.H),
                     flat(a.w, 4 * a.H * a.K), flat(a.bias, 4 * a.H), flat(a.state, rows),
                     flat(a.dlast, rows), flat(a.reset, a.B * a.L)};
  const Area out[] = {strided(a.dx, a.type, a.B, a.L, a.H), flat(a.dw, 4 * a.H * a.K),
                      flat(a.dbias, 4 * a.H), flat(a.dstate, rows),
                      flat(a.workspace, (int64_t)need)};
  if (!distinct(out[0]) || meet(in, out)) return DLR_ERR_INVALID_ARG;
  return dlr::status_from_cuda(dlr::ssm::launch_conv_backward(a, s));
}

dlr_status ssm_conv_step(const ssm_conv_step_args* args, dlr_stream_t stream) {
  if (!args) return DLR_ERR_INVALID_ARG;
  const ssm_conv_step_args& a = *args;
  const dlr_status st = conv_sizes(a.type, a.B, 1, a.H, a.K, a.act);
  if (st != DLR_OK) return st;
  const bool keeps = a.K > 1;
  if (bad_view(a.x, a.type, a.B, 1) || bad_view(a.y, a.type, a.B, 1) || bad_f32(a.w) ||
      bad_f32_or_null(a.bias) || bad_data(a.state, a.type) || bad_data(a.state_out, a.type) ||
      keeps != (a.state != nullptr) || keeps != (a.state_out != nullptr))
    return DLR_ERR_INVALID_ARG;
  const int64_t rows = a.B * (a.K - 1) * a.H * type_bytes(a.type);
  const Area in[] = {strided(a.x, a.type, a.B, 1, a.H), flat(a.w, 4 * a.H * a.K),
                     flat(a.bias, 4 * a.H), flat(a.state == a.state_out ? nullptr : a.state, rows),
                     flat(a.reset, a.B)};
  const Area out[] = {strided(a.y, a.type, a.B, 1, a.H), flat(a.state_out, rows)};
  if (!distinct(out[0]) || meet(in, out)) return DLR_ERR_INVALID_ARG;
  return dlr::status_from_cuda(dlr::ssm::launch_conv_step(a, (cudaStream_t)stream));
}

int64_t ssm_states(int64_t L) { return L < 1 ? 0 : (L - 1) / SSM_STATE_STEPS + 1; }

size_t ssm_scan_workspace_size(int64_t B, int64_t L, int64_t H, int64_t N, int64_t G) {
  if (L < 1 || scan_sizes(GLR_F32, B, L, H, N, G, 1) != DLR_OK) return 0;
  return dlr::ssm::scan_workspace_bytes(B, L, H, N, G);
}

dlr_status ssm_scan(const ssm_scan_args* args, dlr_stream_t stream) {
  if (!args) return DLR_ERR_INVALID_ARG;
  const ssm_scan_args& a = *args;
  dlr_status st = scan_sizes(a.type, a.B, a.L, a.H, a.N, a.G, a.softplus);
  if (st != DLR_OK) return st;
  if (bad_f32_or_null(a.h0) || bad_f32_or_null(a.h_last)) return DLR_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t bhn = 4 * a.B * a.H * a.N, gn = a.G * a.N;
  if (a.L == 0) {
    if (a.h0 != a.h_last && may_overlap(flat(a.h0, bhn), flat(a.h_last, bhn)))
      return DLR_ERR_INVALID_ARG;
    return copy_or_clear(a.h_last, a.h0, bhn, s);
  }
  if (bad_view(a.x, a.type, a.B, a.L) || bad_view(a.dt, a.type, a.B, a.L) ||
      (a.z.data && bad_view(a.z, a.type, a.B, a.L)) || bad_view(a.Bm, a.type, a.B, a.L) ||
      bad_view(a.Cm, a.type, a.B, a.L) || bad_view(a.y, a.type, a.B, a.L) || bad_f32(a.A) ||
      bad_f32_or_null(a.D) || bad_f32_or_null(a.dt_bias) || bad_f32_or_null(a.states))
    return DLR_ERR_INVALID_ARG;
  const size_t need = dlr::ssm::scan_workspace_bytes(a.B, a.L, a.H, a.N, a.G);
  if ((st = bad_workspace(a.workspace, a.workspace_bytes, need)) != DLR_OK) return st;
  auto act = [&](const auto& v, int64_t n) { return strided(v, a.type, a.B, a.L, n); };
  const Area in[] = {act(a.x, a.H), act(a.dt, a.H), act(a.z, a.H), act(a.Bm, gn), act(a.Cm, gn),
                     flat(a.A, 4 * a.H * a.N), flat(a.D, 4 * a.H), flat(a.dt_bias, 4 * a.H),
                     flat(a.h0, bhn), flat(a.reset, a.B * a.L)};
  const Area out[] = {act(a.y, a.H), flat(a.h_last, bhn), flat(a.states, bhn * ssm_states(a.L)),
                      flat(need ? a.workspace : nullptr, (int64_t)need)};
  if (!distinct(out[0]) || meet(in, out)) return DLR_ERR_INVALID_ARG;
  return dlr::status_from_cuda(dlr::ssm::launch_scan(a, s));
}

size_t ssm_scan_backward_workspace_size(int64_t B, int64_t L, int64_t H, int64_t N, int64_t G) {
  if (L < 1 || scan_sizes(GLR_F32, B, L, H, N, G, 1) != DLR_OK) return 0;
  return dlr::ssm::scan_backward_workspace_bytes(B, L, H, N, G);
}

dlr_status ssm_scan_backward(const ssm_scan_backward_args* args, dlr_stream_t stream) {
  if (!args) return DLR_ERR_INVALID_ARG;
  const ssm_scan_backward_args& a = *args;
  dlr_status st = scan_sizes(a.type, a.B, a.L, a.H, a.N, a.G, a.softplus);
  if (st != DLR_OK) return st;
  if (bad_f32_or_null(a.h0) || bad_f32_or_null(a.dh_last) || bad_f32_or_null(a.dh0) ||
      bad_f32(a.dA) || bad_f32_or_null(a.D) || bad_f32_or_null(a.dD) ||
      bad_f32_or_null(a.ddt_bias) || (a.D != nullptr) != (a.dD != nullptr))
    return DLR_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t bhn = 4 * a.B * a.H * a.N, gn = a.G * a.N, h4 = 4 * a.H;
  if (a.L == 0) {
    const Area in[] = {flat(a.dh_last == a.dh0 ? nullptr : a.dh_last, bhn)};
    const Area out[] = {flat(a.dA, h4 * a.N), flat(a.dD, h4), flat(a.ddt_bias, h4),
                        flat(a.dh0, bhn)};
    if (meet(in, out)) return DLR_ERR_INVALID_ARG;
    st = copy_or_clear(a.dA, nullptr, h4 * a.N, s);
    if (st == DLR_OK) st = copy_or_clear(a.dD, nullptr, h4, s);
    if (st == DLR_OK) st = copy_or_clear(a.ddt_bias, nullptr, h4, s);
    return st == DLR_OK ? copy_or_clear(a.dh0, a.dh_last, bhn, s) : st;
  }
  const bool gated = a.z.data;
  if (bad_view(a.x, a.type, a.B, a.L) || bad_view(a.dt, a.type, a.B, a.L) ||
      bad_view(a.Bm, a.type, a.B, a.L) || bad_view(a.Cm, a.type, a.B, a.L) ||
      bad_view(a.dy, a.type, a.B, a.L) || bad_view(a.dx, a.type, a.B, a.L) ||
      bad_view(a.ddt, a.type, a.B, a.L) || bad_view(a.dBm, a.type, a.B, a.L) ||
      bad_view(a.dCm, a.type, a.B, a.L) || bad_f32(a.A) || bad_f32_or_null(a.dt_bias) ||
      bad_f32(a.states))
    return DLR_ERR_INVALID_ARG;
  if (gated ? bad_view(a.z, a.type, a.B, a.L) || bad_view(a.dz, a.type, a.B, a.L)
            : a.dz.data != nullptr)
    return DLR_ERR_INVALID_ARG;
  const size_t need = dlr::ssm::scan_backward_workspace_bytes(a.B, a.L, a.H, a.N, a.G);
  if ((st = bad_workspace(a.workspace, a.workspace_bytes, need)) != DLR_OK) return st;
  auto act = [&](const auto& v, int64_t n) { return strided(v, a.type, a.B, a.L, n); };
  const Area in[] = {act(a.x, a.H), act(a.dt, a.H), act(a.z, a.H), act(a.Bm, gn), act(a.Cm, gn),
                     act(a.dy, a.H), flat(a.A, h4 * a.N), flat(a.D, h4), flat(a.dt_bias, h4),
                     flat(a.h0, bhn), flat(a.reset, a.B * a.L),
                     flat(a.states, bhn * ssm_states(a.L)), flat(a.dh_last, bhn)};
  const Area out[] = {act(a.dx, a.H), act(a.ddt, a.H), act(a.dBm, gn), act(a.dCm, gn),
                      act(a.dz, a.H), flat(a.dA, h4 * a.N), flat(a.dD, h4), flat(a.ddt_bias, h4),
                      flat(a.dh0, bhn), flat(a.workspace, (int64_t)need)};
  for (int k = 0; k < 5; ++k)
    if (out[k].p && !distinct(out[k])) return DLR_ERR_INVALID_ARG;
  if (meet(in, out)) return DLR_ERR_INVALID_ARG;
  return dlr::status_from_cuda(dlr::ssm::launch_scan_backward(a, s));
}

dlr_status ssm_step(const ssm_step_args* args, dlr_stream_t stream) {
  if (!args) return DLR_ERR_INVALID_ARG;
  const ssm_step_args& a = *args;
  const dlr_status st = scan_sizes(a.type, a.B, 1, a.H, a.N, a.G, a.softplus);
  if (st != DLR_OK) return st;
  if (bad_view(a.x, a.type, a.B, 1) || bad_view(a.dt, a.type, a.B, 1) ||
      (a.z.data && bad_view(a.z, a.type, a.B, 1)) || bad_view(a.Bm, a.type, a.B, 1) ||
      bad_view(a.Cm, a.type, a.B, 1) || bad_view(a.y, a.type, a.B, 1) || bad_f32(a.A) ||
      bad_f32_or_null(a.D) || bad_f32_or_null(a.dt_bias) || bad_f32(a.h) || bad_f32(a.h_out))
    return DLR_ERR_INVALID_ARG;
  const int64_t bhn = 4 * a.B * a.H * a.N, gn = a.G * a.N;
  auto act = [&](const auto& v, int64_t n) { return strided(v, a.type, a.B, 1, n); };
  const Area in[] = {act(a.x, a.H), act(a.dt, a.H), act(a.z, a.H), act(a.Bm, gn), act(a.Cm, gn),
                     flat(a.A, 4 * a.H * a.N), flat(a.D, 4 * a.H), flat(a.dt_bias, 4 * a.H),
                     flat(a.h == a.h_out ? nullptr : a.h, bhn), flat(a.reset, a.B)};
  const Area out[] = {act(a.y, a.H), flat(a.h_out, bhn)};
  if (!distinct(out[0]) || meet(in, out)) return DLR_ERR_INVALID_ARG;
  return dlr::status_from_cuda(dlr::ssm::launch_step(a, (cudaStream_t)stream));
}

}  // extern "C"
