// xent_api.cu -- the extern "C" entry points declared in include/xent.h: argument validation and
// kernel dispatch on the caller's stream.
#include <cuda_runtime.h>

#include "call_args.cuh"
#include "xent.h"

namespace dlr {
dlr_status status_from_cuda(cudaError_t e);

namespace xent {
size_t loss_workspace_bytes(int64_t type, int64_t M, int64_t V, int64_t D, bool h_there,
                            bool w_there);
size_t loss_workspace_bytes(const xent_loss_args& a);
size_t loss_backward_workspace_bytes(int64_t type, int64_t M, int64_t V, int64_t D, bool w_there);
size_t loss_backward_workspace_bytes(const xent_loss_backward_args& a);
cudaError_t launch_loss(const xent_loss_args& a, cudaStream_t s);
cudaError_t launch_loss_backward(const xent_loss_backward_args& a, cudaStream_t s);
cudaError_t clear_gradient(const glr_out& dW, int64_t type, int64_t V, int64_t D, cudaStream_t s);
}  // namespace xent
}  // namespace dlr

namespace {

using namespace dlr::args;

constexpr int64_t kMaxD = int64_t(1) << 20;
constexpr int64_t kMaxItems = int64_t(1) << 36;  // of h and of W

dlr_status sizes(int64_t type, int64_t M, int64_t V, int64_t D) {
  if (bad_type(type) || M < 0 || V < 1 || D < 1) return DLR_ERR_INVALID_ARG;
  if (M > kMaxGrid - 256 || V > kMaxGrid - 256 || D > kMaxD || M > kMaxItems / D ||
      V > kMaxItems / D)
    return DLR_ERR_UNSUPPORTED;
  return DLR_OK;
}

// The flags of a size query's type, which is left without them; those of float32 are not flags.
int64_t take_flags(int64_t& type) {
  const int64_t all = XENT_H_IN_PLACE | XENT_W_IN_PLACE, flags = type & all;
  if (type < 0 || (type & ~all) == GLR_F32) return 0;
  type &= ~all;
  return flags;
}

dlr_status bad_space(const void* ws, uint64_t bytes, size_t need) {
  return !ws || !aligned(ws, 256) || bytes < need ? DLR_ERR_WORKSPACE : DLR_OK;
}
bool bad_i64(const int64_t* p) { return !p || !aligned(p, 8); }

}  // namespace

extern "C" {

int xent_abi_version(void) { return 1; }

size_t xent_loss_workspace_size(int64_t type, int64_t M, int64_t V, int64_t D) {
  const int64_t there = take_flags(type);
  if (M < 1 || sizes(type, M, V, D) != DLR_OK) return 0;
  return dlr::xent::loss_workspace_bytes(type, M, V, D, there & XENT_H_IN_PLACE,
                                         there & XENT_W_IN_PLACE);
}

dlr_status xent_loss(const xent_loss_args* args, dlr_stream_t stream) {
  if (!args) return DLR_ERR_INVALID_ARG;
  const xent_loss_args& a = *args;
  dlr_status st = sizes(a.type, a.M, a.V, a.D);
  if (st != DLR_OK || a.M == 0) return st;
  if (bad_view(a.h, a.type, 1, a.M) || bad_view(a.W, a.type, 1, a.V) || bad_i64(a.target) ||
      bad_f32(a.loss) || bad_f32(a.lse))
    return DLR_ERR_INVALID_ARG;
  const size_t need = dlr::xent::loss_workspace_bytes(a);
  if ((st = bad_space(a.workspace, a.workspace_bytes, need)) != DLR_OK) return st;
  const Area in[] = {strided(a.h, a.type, 1, a.M, a.D), strided(a.W, a.type, 1, a.V, a.D),
                     flat(a.target, 8 * a.M)};
  const Area out[] = {flat(a.loss, 4 * a.M), flat(a.lse, 4 * a.M),
                      flat(a.workspace, (int64_t)need)};
  if (meet(in, out)) return DLR_ERR_INVALID_ARG;
  return dlr::status_from_cuda(dlr::xent::launch_loss(a, (cudaStream_t)stream));
}

size_t xent_loss_backward_workspace_size(int64_t type, int64_t M, int64_t V, int64_t D) {
  const int64_t there = take_flags(type);
  if (M < 1 || sizes(type, M, V, D) != DLR_OK) return 0;
  return dlr::xent::loss_backward_workspace_bytes(type, M, V, D, there & XENT_W_IN_PLACE);
}

dlr_status xent_loss_backward(const xent_loss_backward_args* args, dlr_stream_t stream) {
  if (!args) return DLR_ERR_INVALID_ARG;
  const xent_loss_backward_args& a = *args;
  dlr_status st = sizes(a.type, a.M, a.V, a.D);
  if (st != DLR_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (a.dW.data && bad_view(a.dW, a.type, 1, a.V)) return DLR_ERR_INVALID_ARG;
  const Area dW = strided(a.dW, a.type, 1, a.V, a.D);
  if (a.dW.data && !distinct(dW)) return DLR_ERR_INVALID_ARG;
  if (a.M == 0)
    return a.dW.data
               ? dlr::status_from_cuda(dlr::xent::clear_gradient(a.dW, a.type, a.V, a.D, s))
               : DLR_OK;
  if (bad_view(a.h, a.type, 1, a.M) || bad_view(a.W, a.type, 1, a.V) || bad_i64(a.target) ||
      bad_f32(a.lse) || bad_f32(a.dloss) || (a.dh.data && bad_view(a.dh, a.type, 1, a.M)))
    return DLR_ERR_INVALID_ARG;
  const size_t need = dlr::xent::loss_backward_workspace_bytes(a);
  if ((st = bad_space(a.workspace, a.workspace_bytes, need)) != DLR_OK) return st;
  const Area in[] = {strided(a.h, a.type, 1, a.M, a.D), strided(a.W, a.type, 1, a.V, a.D),
                     flat(a.target, 8 * a.M), flat(a.lse, 4 * a.M), flat(a.dloss, 4 * a.M)};
  const Area out[] = {strided(a.dh, a.type, 1, a.M, a.D), dW, flat(a.workspace, (int64_t)need)};
  if ((a.dh.data && !distinct(out[0])) || meet(in, out)) return DLR_ERR_INVALID_ARG;
  if (!a.dh.data && !a.dW.data) return DLR_OK;
  return dlr::status_from_cuda(dlr::xent::launch_loss_backward(a, s));
}

}  // extern "C"
