// glr_api.cu -- the extern "C" entry points declared in include/glr.h: argument validation and
// kernel dispatch on the caller's stream.
#include <cuda_runtime.h>

#include <cmath>

#include "call_args.cuh"
#include "glr.h"

namespace dlr {
dlr_status status_from_cuda(cudaError_t e);

namespace glr {
size_t scan_workspace_bytes(int64_t B, int64_t L, int64_t H);
size_t scan_backward_workspace_bytes(int64_t B, int64_t L, int64_t H);
int64_t scan_tiles(int64_t B, int64_t L, int64_t H);
cudaError_t launch_scan(const glr_scan_args& a, cudaStream_t s);
cudaError_t launch_scan_backward(const glr_scan_backward_args& a, cudaStream_t s);
cudaError_t launch_step(const glr_step_args& a, cudaStream_t s);
size_t join_backward_workspace_bytes(int64_t H);
cudaError_t launch_join(const glr_join_args& a, cudaStream_t s);
cudaError_t launch_join_backward(const glr_join_backward_args& a, cudaStream_t s);
cudaError_t launch_pack(int64_t type, int64_t M, int64_t H, const void* t, int64_t st,
                        uint8_t* codes, uint8_t* scales, cudaStream_t s);
cudaError_t launch_unpack(int64_t type, int64_t M, int64_t H, const uint8_t* codes,
                          const uint8_t* scales, void* t, int64_t st, cudaStream_t s);
}  // namespace glr
}  // namespace dlr

namespace {

using namespace dlr::args;

constexpr int64_t kMaxH = int64_t(1) << 24;   // channels of the recurrence
constexpr int64_t kMaxRowH = 16384;           // channels of a joined row (held in registers)

dlr_status scan_sizes(int64_t type, int64_t B, int64_t L, int64_t H, double c) {
  if (bad_type(type) || B < 1 || L < 0 || H < 1) return DLR_ERR_INVALID_ARG;
  if (!(c >= 0.0) || !std::isfinite((float)c)) return DLR_ERR_INVALID_ARG;
  if (B > kMaxGrid || L > kMaxGrid || H > kMaxH) return DLR_ERR_UNSUPPORTED;
  // B * L * H < 2^86 could overflow: bound the rows first
  if (B * ((L + 63) / 64 + 1) > kMaxGrid || dlr::glr::scan_tiles(B, L, H) > kMaxGrid)
    return DLR_ERR_UNSUPPORTED;
  return DLR_OK;
}

}  // namespace

extern "C" {

int glr_abi_version(void) { return 1; }

int64_t glr_states(int64_t L) { return L < 1 ? 0 : (L - 1) / GLR_STATE_STEPS + 1; }

size_t glr_scan_workspace_size(int64_t B, int64_t L, int64_t H) {
  if (L < 1 || scan_sizes(GLR_F32, B, L, H, 1.0) != DLR_OK) return 0;
  return dlr::glr::scan_workspace_bytes(B, L, H);
}

dlr_status glr_scan(const glr_scan_args* args, dlr_stream_t stream) {
  if (!args) return DLR_ERR_INVALID_ARG;
  const glr_scan_args& a = *args;
  dlr_status st = scan_sizes(a.type, a.B, a.L, a.H, a.c);
  if (st != DLR_OK) return st;
  if (bad_f32_or_null(a.h0) || bad_f32_or_null(a.h_last)) return DLR_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t bh = 4 * a.B * a.H;
  if (a.L == 0) {
    if (!a.h_last) return DLR_OK;
    if (a.h0 == a.h_last) return DLR_OK;
    if (may_overlap(flat(a.h0, bh), flat(a.h_last, bh))) return DLR_ERR_INVALID_ARG;
    return dlr::status_from_cuda(
        a.h0 ? cudaMemcpyAsync(a.h_last, a.h0, (size_t)bh, cudaMemcpyDeviceToDevice, s)
             : cudaMemsetAsync(a.h_last, 0, (size_t)bh, s));
  }
  if (bad_view(a.x, a.type) || bad_view(a.r, a.type) || bad_view(a.i, a.type) ||
      bad_view(a.y, a.type) || bad_f32(a.p) || bad_f32_or_null(a.states))
    return DLR_ERR_INVALID_ARG;
  const size_t need = dlr::glr::scan_workspace_bytes(a.B, a.L, a.H);
  if ((st = bad_workspace(a.workspace, a.workspace_bytes, need)) != DLR_OK) return st;
  const Area in[] = {strided(a.x, a.type, a.B, a.L, a.H), strided(a.r, a.type, a.B, a.L, a.H),
                     strided(a.i, a.type, a.B, a.L, a.H), flat(a.p, 4 * a.H), flat(a.h0, bh),
                     flat(a.reset, a.B * a.L)};
  const Area out[] = {strided(a.y, a.type, a.B, a.L, a.H), flat(a.h_last, bh),
                      flat(a.states, bh * glr_states(a.L)),
                      flat(need ? a.workspace : nullptr, (int64_t)need)};
  if (!distinct(out[0]) || meet(in, out)) return DLR_ERR_INVALID_ARG;
  return dlr::status_from_cuda(dlr::glr::launch_scan(a, s));
}

size_t glr_scan_backward_workspace_size(int64_t B, int64_t L, int64_t H) {
  if (L < 1 || scan_sizes(GLR_F32, B, L, H, 1.0) != DLR_OK) return 0;
  return dlr::glr::scan_backward_workspace_bytes(B, L, H);
}

dlr_status glr_scan_backward(const glr_scan_backward_args* args, dlr_stream_t stream) {
  if (!args) return DLR_ERR_INVALID_ARG;
  const glr_scan_backward_args& a = *args;
  dlr_status st = scan_sizes(a.type, a.B, a.L, a.H, a.c);
  if (st != DLR_OK) return st;
  if (bad_f32_or_null(a.h0) || bad_f32_or_null(a.dh_last) || bad_f32_or_null(a.dh0) ||
      bad_f32(a.dp))
    return DLR_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t bh = 4 * a.B * a.H;
  if (a.L == 0) {
    const Area in[] = {flat(a.dh_last, bh)};
    const Area out[] = {flat(a.dp, 4 * a.H), flat(a.dh0, bh)};
    if (meet(in, out)) return DLR_ERR_INVALID_ARG;
    cudaError_t e = cudaMemsetAsync(a.dp, 0, 4 * (size_t)a.H, s);
    if (e == cudaSuccess && a.dh0)
      e = a.dh_last ? cudaMemcpyAsync(a.dh0, a.dh_last, (size_t)bh, cudaMemcpyDeviceToDevice, s)
                    : cudaMemsetAsync(a.dh0, 0, (size_t)bh, s);
    return dlr::status_from_cuda(e);
  }
  if (bad_view(a.x, a.type) || bad_view(a.r, a.type) || bad_view(a.i, a.type) ||
      bad_view(a.dy, a.type) || bad_view(a.dx, a.type) || bad_view(a.dr, a.type) ||
      bad_view(a.di, a.type) || bad_f32(a.p) || bad_f32(a.states))
    return DLR_ERR_INVALID_ARG;
  const size_t need = dlr::glr::scan_backward_workspace_bytes(a.B, a.L, a.H);
  if ((st = bad_workspace(a.workspace, a.workspace_bytes, need)) != DLR_OK) return st;
  const Area in[] = {strided(a.x, a.type, a.B, a.L, a.H), strided(a.r, a.type, a.B, a.L, a.H),
                     strided(a.i, a.type, a.B, a.L, a.H), strided(a.dy, a.type, a.B, a.L, a.H),
                     flat(a.p, 4 * a.H), flat(a.h0, bh), flat(a.reset, a.B * a.L),
                     flat(a.states, bh * glr_states(a.L)), flat(a.dh_last, bh)};
  const Area out[] = {strided(a.dx, a.type, a.B, a.L, a.H), strided(a.dr, a.type, a.B, a.L, a.H),
                      strided(a.di, a.type, a.B, a.L, a.H), flat(a.dp, 4 * a.H), flat(a.dh0, bh),
                      flat(a.workspace, (int64_t)need)};
  if (!distinct(out[0]) || !distinct(out[1]) || !distinct(out[2]) || meet(in, out))
    return DLR_ERR_INVALID_ARG;
  return dlr::status_from_cuda(dlr::glr::launch_scan_backward(a, s));
}

dlr_status glr_step(const glr_step_args* args, dlr_stream_t stream) {
  if (!args) return DLR_ERR_INVALID_ARG;
  const glr_step_args& a = *args;
  dlr_status st = scan_sizes(a.type, a.B, 1, a.H, a.c);
  if (st != DLR_OK) return st;
  if (a.B > 4 * 65535) return DLR_ERR_UNSUPPORTED;  // four batch entries to a row of blocks
  if (bad_view(a.x, a.type) || bad_view(a.r, a.type) || bad_view(a.i, a.type) ||
      bad_view(a.y, a.type) || bad_f32(a.p) || bad_f32(a.h) || bad_f32(a.h_out))
    return DLR_ERR_INVALID_ARG;
  const int64_t bh = 4 * a.B * a.H;
  const Area in[] = {strided(a.x, a.type, a.B, 1, a.H), strided(a.r, a.type, a.B, 1, a.H),
                     strided(a.i, a.type, a.B, 1, a.H), flat(a.p, 4 * a.H), flat(a.reset, a.B),
                     flat(a.h == a.h_out ? nullptr : a.h, bh)};
  const Area out[] = {strided(a.y, a.type, a.B, 1, a.H), flat(a.h_out, bh)};
  if (!distinct(out[0]) || meet(in, out)) return DLR_ERR_INVALID_ARG;
  return dlr::status_from_cuda(dlr::glr::launch_step(a, (cudaStream_t)stream));
}

static dlr_status join_sizes(int64_t type, int64_t M, int64_t H, int64_t norm, int64_t act,
                             double eps) {
  if (bad_type(type) || M < 0 || H < 1) return DLR_ERR_INVALID_ARG;
  if (norm != GLR_NORM_RMS && norm != GLR_NORM_LAYER) return DLR_ERR_INVALID_ARG;
  if (act != GLR_ACT_SILU && act != GLR_ACT_SIGMOID && act != GLR_ACT_NONE)
    return DLR_ERR_INVALID_ARG;
  if (!((float)eps > 0.0f) || !std::isfinite((float)eps)) return DLR_ERR_INVALID_ARG;
  if (H > kMaxRowH || M > kMaxGrid) return DLR_ERR_UNSUPPORTED;
  return DLR_OK;
}

dlr_status glr_join(const glr_join_args* args, dlr_stream_t stream) {
  if (!args) return DLR_ERR_INVALID_ARG;
  const glr_join_args& a = *args;
  dlr_status st = join_sizes(a.type, a.M, a.H, a.norm, a.act, a.eps);
  if (st != DLR_OK) return st;
  const bool block = a.h.data, gated = block && a.act != GLR_ACT_NONE, next = a.v;
  if (a.M == 0) return DLR_OK;
  if (bad_view(a.x, a.type) || (!block && !next)) return DLR_ERR_INVALID_ARG;
  if (block ? bad_view(a.h, a.type) || bad_view(a.y, a.type) || bad_f32(a.w) || bad_f32(a.alpha)
            : a.y.data || a.w || a.alpha)
    return DLR_ERR_INVALID_ARG;
  if (gated ? bad_view(a.g, a.type) : a.g.data != nullptr) return DLR_ERR_INVALID_ARG;
  if (next ? bad_view(a.n, a.type) || bad_f32(a.v) : a.n.data != nullptr)
    return DLR_ERR_INVALID_ARG;
  const bool keep = a.hc || a.hs || a.gc || a.gs;
  if (keep && (!block || !a.hc || !a.hs || gated != (a.gc != nullptr) ||
               gated != (a.gs != nullptr)))
    return DLR_ERR_INVALID_ARG;
  const int64_t nc = a.M * a.H, ns = a.M * ((a.H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP);
  auto rows = [&](const auto& v) { return strided(v, a.type, 1, a.M, a.H); };
  // y may be x, and n may be h or g, in place
  auto same = [](const auto& p, const auto& q) {
    return p.data && p.data == q.data && p.stride_t == q.stride_t;
  };
  const Area x = rows(a.x), h = rows(a.h), g = rows(a.g), y = rows(a.y), n = rows(a.n);
  const Area in[] = {flat(a.w, 4 * a.H), flat(a.alpha, 4), flat(a.v, 4 * a.H)};
  const Area out[] = {y, n, flat(a.hc, nc), flat(a.hs, ns), flat(a.gc, nc), flat(a.gs, ns)};
  if ((y.p && !distinct(y)) || (n.p && !distinct(n)) || meet(in, out)) return DLR_ERR_INVALID_ARG;
  if ((may_overlap(x, y) && !same(a.x, a.y)) || may_overlap(h, y) || may_overlap(g, y) ||
      may_overlap(x, n) || (may_overlap(h, n) && !same(a.h, a.n)) ||
      (may_overlap(g, n) && !same(a.g, a.n)))
    return DLR_ERR_INVALID_ARG;
  for (int k = 2; k < 6; ++k)
    if (may_overlap(x, out[k]) || may_overlap(h, out[k]) || may_overlap(g, out[k]))
      return DLR_ERR_INVALID_ARG;
  return dlr::status_from_cuda(dlr::glr::launch_join(a, (cudaStream_t)stream));
}

size_t glr_join_backward_workspace_size(int64_t M, int64_t H) {
  if (M < 0 || H < 1 || H > kMaxRowH) return 0;
  return dlr::glr::join_backward_workspace_bytes(H);
}

dlr_status glr_join_backward(const glr_join_backward_args* args, dlr_stream_t stream) {
  if (!args) return DLR_ERR_INVALID_ARG;
  const glr_join_backward_args& a = *args;
  dlr_status st = join_sizes(a.type, a.M, a.H, a.norm, a.act, a.eps);
  if (st != DLR_OK) return st;
  const bool block = a.w, gated = block && a.act != GLR_ACT_NONE, next = a.v, kept = a.hc;
  const bool some = a.M > 0;
  if (!block && !next) return DLR_ERR_INVALID_ARG;
  if (some && (bad_view(a.x, a.type) || bad_view(a.dx, a.type))) return DLR_ERR_INVALID_ARG;
  if (some && a.dy.data && bad_view(a.dy, a.type)) return DLR_ERR_INVALID_ARG;
  if (next ? (some && bad_view(a.dn, a.type)) || bad_f32(a.v) || bad_f32(a.dv)
           : a.dn.data || a.dv)
    return DLR_ERR_INVALID_ARG;
  if (block ? bad_f32(a.w) || bad_f32(a.alpha) || bad_f32(a.dw) || bad_f32(a.dalpha) ||
                  (some && bad_view(a.dh, a.type))
            : a.alpha || a.dw || a.dalpha || a.dh.data || a.h.data || a.hc)
    return DLR_ERR_INVALID_ARG;
  if (gated ? some && bad_view(a.dg, a.type) : a.dg.data || a.g.data || a.gc)
    return DLR_ERR_INVALID_ARG;
  if (kept ? !a.hs || a.h.data || a.g.data || gated != (a.gc != nullptr) ||
                 gated != (a.gs != nullptr)
           : a.hs || a.gc || a.gs || (some && block && bad_view(a.h, a.type)) ||
                 (some && gated && bad_view(a.g, a.type)))
    return DLR_ERR_INVALID_ARG;
  const size_t need = dlr::glr::join_backward_workspace_bytes(a.H);
  if ((st = bad_workspace(a.workspace, a.workspace_bytes, need)) != DLR_OK) return st;
  const int64_t nc = a.M * a.H, ns = a.M * ((a.H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP);
  auto rows = [&](const auto& v) {
    return strided(v, a.type, 1, some ? a.M : 1, a.H);
  };
  const bool inplace = a.dy.data && a.dy.data == a.dx.data && a.dy.stride_t == a.dx.stride_t;
  const Area in[] = {rows(a.dn), rows(a.x), rows(a.h), rows(a.g), flat(a.hc, nc), flat(a.hs, ns),
                     flat(a.gc, nc), flat(a.gs, ns), flat(a.w, 4 * a.H), flat(a.alpha, 4),
                     flat(a.v, 4 * a.H), inplace ? flat(nullptr, 0) : rows(a.dy)};
  const Area out[] = {rows(a.dx), rows(a.dh), rows(a.dg), flat(a.dw, 4 * a.H), flat(a.dalpha, 4),
                      flat(a.dv, 4 * a.H), flat(a.workspace, (int64_t)need)};
  for (int k = 0; k < 3; ++k)
    if (out[k].p && !distinct(out[k])) return DLR_ERR_INVALID_ARG;
  if (meet(in, out)) return DLR_ERR_INVALID_ARG;
  return dlr::status_from_cuda(dlr::glr::launch_join_backward(a, (cudaStream_t)stream));
}

static dlr_status ckpt_args(int64_t type, int64_t M, int64_t H, const void* t, int64_t st,
                            const uint8_t* codes, const uint8_t* scales) {
  if (bad_type(type) || M < 0 || H < 1) return DLR_ERR_INVALID_ARG;
  // A thread for each channel at most, rows in whole groups and groups in blocks of 256 threads: as
  // many blocks as a launch may have, and channels that a kernel counts in 32 bits.
  if (H > kMaxGrid - GLR_CKPT_GROUP + 1) return DLR_ERR_UNSUPPORTED;
  const int64_t groups = (H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP;
  if (M > kMaxGrid * (256 / GLR_CKPT_GROUP) / groups) return DLR_ERR_UNSUPPORTED;
  if (M == 0) return DLR_OK;
  if (!t || !codes || !scales || !aligned(t, type_bytes(type)) || bad_strides(0, st))
    return DLR_ERR_INVALID_ARG;
  return DLR_OK;
}

dlr_status glr_ckpt_pack(int64_t type, int64_t M, int64_t H, const void* t, int64_t stride_t,
                         uint8_t* codes, uint8_t* scales, dlr_stream_t stream) {
  dlr_status st = ckpt_args(type, M, H, t, stride_t, codes, scales);
  if (st != DLR_OK || M == 0) return st;
  const int64_t groups = (H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP;
  const Area in[] = {strided(glr_view{t, 0, stride_t}, type, 1, M, H)};
  const Area out[] = {flat(codes, M * H), flat(scales, M * groups)};
  if (meet(in, out)) return DLR_ERR_INVALID_ARG;
  return dlr::status_from_cuda(
      dlr::glr::launch_pack(type, M, H, t, stride_t, codes, scales, (cudaStream_t)stream));
}

dlr_status glr_ckpt_unpack(int64_t type, int64_t M, int64_t H, const uint8_t* codes,
                           const uint8_t* scales, void* t, int64_t stride_t, dlr_stream_t stream) {
  dlr_status st = ckpt_args(type, M, H, t, stride_t, codes, scales);
  if (st != DLR_OK || M == 0) return st;
  const int64_t groups = (H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP;
  const Area in[] = {flat(codes, M * H), flat(scales, M * groups)};
  const Area out[] = {strided(glr_out{t, 0, stride_t}, type, 1, M, H)};
  if (!distinct(out[0]) || meet(in, out)) return DLR_ERR_INVALID_ARG;
  return dlr::status_from_cuda(
      dlr::glr::launch_unpack(type, M, H, codes, scales, t, stride_t, (cudaStream_t)stream));
}

}  // extern "C"
