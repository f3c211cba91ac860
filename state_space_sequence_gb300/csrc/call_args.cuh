// call_args.cuh -- checks of a call's arguments shared by the extern "C" entry points: types,
// alignment, strides, workspaces, and the rule that no output meets an input or another output.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "glr.h"

namespace dlr {
namespace args {

constexpr int64_t kMaxGrid = 2147483647;
constexpr int64_t kMaxStride = int64_t(1) << 40;

inline bool bad_type(int64_t t) { return t != GLR_F32 && t != GLR_BF16 && t != GLR_F16; }
inline int64_t type_bytes(int64_t t) { return t == GLR_F32 ? 4 : 2; }
inline bool aligned(const void* p, int64_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(n - 1)) == 0;
}

// An array of `ob` x `ot` rows of `n` elements of `size` bytes, for the overlap rules.
struct Area {
  uintptr_t p;
  int64_t size, n, ob, ot, sb, st;
  uintptr_t end() const {
    return p + (uintptr_t)(((ob - 1) * sb + (ot - 1) * st + n) * size);
  }
};
inline Area flat(const void* p, int64_t bytes) {
  return {reinterpret_cast<uintptr_t>(p), 1, bytes, 1, 1, 0, 0};
}
template <typename V>
Area strided(const V& v, int64_t type, int64_t B, int64_t L, int64_t H) {
  return {reinterpret_cast<uintptr_t>(v.data), type_bytes(type), H, B, L,
          B > 1 ? v.stride_b : 0, L > 1 ? v.stride_t : 0};
}

// True unless the two are known to share no element: their ranges are apart, or they are columns
// of the same rows (equal strides of which every one is a multiple of the smallest, the pitch)
// that do not meet.
inline bool may_overlap(const Area& a, const Area& b) {
  if (!a.p || !b.p || a.end() <= b.p || b.end() <= a.p) return false;
  if (a.size != b.size || a.ob != b.ob || a.ot != b.ot || a.sb != b.sb || a.st != b.st) return true;
  int64_t pitch = 0;
  if (a.ob > 1) pitch = a.sb;
  if (a.ot > 1 && (pitch == 0 || a.st < pitch)) pitch = a.st;
  if (pitch <= 0 || (a.ob > 1 && a.sb % pitch) || (a.ot > 1 && a.st % pitch)) return true;
  const int64_t bytes = (int64_t)(b.p - a.p);
  if (bytes % a.size) return true;
  int64_t d = (bytes / a.size) % pitch;
  if (d < 0) d += pitch;
  return d < a.n || d + b.n > pitch;
}

// An output's rows must be distinct: one of the two strides steps over all that the other spans.
inline bool distinct(const Area& a) {
  if (a.ob > 1 && a.sb < a.n) return false;
  if (a.ot > 1 && a.st < a.n) return false;
  if (a.ob <= 1 || a.ot <= 1) return true;
  return a.sb >= (a.ot - 1) * a.st + a.n || a.st >= (a.ob - 1) * a.sb + a.n;
}

inline bool bad_strides(int64_t sb, int64_t st) {
  return sb < 0 || st < 0 || sb > kMaxStride || st > kMaxStride;
}
template <typename V>
bool bad_view(const V& v, int64_t type) {
  return !v.data || !aligned(v.data, type_bytes(type)) || bad_strides(v.stride_b, v.stride_t);
}
// The same for an array of B x L rows, whose last must not lie past what addresses reach.
template <typename V>
bool bad_view(const V& v, int64_t type, int64_t B, int64_t L) {
  return bad_view(v, type) ||
         (__int128)(B - 1) * v.stride_b + (__int128)(L - 1) * v.stride_t > (int64_t(1) << 45);
}
inline bool bad_f32(const float* p) { return !p || !aligned(p, 4); }
inline bool bad_f32_or_null(const float* p) { return p && !aligned(p, 4); }

// No output may meet an input or another output.
template <int I, int O>
bool meet(const Area (&in)[I], const Area (&out)[O]) {
  for (int o = 0; o < O; ++o) {
    if (!out[o].p) continue;
    for (int i = 0; i < I; ++i)
      if (may_overlap(in[i], out[o])) return true;
    for (int k = o + 1; k < O; ++k)
      if (may_overlap(out[o], out[k])) return true;
  }
  return false;
}

inline dlr_status bad_workspace(const void* ws, uint64_t bytes, size_t need) {
  return need && (!ws || !aligned(ws, 16) || bytes < need) ? DLR_ERR_WORKSPACE : DLR_OK;
}

}  // namespace args
}  // namespace dlr
