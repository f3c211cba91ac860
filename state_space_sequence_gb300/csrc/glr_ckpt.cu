// glr_ckpt.cu -- activations packed into 8-bit checkpoints and read back (include/glr.h): VEC
// channels to a thread, 32 / VEC threads to a group. Bound by memory, or by the launch where the
// array is small: 2041 x 1000 bfloat16 is packed and read back in 4.6 us.
#include "glr_join.cuh"

namespace dlr {
// source file number of the bounds-checked build's failing sites
[[maybe_unused]] constexpr int kSiteFile = 18;

namespace glr {
namespace {

template <typename T, int VEC>
__global__ void __launch_bounds__(256)
pack_kernel(Rows<const T> t, int64_t M, int H, uint8_t* __restrict__ codes,
            uint8_t* __restrict__ scales) {
  const int groups = (H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP;
  const int64_t k = (blockIdx.x * (int64_t)256 + threadIdx.x) * VEC;
  const int64_t group = k / GLR_CKPT_GROUP;
  const int64_t row = group / groups;
  const int c = (int)(group % groups) * GLR_CKPT_GROUP + (int)(k % GLR_CKPT_GROUP);
  const bool on = row < M && c < H && DLR_IN(row * H + c + VEC - 1, M * H);
  words<T, VEC> v;
  if (on) v.get(t.at(row, c));
  keep<T, VEC>(v, on, codes + row * H + c, scales + group);
}
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
unpack_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t M,
              int H, Rows<T> t) {
  const int groups = (H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP;
  const int64_t k = (blockIdx.x * (int64_t)256 + threadIdx.x) * VEC;
  const int64_t group = k / GLR_CKPT_GROUP;
  const int64_t row = group / groups;
  const int c = (int)(group % groups) * GLR_CKPT_GROUP + (int)(k % GLR_CKPT_GROUP);
  if (row >= M || c >= H || !DLR_IN(row * H + c + VEC - 1, M * H)) return;
  float v[VEC];
  words<uint8_t, VEC> item;
  item.get(codes + row * H + c);
  kept<VEC>(item, scales[group], v);
  store<T, VEC>(t.at(row, c), v);
}

template <typename T>
cudaError_t pack_t(int64_t M, int64_t H, const void* t, int64_t st, uint8_t* codes,
                   uint8_t* scales, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  const int64_t n = M * ((H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP) * GLR_CKPT_GROUP;
  const Rows<const T> r = rows<const T>(t, st);
  if (H % W == 0 && wide(t, st, sizeof(T)) && wide(codes, 0, 1))
    pack_kernel<T, W><<<(unsigned)((n / W + 255) / 256), 256, 0, s>>>(r, M, (int)H, codes, scales);
  else
    pack_kernel<T, 1><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(r, M, (int)H, codes, scales);
  return cudaGetLastError();
}
template <typename T>
cudaError_t unpack_t(int64_t M, int64_t H, const uint8_t* codes, const uint8_t* scales, void* t,
                     int64_t st, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  const int64_t n = M * ((H + GLR_CKPT_GROUP - 1) / GLR_CKPT_GROUP) * GLR_CKPT_GROUP;
  const Rows<T> r = rows<T>(t, st);
  if (H % W == 0 && wide(t, st, sizeof(T)) && wide(codes, 0, 1))
    unpack_kernel<T, W>
        <<<(unsigned)((n / W + 255) / 256), 256, 0, s>>>(codes, scales, M, (int)H, r);
  else
    unpack_kernel<T, 1><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(codes, scales, M, (int)H, r);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_pack(int64_t type, int64_t M, int64_t H, const void* t, int64_t st,
                        uint8_t* codes, uint8_t* scales, cudaStream_t s) {
  if (type == GLR_BF16) return pack_t<__nv_bfloat16>(M, H, t, st, codes, scales, s);
  if (type == GLR_F16) return pack_t<__half>(M, H, t, st, codes, scales, s);
  return pack_t<float>(M, H, t, st, codes, scales, s);
}
cudaError_t launch_unpack(int64_t type, int64_t M, int64_t H, const uint8_t* codes,
                          const uint8_t* scales, void* t, int64_t st, cudaStream_t s) {
  if (type == GLR_BF16) return unpack_t<__nv_bfloat16>(M, H, codes, scales, t, st, s);
  if (type == GLR_F16) return unpack_t<__half>(M, H, codes, scales, t, st, s);
  return unpack_t<float>(M, H, codes, scales, t, st, s);
}

}  // namespace glr
}  // namespace dlr
