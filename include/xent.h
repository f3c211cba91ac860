/*
 * xent.h -- C ABI of libdlr.so, fourth header: the softmax cross entropy of a projection onto a
 * vocabulary, the loss that trains a language model, on one NVIDIA GB300 GPU (sm_103a). The logits
 * are formed tile by tile and piece by piece of the vocabulary and never kept whole.
 *
 * Status codes, streams, workspaces and the device status word are those of dlr.h; types and the
 * rules for outputs are those of glr.h. Arguments come in one struct per call (all fields 8 bytes
 * wide; unused pointers NULL).
 */
#ifndef XENT_H_
#define XENT_H_

#include "glr.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rows h and W are read as they lie where they have 16 bits, begin on multiples of 16 bytes and are a
 * multiple of 8 elements and no less than D apart (M = 1 or V = 1: at any distance); other rows, and
 * float32's, are laid out anew in the workspace. The size queries count on that for both. Their answer
 * is without it for the rows that a flag added to the (16-bit) type names, and is then what calls with
 * such rows need.
 */
#define XENT_H_IN_PLACE 16 /* of xent_loss; xent_loss_backward always lays h out */
#define XENT_W_IN_PLACE 32

/*
 * xent_loss -- for rows h [M, D] and the vocabulary's rows W [V, D] (contiguous channels, rows
 * `stride_t` elements apart, stride_b unused, one type), with z = h W^T:
 *   lse[m] = log sum_v exp z[m, v],   loss[m] = lse[m] - z[m, target[m]]
 * target: int64 [M]. A row whose target is outside 0 .. V-1 (-1, -100: the end of a sequence,
 * padding) has the loss 0, whatever h holds there. loss and lse are float32 [M]. Products are exact
 * and summed in float32 (float32 inputs: as three bfloat16 parts of each value, six products of the nine).
 * The tensor core adds 16 of them at a time and cuts off where it adds, up to 2^-23 of the sum so far; so
 * sums are formed in pieces that are added up with rounding: of 256 terms for up to 128 rows of 16 bits, of
 * the whole sum for more rows as far as D = 4096 and of 2048 terms beyond, of 512 for float32. The
 * target's logit of more than 128 rows of 16 bits is formed once more by itself, rounded to nearest. A
 * row's loss may therefore differ in its last digits with the number of rows in the call.
 * M >= 0; V, D >= 1; M, V < 2^31 - 256; D <= 2^20. workspace: xent_loss_workspace_size(type, M, V,
 * D) bytes, 256-byte aligned.
 */
typedef struct {
  int64_t type, M, V, D;
  glr_view h, W;
  const int64_t* target;
  float* loss;
  float* lse;
  void* workspace;
  uint64_t workspace_bytes;
} xent_loss_args;
size_t xent_loss_workspace_size(int64_t type, int64_t M, int64_t V, int64_t D);
dlr_status xent_loss(const xent_loss_args* args, dlr_stream_t stream);

/*
 * xent_loss_backward -- the gradients of xent_loss for a loss whose gradient with respect to
 * loss[m] is dloss[m] (float32 [M]); h, W and target as the forward call had them, lse as it left
 * it:
 *   d[m, v] = dloss[m] (exp(z[m, v] - lse[m]) - (v == target[m])),   0 in rows without a target
 *   dh = d W [M, D],   dW = d^T h [V, D]
 * dh or dW may have data NULL: not wanted. Rows without a target add nothing to dW, whatever h
 * holds there, and their dh is 0 where W is finite. The logits are formed again, piece by piece of
 * the vocabulary (of columns whose d takes 256 MB, or of 256 columns where they take more); d is rounded
 * to the inputs' type before its two products (float32: kept in three parts), whose sums are formed whole
 * as far as 16384 terms and in pieces of 4096 beyond (float32: of 512). In 16 bits d is first
 * divided by the largest |dloss| (float16: over 2^14): under a mean the weights are then 1. workspace:
 * xent_loss_backward_workspace_size(type, M, V, D) bytes, 256-byte aligned. M = 0 writes dW = 0.
 */
typedef struct {
  int64_t type, M, V, D;
  glr_view h, W;
  const int64_t* target;
  const float* lse;
  const float* dloss;
  glr_out dh, dW;
  void* workspace;
  uint64_t workspace_bytes;
} xent_loss_backward_args;
size_t xent_loss_backward_workspace_size(int64_t type, int64_t M, int64_t V, int64_t D);
dlr_status xent_loss_backward(const xent_loss_backward_args* args, dlr_stream_t stream);

/* Version of this header's interface (incremented on any signature change or added entry point). */
int xent_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* XENT_H_ */
