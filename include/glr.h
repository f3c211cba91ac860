/*
 * glr.h -- C ABI of libdlr.so, second header: the operators of a gated recurrent block on one
 * NVIDIA GB300 GPU (sm_103a).
 *   - the gated linear recurrence (the diagonal recurrence of dlr.h with a decay that the token
 *     chooses): over a sequence, its gradients, and one token from a carried state;
 *   - the block's join: gate, norm, residual scale and add, and the next block's norm, with
 *     its gradients;
 *   - activation checkpoints in 8 bits, written by the join and read by its gradients.
 *
 * Status codes, streams, workspaces and the device status word are those of dlr.h: device
 * pointers owned by the caller, nothing allocated or kept, every call asynchronous on `stream`,
 * arguments checked on the host before anything is launched. Arguments come in one struct per
 * call (all fields 8 bytes wide; unused pointers NULL).
 *
 * Activations are float32, bfloat16 or float16 (`type`, one for all activations of a call),
 * aligned to their own size. A glr_view is an array [B, L, H] whose channels are contiguous;
 * `stride_b` and `stride_t` are in elements, so a view may be the columns of a wider projection
 * or a transposed batch. An input's strides may be 0 (broadcast); negative strides are refused.
 * An output's elements must be distinct, and no output may share an element with an input or
 * another output (the columns of one buffer do not). Parameters, states and their gradients are
 * float32 and contiguous. All arithmetic is float32; results are rounded once, to nearest even,
 * where they are stored in 16 bits.
 */
#ifndef GLR_H_
#define GLR_H_

#include "dlr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of the activations. */
typedef enum { GLR_F32 = 0, GLR_BF16 = 1, GLR_F16 = 2 } glr_type;

/* Norm of the join: root mean square, or layer (the mean taken off first). */
typedef enum { GLR_NORM_RMS = 0, GLR_NORM_LAYER = 1 } glr_norm;

/* Gate of the join: act(g) = g sigmoid(g), sigmoid(g), or 1 (no gate: g NULL). */
typedef enum { GLR_ACT_SILU = 0, GLR_ACT_SIGMOID = 1, GLR_ACT_NONE = 2 } glr_act;

typedef struct {
  const void* data;
  int64_t stride_b, stride_t;
} glr_view;

typedef struct {
  void* data;
  int64_t stride_b, stride_t;
} glr_out;

/* Steps between the states that glr_scan keeps for its gradients. */
#define GLR_STATE_STEPS 8

/*
 * glr_scan -- the gated linear recurrence over x [B, L, H] with the recurrence gate r and the
 * input gate i (both before their sigmoid), the decay parameter p [H] and the scale c >= 0:
 *   a_t = exp(-c softplus(p) sigmoid(r_t)),   b_t = sqrt(1 - a_t^2) sigmoid(i_t) x_t
 *   h_t = abar_t h_{t-1} + b_t,   abar_t = 0 where reset[b, t] != 0, else a_t
 * per channel, h_{-1} = h0 (float32 [B, H]; NULL: zero). y = h; h_last (float32 [B, H], may be
 * NULL) = h_{L-1}. reset: bytes [B, L], contiguous, NULL for none; a step that it marks begins a
 * new sequence: nothing before it, not even an infinity or a NaN, reaches it. Its input keeps the
 * factor sqrt(1 - a_t^2), as that of a sequence begun from a zero state (a model that was trained
 * with a factor of 1 at its documents' first steps gives other values there). A step whose i is
 * -inf adds nothing, whatever finite x it has.
 * states (NULL: not kept): float32 [B, glr_states(L), H], the state before each run of
 * GLR_STATE_STEPS steps, for glr_scan_backward.
 * workspace: glr_scan_workspace_size(B, L, H) bytes, 16-byte aligned (0 for short rows: none).
 * L = 0 copies h0 (or zero) to h_last. B, H >= 1; B and L < 2^31, H < 2^24.
 * Results do not depend on the order in which the GPU runs the blocks.
 */
typedef struct {
  int64_t type, B, L, H;
  double c;
  glr_view x, r, i;
  const float* p;
  const float* h0;
  const uint8_t* reset;
  glr_out y;
  float* h_last;
  float* states;
  void* workspace;
  uint64_t workspace_bytes;
} glr_scan_args;
int64_t glr_states(int64_t L);
size_t glr_scan_workspace_size(int64_t B, int64_t L, int64_t H);
dlr_status glr_scan(const glr_scan_args* args, dlr_stream_t stream);

/*
 * glr_scan_backward -- the gradients of glr_scan for a loss whose gradient with respect to y is
 * dy and, when dh_last (float32 [B, H]) is not NULL, with respect to h_last is dh_last. x, r, i,
 * p, c, h0 and reset as the forward call had them, states as it left them:
 *   G_t = dy_t + abar_{t+1} G_{t+1}  (G_{L-1} = dy_{L-1} + dh_last),  m = sqrt(1 - a^2)
 *   E_t = G_t (abar_t h_{t-1} - (a_t^2 / m_t) sigmoid(i_t) x_t)
 *   dx = G m sigmoid(i),   di = G m x sigmoid(i) (1 - sigmoid(i)),
 *   dr = -c softplus(p) E sigmoid(r) (1 - sigmoid(r)),
 *   dp [H] = -c sigmoid(p) sum_{b,t} E sigmoid(r),   dh0 [B, H] (may be NULL) = abar_0 G_0.
 * The states between the kept ones are computed again in float32. The sums of dp run in a fixed
 * order. workspace: glr_scan_backward_workspace_size(B, L, H) bytes, 16-byte aligned.
 * L = 0 writes dp = 0 and dh0 = dh_last (or 0).
 */
typedef struct {
  int64_t type, B, L, H;
  double c;
  glr_view x, r, i, dy;
  const float* p;
  const float* h0;
  const uint8_t* reset;
  const float* states;
  const float* dh_last;
  glr_out dx, dr, di;
  float* dp;
  float* dh0;
  void* workspace;
  uint64_t workspace_bytes;
} glr_scan_backward_args;
size_t glr_scan_backward_workspace_size(int64_t B, int64_t L, int64_t H);
dlr_status glr_scan_backward(const glr_scan_backward_args* args, dlr_stream_t stream);

/*
 * glr_step -- glr_scan for one token (L = 1; stride_t unused): y [B, H] and the state h_out from
 * the state h (float32 [B, H] both; h_out may be h). reset: bytes [B] or NULL. One launch.
 * B <= 262140.
 */
typedef struct {
  int64_t type, B, H;
  double c;
  glr_view x, r, i;
  const float* p;
  const float* h;
  const uint8_t* reset;
  glr_out y;
  float* h_out;
} glr_step_args;
dlr_status glr_step(const glr_step_args* args, dlr_stream_t stream);

/*
 * glr_join -- the end of a block and the norm that begins the next one, per row of H channels:
 *   u = h act(g),   y = x + alpha w norm(u),   n = v norm(y)
 *   norm(z) = z / sqrt(mean(z^2) + eps)                                   (GLR_NORM_RMS)
 *           = (z - mean(z)) / sqrt(mean((z - mean(z))^2) + eps)           (GLR_NORM_LAYER)
 * w, v: float32 [H]; alpha: one float32 on the device. x, h, g, y, n: rows of H contiguous
 * channels, `stride_t` elements apart (stride_b unused). n is formed from y before its rounding.
 * v and n NULL: no next norm. act GLR_ACT_NONE: no gate, g NULL. h NULL: y = x is not written
 * (y.data NULL) and only n = v norm(x) is formed (the norm before the first block); then w,
 * alpha and g are NULL.
 * y may be x, and n may be h or g, with the same stride: every row is read before it is written.
 * hc, hs, gc, gs (all NULL: none): h and g as 8-bit checkpoints in the layout of glr_ckpt_pack
 * (gc and gs NULL without a gate). M >= 0 rows; 1 <= H <= 16384; eps > 0.
 */
typedef struct {
  int64_t type, M, H, norm, act;
  double eps;
  glr_view x, h, g;
  const float* w;
  const float* alpha;
  const float* v;
  glr_out y, n;
  uint8_t* hc;
  uint8_t* hs;
  uint8_t* gc;
  uint8_t* gs;
} glr_join_args;
dlr_status glr_join(const glr_join_args* args, dlr_stream_t stream);

/*
 * glr_join_backward -- the gradients of glr_join for a loss with gradients dy and dn with respect
 * to y and n (dy.data NULL: zero; dn given exactly when v is), everything else as the forward
 * call had it. The row's statistics are computed again from x, h and g. With hc (and gc) given,
 * h (and g) are read from their 8-bit checkpoints instead, and h.data (and g.data) are NULL: the
 * gradients are then those at the values kept.
 *   D = dy + rstd_y (q - yhat mean(q yhat) [- mean(q)]),   q = v dn,   yhat = norm(y)
 *   dx = D,   dU = rstd_u (s - uhat mean(s uhat) [- mean(s)]),   s = alpha w D,   uhat = norm(u)
 *   dh = dU act(g),   dg = dU h act'(g)
 *   dw = alpha sum D uhat,   dalpha = sum w D uhat,   dv = sum dn yhat   (sums over the rows)
 * dw, dv [H] and dalpha [1] are float32, summed in a fixed order. h NULL and hc NULL: the norm
 * alone (dx and dv). Outputs that the call does not have are NULL. dx may be dy with the same
 * stride; no other output may share an element with an input. workspace:
 * glr_join_backward_workspace_size(M, H) bytes, 16-byte aligned.
 */
typedef struct {
  int64_t type, M, H, norm, act;
  double eps;
  glr_view dy, dn, x, h, g;
  const uint8_t* hc;
  const uint8_t* hs;
  const uint8_t* gc;
  const uint8_t* gs;
  const float* w;
  const float* alpha;
  const float* v;
  glr_out dx, dh, dg;
  float* dw;
  float* dalpha;
  float* dv;
  void* workspace;
  uint64_t workspace_bytes;
} glr_join_backward_args;
size_t glr_join_backward_workspace_size(int64_t M, int64_t H);
dlr_status glr_join_backward(const glr_join_backward_args* args, dlr_stream_t stream);

/*
 * glr_ckpt_pack / glr_ckpt_unpack -- an activation t [M, H] (rows `stride_t` elements apart) kept
 * in 8 bits. Each row is cut into groups of GLR_CKPT_GROUP channels (the last may be short). A
 * group has the scale 2^s, s the least integer with max|t| <= 448 * 2^s, held within -127 ..
 * 127; scales [M, ceil(H / GLR_CKPT_GROUP)] keeps s + 127 in a byte. codes [M, H] keep t / 2^s in
 * e4m3 (4 exponent and 3 mantissa bits), rounded to nearest even. The maximum runs over the
 * finite values; an infinity or a NaN becomes a NaN code and disturbs no other value. Unpacking
 * gives code * 2^s, rounded to `type` (exact in float32 and bfloat16 for normal values). M >= 0,
 * 1 <= H <= 2^31 - 32, and M * ceil(H / GLR_CKPT_GROUP) <= 2^34 - 8.
 */
#define GLR_CKPT_GROUP 32
dlr_status glr_ckpt_pack(int64_t type, int64_t M, int64_t H, const void* t, int64_t stride_t,
                         uint8_t* codes, uint8_t* scales, dlr_stream_t stream);
dlr_status glr_ckpt_unpack(int64_t type, int64_t M, int64_t H, const uint8_t* codes,
                           const uint8_t* scales, void* t, int64_t stride_t, dlr_stream_t stream);

/* Version of this header's interface (incremented on any signature change or added entry
 * point; dlr_abi_version() counts those of dlr.h). */
int glr_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GLR_H_ */
