/*
 * ssm.h -- C ABI of libdlr.so, third header: the operators of a selective state space block on one
 * NVIDIA GB300 GPU (sm_103a).
 *   - the short causal convolution before the scan: over a sequence, its gradients, one token;
 *   - the selective scan, the bank of diagonal recurrences of dlr.h with real states whose step,
 *     input map and output map the token chooses: over a sequence, its gradients, one token.
 *
 * Status codes, streams, workspaces and the device status word are those of dlr.h; activations,
 * types and views (glr_view, glr_out, contiguous channels and strides in elements) are those of
 * glr.h, with its rules: an input's strides may be 0, negative ones are refused, an output's
 * elements must be distinct, and no output may share an element with an input or another output
 * unless a call says so. Arguments come in one struct per call (all fields 8 bytes wide; unused
 * pointers NULL). Parameters, scan states and their gradients are float32 and contiguous. All
 * arithmetic is float32 (what ssm_scan_backward sums over channels for dBm and dCm is cut to 21 bits
 * first); results are rounded once, to nearest even, where they are stored in 16 bits. Sums over rows
 * and channels run in a fixed order: results repeat bit for bit.
 *
 * A decay exp(s A) of float32 activations keeps its digits down to 2^-126 (below it is 0): next to 1 it
 * is 1 - a that is rounded. That of 16-bit activations is one number, off by up to 1.5 * 2^-24 of
 * itself: over a memory of 8192 steps a state, and h_last with it, may be 7.4e-4 off.
 *
 * reset: bytes [B, L], contiguous, NULL for none; a step that it marks begins a new sequence:
 * nothing before it, not even an infinity or a NaN, reaches it.
 */
#ifndef SSM_H_
#define SSM_H_

#include "glr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activation of the convolution: p sigmoid(p), or p. */
typedef enum { SSM_ACT_SILU = 0, SSM_ACT_NONE = 1 } ssm_act;

#define SSM_MAX_TAPS 8     /* of the convolution */
#define SSM_MAX_STATES 64  /* of a channel of the scan */

/* Steps between the states that ssm_scan keeps for its gradients. */
#define SSM_STATE_STEPS 16

/*
 * ssm_conv -- per channel of x [B, L, H], with the taps w [H, K] and the bias (float32 [H], NULL:
 * zero):
 *   p_t = bias + sum_{j < K} w_j x_{t-(K-1)+j},   y_t = act(p_t)
 * x_{-(K-1)} .. x_{-1} are the rows of `state` [B, K-1, H] (activations, contiguous; NULL: zero).
 * Inputs before a step that reset marks count as zero from that step on. last [B, K-1, H]
 * (activations, contiguous, may be NULL): what the next step would see as its K-1 inputs before
 * it, a `state` for the sequence's continuation. 1 <= K <= SSM_MAX_TAPS; with K = 1 state and last
 * are NULL. L = 0 copies state (or zero) to last.
 */
typedef struct {
  int64_t type, B, L, H, K, act;
  glr_view x;
  const float* w;
  const float* bias;
  const void* state;
  const uint8_t* reset;
  glr_out y;
  void* last;
} ssm_conv_args;
dlr_status ssm_conv(const ssm_conv_args* args, dlr_stream_t stream);

/*
 * ssm_conv_backward -- the gradients of ssm_conv for a loss with gradients dy with respect to y
 * and, when dlast (activations [B, K-1, H]) is not NULL, dlast with respect to last; everything
 * else as the forward call had it. With g = dy act'(p):
 *   dx_t = sum_j w_j g_{t+(K-1)-j} (+ dlast),  dw_j = sum g_t x_{t-(K-1)+j},  dbias = sum g
 * over the steps that see the input. dw [H, K], dbias [H] (NULL: not wanted) float32; dstate
 * (activations [B, K-1, H], NULL: not wanted). workspace:
 * ssm_conv_backward_workspace_size(B, L, H, K) bytes, 16-byte aligned.
 */
typedef struct {
  int64_t type, B, L, H, K, act;
  glr_view x, dy;
  const float* w;
  const float* bias;
  const void* state;
  const uint8_t* reset;
  const void* dlast;
  glr_out dx;
  float* dw;
  float* dbias;
  void* dstate;
  void* workspace;
  uint64_t workspace_bytes;
} ssm_conv_backward_args;
size_t ssm_conv_backward_workspace_size(int64_t B, int64_t L, int64_t H, int64_t K);
dlr_status ssm_conv_backward(const ssm_conv_backward_args* args, dlr_stream_t stream);

/*
 * ssm_conv_step -- ssm_conv for one token (L = 1; stride_t unused): y [B, H] and state_out
 * [B, K-1, H] from state [B, K-1, H] (both needed when K > 1; state_out may be state). reset:
 * bytes [B] or NULL. One launch.
 */
typedef struct {
  int64_t type, B, H, K, act;
  glr_view x;
  const float* w;
  const float* bias;
  const void* state;
  const uint8_t* reset;
  glr_out y;
  void* state_out;
} ssm_conv_step_args;
dlr_status ssm_conv_step(const ssm_conv_step_args* args, dlr_stream_t stream);

/*
 * ssm_scan -- the selective scan over x and dt [B, L, H] with the rates A [H, N], the maps Bm and
 * Cm [B, L, G N] (views whose G N channels are contiguous; channel h of x uses the N of group
 * h / (H / G)), the skip D [H] (NULL: none), the gate z [B, L, H] (data NULL: none) and dt_bias [H]
 * (NULL: zero):
 *   s_t = softplus(dt_t + dt_bias) (softplus = 0: dt_t + dt_bias)
 *   h_t = exp(s_t A) h_{t-1} + s_t x_t Bm_t           N states of each channel, h_{-1} = h0
 *   o_t = sum_n Cm_t h_t + D x_t,   y_t = o_t z_t sigmoid(z_t) (o_t without a gate)
 * h0, h_last: float32 [B, H, N] (either may be NULL). A marked step has no h_{t-1}; its input keeps
 * the factor s_t. A step whose dt is -inf leaves the state as it is (with softplus, for finite x).
 * states (NULL: not kept): float32 [B, ssm_states(L), H, N], the state before each run of
 * SSM_STATE_STEPS steps, for ssm_scan_backward. workspace:
 * ssm_scan_workspace_size(B, L, H, N, G) bytes, 16-byte aligned (0: none needed). L = 0 copies h0 (or zero) to h_last.
 * G >= 1 divides H; 1 <= N <= SSM_MAX_STATES; B and L < 2^31, H < 2^24.
 */
typedef struct {
  int64_t type, B, L, H, N, G, softplus;
  glr_view x, dt, z, Bm, Cm;
  const float* A;
  const float* D;
  const float* dt_bias;
  const float* h0;
  const uint8_t* reset;
  glr_out y;
  float* h_last;
  float* states;
  void* workspace;
  uint64_t workspace_bytes;
} ssm_scan_args;
int64_t ssm_states(int64_t L);
size_t ssm_scan_workspace_size(int64_t B, int64_t L, int64_t H, int64_t N, int64_t G);
dlr_status ssm_scan(const ssm_scan_args* args, dlr_stream_t stream);

/*
 * ssm_scan_backward -- the gradients of ssm_scan for a loss with gradients dy with respect to y and,
 * when dh_last (float32 [B, H, N]) is not NULL, dh_last with respect to h_last; everything else as
 * the forward call had it, states as it left them. With a = exp(s A), g = dy silu(z):
 *   G_t = g_t Cm_t + a_{t+1} G_{t+1}   (G_{L-1} = g Cm + dh_last; nothing passes a marked step)
 *   q = sum_n G Bm,   e = sum_n A G a h_{t-1}
 *   dx = s q + D g,   ddt = (x q + e) sigmoid(dt + dt_bias)  (softplus = 0: x q + e)
 *   dz = dy o silu'(z),   dBm = sum_h G s x,   dCm = sum_h g h_t   (over a group's channels)
 *   dA = sum s G a h_{t-1},   dD = sum g x,   ddt_bias = sum ddt,   dh0 = a_0 G_0
 * Where an input is not finite and no step near it is marked, the dBm and dCm of the steps of its run
 * of four may be NaN too. dBm, dCm: views [B, L, G N]. dA [H, N], dD, ddt_bias [H] and dh0 [B, H, N] are float32; dD is
 * given exactly when D is, dz when z is; ddt_bias and dh0 may be NULL. The states between the kept
 * ones are computed again. workspace: ssm_scan_backward_workspace_size(B, L, H, N, G) bytes,
 * 16-byte aligned. L = 0 writes zero to the parameters' gradients and dh_last (or 0) to dh0.
 */
typedef struct {
  int64_t type, B, L, H, N, G, softplus;
  glr_view x, dt, z, Bm, Cm, dy;
  const float* A;
  const float* D;
  const float* dt_bias;
  const float* h0;
  const uint8_t* reset;
  const float* states;
  const float* dh_last;
  glr_out dx, ddt, dz, dBm, dCm;
  float* dA;
  float* dD;
  float* ddt_bias;
  float* dh0;
  void* workspace;
  uint64_t workspace_bytes;
} ssm_scan_backward_args;
size_t ssm_scan_backward_workspace_size(int64_t B, int64_t L, int64_t H, int64_t N, int64_t G);
dlr_status ssm_scan_backward(const ssm_scan_backward_args* args, dlr_stream_t stream);

/*
 * ssm_step -- ssm_scan for one token (L = 1; stride_t unused): y [B, H] and the state h_out from the
 * state h (float32 [B, H, N] both; h_out may be h). reset: bytes [B] or NULL. One launch.
 */
typedef struct {
  int64_t type, B, H, N, G, softplus;
  glr_view x, dt, z, Bm, Cm;
  const float* A;
  const float* D;
  const float* dt_bias;
  const float* h;
  const uint8_t* reset;
  glr_out y;
  float* h_out;
} ssm_step_args;
dlr_status ssm_step(const ssm_step_args* args, dlr_stream_t stream);

/* Version of this header's interface (incremented on any signature change or added entry point). */
int ssm_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SSM_H_ */
