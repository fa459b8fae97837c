/*
 * ssm_block.h -- C ABI of the operators that surround a scan in a block, in the
 * same library (libssm_scan.so) for AMD MI355X (gfx950):
 *
 *   - decay attention: linear attention with a decay for each head (a scan whose
 *     state is a dk x dv matrix per head and whose decay is one number per head
 *     and step), over whole sequences, its gradients, and one token of it;
 *   - residual norm: the RMS norm before a block, fused with the residual sum
 *     and its scale, and its gradients;
 *   - gated norm: the RMS norm after a block's mixing, by groups of channels,
 *     fused with the SiLU gate, and its gradients;
 *   - gated recurrence: a scan whose state is one number per channel, with gates
 *     for its decay and its input, over whole sequences, its gradients, and one
 *     token of it;
 *   - causal convolution: the short depthwise convolution in front of a mixing,
 *     with a state of the last inputs, its gradients, and one token of it;
 *   - head norm and rotation: the RMS norm of every head of queries and keys and
 *     the rotation of its elements by position, in one pass, and its gradients.
 *
 * Conventions are those of ssm_scan.h: io_dtype is SSM_F32 or SSM_BF16,
 * arithmetic and states are fp32, bf16 results are rounded once to nearest
 * even; the caller owns all memory and the library never allocates, frees or
 * synchronises; kernels are enqueued on hip_stream; every argument is checked
 * before anything is enqueued and an error (ssm_status) writes nothing;
 * ssm_last_error() has the message.  Outputs must not overlap inputs unless it
 * is said.  Sums are taken in a fixed order: repeated calls give the same bits.
 */
#ifndef SSM_BLOCK_H_
#define SSM_BLOCK_H_

#include <stdint.h>

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_BLOCK_ABI_VERSION 2

/* SSM_BLOCK_ABI_VERSION of the built library. */
int ssm_block_abi_version(void);

/*
 * A read-only tensor indexed (batch, step, head, element).  Strides are in
 * elements; the elements of one head are adjacent.  A stride may be zero (a
 * broadcast input) but not negative.  ptr and every stride must keep 16-byte
 * alignment (strides multiples of 4 in fp32, of 8 in bf16).
 */
typedef struct ssm_view4 {
  const void *ptr;
  int64_t stride_batch, stride_step, stride_head;
} ssm_view4;

/*
 * Decay attention.  Per batch row and head h, with j = h / (heads / key_heads):
 *
 *   S_t = exp(g_t) S_{t-1} + k_t v_t^T      S is (dk, dv), S_{-1} = state0 or 0
 *   o_t = scale * S_t^T q_t
 *
 *   q, k:      (batch, seqlen, key_heads, dk) views; heads % key_heads == 0
 *   v:         (batch, seqlen, heads, dv) view
 *   log_decay: g, fp32, contiguous: (batch, seqlen, heads) if decay_per_token,
 *              else (heads).  g = -inf (any g below -177, where exp(g) is zero
 *              in fp32 many times over) clears the state: packed documents.
 *              g > 0 grows the state and is not refused; the decays of several
 *              steps together may exceed fp32's range where states, outputs and
 *              gradients do not.
 *   state0:    (batch, heads, dk, dv) fp32 or NULL
 *   state_final: the same shape, NULL = not wanted
 *   o:         (batch, seqlen, heads, dv) contiguous, io_dtype
 *
 * Sizes: batch, seqlen >= 1; 1 <= heads <= 65536; batch * heads <= 2^26; dk, dv
 * multiples of 8 from 8 to 256; heads * dk, heads * dv and step strides <= 2^23.
 * A NaN or an infinity at one step reaches no earlier step.  fp32 values and
 * states of 3.396e38 and more, half a step of bf16 below 2^128, count as infinite.
 */
int64_t ssm_decay_attn_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads,
                                           int64_t key_heads, int64_t dk, int64_t dv, int io_dtype);

int ssm_decay_attn_fwd(int64_t batch, int64_t seqlen, int64_t heads, int64_t key_heads, int64_t dk,
                       int64_t dv, int io_dtype, const ssm_view4 *q, const ssm_view4 *k,
                       const ssm_view4 *v, const float *log_decay, int decay_per_token, float scale,
                       const float *state0, float *state_final, void *o, void *workspace,
                       int64_t workspace_bytes, void *hip_stream);

/*
 * Its gradients.  dout is dLoss/do (a view of v's shape), dstate_final
 * dLoss/dS_last (optional, NULL = 0).  With R_t = exp(g_{t+1}) R_{t+1} + scale q_t dout_t^T
 * (R beyond the end: dstate_final):
 *
 *   dq_t = scale S_t dout_t   dk_t = R_t v_t   dv_t = R_t^T k_t
 *   dg_t = exp(g_t) <S_{t-1}, R_t>   dstate0 = exp(g_0) R_0
 *
 *   dq, dk: (batch, seqlen, key_heads, dk) contiguous, io_dtype, summed over
 *           the heads that share a key head; dv: (batch, seqlen, heads, dv)
 *   dlog_decay: log_decay's shape, fp32, NULL = not wanted (0 where the state
 *           is cleared); dstate0: (batch, heads, dk, dv) fp32, NULL = not wanted
 *
 * The workspace is the same for every call of a shape: what dlog_decay of decays
 * by head needs, whether it is wanted or not.  With and without dlog_decay, dq and
 * dk are summed in another order: equal to fp32's rounding, not to the bit.
 */
int64_t ssm_decay_attn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads,
                                           int64_t key_heads, int64_t dk, int64_t dv, int io_dtype);

int ssm_decay_attn_bwd(int64_t batch, int64_t seqlen, int64_t heads, int64_t key_heads, int64_t dk,
                       int64_t dv, int io_dtype, const ssm_view4 *q, const ssm_view4 *k,
                       const ssm_view4 *v, const float *log_decay, int decay_per_token, float scale,
                       const float *state0, const ssm_view4 *dout, const float *dstate_final,
                       void *dq, void *dk_out, void *dv_out, float *dlog_decay, float *dstate0,
                       void *workspace, int64_t workspace_bytes, void *hip_stream);

/*
 * One token: state (batch, heads, dk, dv) fp32 is updated in place and read
 * once; q, k (batch, key_heads, dk) and v (batch, heads, dv) are views whose
 * stride_step is not used; log_decay is (batch, heads) if decay_per_token,
 * else (heads); o is (batch, heads, dv) contiguous, io_dtype.
 */
int ssm_decay_attn_update(int64_t batch, int64_t heads, int64_t key_heads, int64_t dk, int64_t dv,
                          int io_dtype, float *state, const ssm_view4 *q, const ssm_view4 *k,
                          const ssm_view4 *v, const float *log_decay, int decay_per_token,
                          float scale, void *o, void *hip_stream);

/*
 * Residual norm, row by row over dim channels:
 *   h = residual + scale * x,  rstd = (mean h^2 + eps)^-1/2,  y = h * rstd * weight
 * x, y in io_dtype with rows row_stride elements apart for x (y contiguous);
 * residual, h (rows, dim) contiguous in residual_dtype (SSM_F32, or SSM_BF16
 * if io_dtype is); weight (dim) fp32; scale (dim) fp32, NULL = 1; rstd (rows)
 * fp32, NULL = not wanted.  y is formed from h before h is rounded.  h may be
 * residual's memory.  dim: a multiple of 8 from 8 to 16384.
 */
int ssm_residual_norm_fwd(int64_t rows, int64_t dim, int io_dtype, int residual_dtype, const void *x,
                          int64_t x_row_stride, const void *residual, const float *weight,
                          const float *scale, float eps, void *y, void *h, float *rstd,
                          void *hip_stream);

/*
 * Its gradients, given dy (io_dtype) and dh (residual_dtype, NULL = 0), the
 * gradient that reaches h by the residual stream; all (rows, dim) contiguous.
 *   dresidual = dh + norm's gradient (residual_dtype);  dx = scale * dresidual
 *   (io_dtype; NULL = not wanted, as where it equals dresidual);
 *   dweight (dim) fp32;  dscale (dim) fp32, NULL = not wanted, needs x.
 */
int64_t ssm_residual_norm_bwd_workspace_bytes(int64_t rows, int64_t dim);

int ssm_residual_norm_bwd(int64_t rows, int64_t dim, int io_dtype, int residual_dtype,
                          const void *dy, const void *dh, const void *h, const float *rstd,
                          const float *weight, const void *x, int64_t x_row_stride,
                          const float *scale, void *dx, void *dresidual, float *dweight,
                          float *dscale, void *workspace, int64_t workspace_bytes, void *hip_stream);

/*
 * Gated norm, over groups of `group` adjacent channels (dim % group == 0):
 *   gate_first = 0: y = x * rstd * weight * silu(z),  rstd = (mean x^2 + eps)^-1/2
 *   gate_first = 1: t = x * silu(z),  y = t * rstd * weight,  rstd = (mean t^2 + eps)^-1/2
 * z NULL = no gate (silu(z) = 1).  x, z: rows row_stride elements apart,
 * io_dtype; y (rows, dim) contiguous; weight (dim) fp32; rstd (rows, dim /
 * group) fp32, NULL = not wanted.  group: a multiple of 8 from 8 to 16384.
 */
int ssm_gated_norm_fwd(int64_t rows, int64_t dim, int64_t group, int io_dtype, const void *x,
                       int64_t x_row_stride, const void *z, int64_t z_row_stride,
                       const float *weight, float eps, int gate_first, void *y, float *rstd,
                       void *hip_stream);

/* Its gradients: dy, dx, dz (rows, dim) contiguous in io_dtype; dz is required
 * iff z is given; dweight (dim) fp32. */
int64_t ssm_gated_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, int64_t group);

int ssm_gated_norm_bwd(int64_t rows, int64_t dim, int64_t group, int io_dtype, const void *dy,
                       const void *x, int64_t x_row_stride, const void *z, int64_t z_row_stride,
                       const float *weight, const float *rstd, int gate_first, void *dx, void *dz,
                       float *dweight, void *workspace, int64_t workspace_bytes, void *hip_stream);

/*
 * A read-only tensor indexed (batch, step, channel).  Strides are in elements;
 * channels are adjacent.  A stride may be zero (a broadcast input) but not
 * negative; a step's is at most 2^23.  ptr and every stride must keep 16-byte
 * alignment.  For one token stride_step is not used.
 */
typedef struct ssm_view3 {
  const void *ptr;
  int64_t stride_batch, stride_step;
} ssm_view3;

/*
 * Gated recurrence.  Per batch row and channel:
 *
 *   h_t = a_t h_{t-1} + s_t sigmoid(input_gate_t) x_t     h_{-1} = state0 or 0
 *   y_t = h_t (silu(z_t))
 *
 *   decay given:  a = exp(-sharpness softplus(decay) sigmoid(decay_gate_t)),  s = sqrt(1 - a^2)
 *   decay NULL:   a = sigmoid(decay_gate_t),                                  s = 1 - a
 *
 *   x, decay_gate, input_gate, z: (batch, seqlen, dim) views in io_dtype;
 *              input_gate NULL = 1, z NULL = no gate
 *   decay:     (dim) fp32; sharpness > 0 and finite (not used without decay)
 *   state0:    (batch, dim) fp32 or NULL
 *   starts:    (batch, seqlen) bytes, NULL = none: where not zero, a document
 *              starts: a = 0 and s = 1 in both forms, whatever the gate holds.
 *              Nothing crosses it, infinities and NaN included, in either
 *              direction.  A first step without a mark has the gate's s, so a
 *              document gives the same in a packed row and in one of its own if
 *              its first step is marked in both
 *   lengths:   (batch), NULL = seqlen: the rows' lengths in a padded batch
 *              (taken as 0 below 0 and as seqlen above).  Inputs behind a row's
 *              length are not used, y is zero there, and the state stays that
 *              of the row's last token.
 *   y:         (batch, seqlen, dim) contiguous, io_dtype
 *   state_final: (batch, dim) fp32, NULL = not wanted
 *   states:    (batch, ceil(seqlen / SSM_RECURRENCE_CHUNK), dim) fp32, NULL = not
 *              wanted: the state before every chunk, which the backward needs
 *
 * dim: a multiple of 8 up to 2^23; batch <= 2^16; batch * ceil(dim / 64) *
 * ceil(seqlen / 128) <= 2^22.
 */
#define SSM_RECURRENCE_CHUNK 128

int64_t ssm_gated_recurrence_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype);

int ssm_gated_recurrence_fwd(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype, const ssm_view3 *x,
                             const ssm_view3 *decay_gate, const ssm_view3 *input_gate, const ssm_view3 *z,
                             const float *decay, float sharpness, const float *state0,
                             const uint8_t *starts, const int32_t *lengths, void *y,
                             float *state_final, float *states, void *workspace,
                             int64_t workspace_bytes, void *hip_stream);

/*
 * Its gradients, given dy (a view) and dstate_final (optional, NULL = 0).  With
 * e_t = dy_t (silu(z_t)) and w_t = e_t + a_{t+1} w_{t+1} (beyond the end: dstate_final):
 *
 *   dx_t = w_t s_t sigmoid(input_gate_t)     ddecay_gate_t = w_t (h_{t-1} da + sigmoid(input_gate_t) x_t ds)
 *   dinput_gate_t = w_t s_t x_t sigmoid'(input_gate_t)      dz_t = dy_t h_t silu'(z_t)
 *
 * dx, ddecay_gate, dinput_gate, dz (batch, seqlen, dim) contiguous, io_dtype,
 * zero behind a row's length; dinput_gate and dz are required iff their inputs
 * are given; ddecay (dim) fp32, required iff decay is given; dstate0 (batch, dim)
 * fp32, NULL = not wanted.  states: as the forward wrote them (state0 is their first).
 */
int64_t ssm_gated_recurrence_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype);

int ssm_gated_recurrence_bwd(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype, const ssm_view3 *dy,
                             const ssm_view3 *x, const ssm_view3 *decay_gate,
                             const ssm_view3 *input_gate, const ssm_view3 *z, const float *decay,
                             float sharpness, const float *states, const uint8_t *starts,
                             const int32_t *lengths, const float *dstate_final, void *dx,
                             void *ddecay_gate, void *dinput_gate, void *dz, float *ddecay,
                             float *dstate0, void *workspace, int64_t workspace_bytes,
                             void *hip_stream);

/*
 * One token: state (batch, dim) fp32 is updated in place; y (batch, dim)
 * contiguous, io_dtype.  batch * dim <= 2^32.  It has no mark: the first token of
 * a document is a sequence of one marked step.
 */
int ssm_gated_recurrence_update(int64_t batch, int64_t dim, int io_dtype, float *state, const ssm_view3 *x,
                                const ssm_view3 *decay_gate, const ssm_view3 *input_gate,
                                const ssm_view3 *z, const float *decay, float sharpness, void *y,
                                void *hip_stream);

/*
 * Causal depthwise convolution, per batch row and channel:
 *
 *   y_t = act(bias + sum_k weight[k] x_{t - (width - 1) + k}),  act = silu or (silu = 0) the identity
 *
 *   x:       (batch, seqlen, dim) view in io_dtype; y contiguous
 *   weight:  (dim, width) fp32, width 1 to 4; bias (dim) fp32 or NULL
 *   state0:  (batch, width - 1, dim) in io_dtype, the inputs before the first,
 *            oldest first; NULL = 0 (and must be NULL if width is 1)
 *   starts, lengths: as of the gated recurrence; taps that reach before the
 *            document of their step are zero, and so is y behind a row's length
 *   state_final: as state0: the last width - 1 inputs of each row, zero where
 *            they are not of the row's last document; NULL = not wanted
 *
 * dim: a multiple of 8 up to 2^23; batch <= 2^16; seqlen <= 2^30; batch * dim / 8 *
 * (ceil(seqlen / 32) + 1) <= 2^30 (and for one token the same with seqlen 1).
 */
int ssm_causal_conv_fwd(int64_t batch, int64_t seqlen, int64_t dim, int width, int io_dtype,
                        const ssm_view3 *x, const float *weight, const float *bias, const void *state0,
                        const uint8_t *starts, const int32_t *lengths, int silu, void *y,
                        void *state_final, void *hip_stream);

/*
 * Its gradients, given dy (a view) and dstate_final (as state_final, optional,
 * NULL = 0): dx (batch, seqlen, dim) contiguous, io_dtype; dweight (dim, width)
 * and dbias (dim) fp32, dbias NULL = not wanted; dstate0 as state0, NULL = not wanted.
 */
int64_t ssm_causal_conv_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int width);

int ssm_causal_conv_bwd(int64_t batch, int64_t seqlen, int64_t dim, int width, int io_dtype,
                        const ssm_view3 *dy, const ssm_view3 *x, const float *weight, const float *bias,
                        const void *state0, const uint8_t *starts, const int32_t *lengths, int silu,
                        const void *dstate_final, void *dx, float *dweight, float *dbias, void *dstate0,
                        void *workspace, int64_t workspace_bytes, void *hip_stream);

/* One token: state (batch, width - 1, dim) in io_dtype moves on by one input, in
 * place (NULL if width is 1); y (batch, dim) contiguous. */
int ssm_causal_conv_update(int64_t batch, int64_t dim, int width, int io_dtype, void *state,
                           const ssm_view3 *x, const float *weight, const float *bias, int silu, void *y,
                           void *hip_stream);

/*
 * Norm and rotation of heads.  For every head of q (q_heads of them) and k:
 *
 *   n = x rstd weight,  rstd = (mean x^2 + eps)^-1/2   (norm = 0: n = x)
 *   (n_i, n_j) <- (n_i cos - n_j sin, n_j cos + n_i sin),  angle = position * inv_freq[p]
 *
 *   pair p < rotary / 2 is (i, j) = (p, p + rotary / 2), or with interleaved
 *   (2p, 2p + 1); elements from rotary on are not rotated
 *   q, k:      (batch, seqlen, heads, dim) views in io_dtype; k NULL = none (k_heads = 0)
 *   q_weight, k_weight: fp32, (heads, dim) if weight_per_head, else (dim);
 *              NULL = 1 (both or neither; NULL if norm = 0)
 *   positions: (batch, seqlen), or with positions_per_batch = 0 (seqlen), int64,
 *              NULL = no rotation (rotary = 0)
 *   inv_freq:  (rotary / 2) fp64, radians per position; the angle is formed in
 *              fp64, so that far positions keep their digits
 *   q_out, k_out: contiguous, io_dtype
 *
 * dim: a multiple of 8 from 8 to 256; rotary: a multiple of 8 up to dim; heads
 * in all <= 65536; batch * seqlen * heads in all * dim <= 2^40.
 */
int ssm_head_norm_rotary_fwd(int64_t batch, int64_t seqlen, int64_t q_heads, int64_t k_heads, int64_t dim,
                             int64_t rotary, int io_dtype, const ssm_view4 *q, const ssm_view4 *k,
                             const float *q_weight, const float *k_weight, int weight_per_head,
                             const int64_t *positions, int positions_per_batch, const double *inv_freq,
                             float eps, int norm, int interleaved, void *q_out, void *k_out,
                             void *hip_stream);

/*
 * Its gradients, given dq_out and dk_out (views): dq, dk contiguous, io_dtype;
 * dq_weight, dk_weight as the weights, fp32, required iff those are given.
 */
int64_t ssm_head_norm_rotary_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t q_heads,
                                                 int64_t k_heads, int64_t dim);

int ssm_head_norm_rotary_bwd(int64_t batch, int64_t seqlen, int64_t q_heads, int64_t k_heads, int64_t dim,
                             int64_t rotary, int io_dtype, const ssm_view4 *dq_out,
                             const ssm_view4 *dk_out, const ssm_view4 *q, const ssm_view4 *k,
                             const float *q_weight, const float *k_weight, int weight_per_head,
                             const int64_t *positions, int positions_per_batch, const double *inv_freq,
                             float eps, int norm, int interleaved, void *dq, void *dk, float *dq_weight,
                             float *dk_weight, void *workspace, int64_t workspace_bytes,
                             void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_BLOCK_H_ */
