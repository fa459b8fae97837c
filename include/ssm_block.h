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
 *     fused with the SiLU gate, and its gradients.
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

#define SSM_BLOCK_ABI_VERSION 1

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

#ifdef __cplusplus
}
#endif

#endif /* SSM_BLOCK_H_ */
