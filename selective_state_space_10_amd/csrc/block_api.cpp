// block_api.cpp -- the extern "C" entry points declared in include/ssm_block.h:
// argument validation (before anything is enqueued), size queries and dispatch
// to the HIP launchers.  No device code lives here.
#include <stdarg.h>
#include <stdio.h>

#include "api_checks.hpp"
#include "block_kernels.hpp"

using ssm::api_fail;
using ssm::api_hip_status;
using ssm::check_dtype;
using ssm::check_workspace;
using ssm::kMaxElems;
using ssm::kMaxStep;
using ssm::product_ok;
using ssm::Ptr;

namespace {

constexpr int64_t kMaxBatchHeads = (int64_t)1 << 26; // workgroups of one launch stay below 2^31
constexpr int64_t kMaxRow = 16384;

int check_attn(int64_t batch, int64_t seqlen, int64_t heads, int64_t key_heads, int64_t dk, int64_t dv, int io_dtype) {
  if (batch < 1 || seqlen < 1 || heads < 1 || key_heads < 1 || dk < 1 || dv < 1)
    return api_fail(SSM_ERR_BAD_SHAPE, "sizes must be >= 1 (batch=%lld seqlen=%lld heads=%lld key_heads=%lld dk=%lld dv=%lld)",
                    (long long)batch, (long long)seqlen, (long long)heads, (long long)key_heads, (long long)dk, (long long)dv);
  if (heads % key_heads != 0)
    return api_fail(SSM_ERR_BAD_SHAPE, "heads=%lld is not a multiple of key_heads=%lld", (long long)heads, (long long)key_heads);
  if (dk % 8 != 0 || dk > 256 || dv % 8 != 0 || dv > 256)
    return api_fail(SSM_ERR_UNSUPPORTED, "dk=%lld and dv=%lld must be multiples of 8 up to 256", (long long)dk, (long long)dv);
  if (heads > 65536) return api_fail(SSM_ERR_UNSUPPORTED, "heads=%lld exceeds 65536", (long long)heads);
  if (batch > kMaxBatchHeads / heads)
    return api_fail(SSM_ERR_UNSUPPORTED, "batch * heads exceeds 2^26 (batch=%lld heads=%lld)", (long long)batch, (long long)heads);
  if (heads * (dk > dv ? dk : dv) > kMaxStep)  // offsets inside a chunk of 64 steps are 32-bit bytes
    return api_fail(SSM_ERR_UNSUPPORTED, "heads * max(dk, dv) exceeds 2^23");
  int64_t n;
  if (!product_ok(batch * heads, seqlen, &n) || !product_ok(n, dk > dv ? dk : dv, &n))
    return api_fail(SSM_ERR_BAD_SHAPE, "tensors of more than 2^40 elements");
  return check_dtype(io_dtype);
}

// one_step: stride_step is not used
int check_view(const char *name, const ssm_view4 *v, int io_dtype, bool one_step = false) {
  SSM_TRY(ssm::check_view_ptr(name, v, v ? v->ptr : nullptr));
  const int64_t step = one_step ? 0 : v->stride_step;
  const int64_t st[] = {v->stride_batch, step, v->stride_head};
  for (int64_t s : st) SSM_TRY(ssm::check_stride(name, s, io_dtype));
  if (step > kMaxStep) return api_fail(SSM_ERR_UNSUPPORTED, "%s has a step stride over 2^23 elements", name);
  return SSM_OK;
}

ssm::View4 view(const ssm_view4 *v, int64_t share) {
  return {v->ptr, v->stride_batch, v->stride_step, v->stride_head, (int)share};
}

ssm::DecayAttnArgs attn_args(int64_t batch, int64_t seqlen, int64_t heads, int64_t key_heads, int64_t dk, int64_t dv) {
  ssm::DecayAttnArgs a{};
  a.B = batch, a.L = seqlen, a.H = heads, a.G = key_heads, a.dk = dk, a.dv = dv;
  return a;
}

int check_row(int64_t rows, int64_t dim, int64_t len, const char *what) {
  if (rows < 1 || dim < 1 || len < 1)
    return api_fail(SSM_ERR_BAD_SHAPE, "sizes must be >= 1 (rows=%lld dim=%lld %s=%lld)", (long long)rows, (long long)dim, what, (long long)len);
  if (len % 8 != 0 || len > kMaxRow)
    return api_fail(SSM_ERR_UNSUPPORTED, "%s=%lld must be a multiple of 8 up to %lld", what, (long long)len, (long long)kMaxRow);
  if (dim % len != 0) return api_fail(SSM_ERR_BAD_SHAPE, "dim=%lld is not a multiple of %s=%lld", (long long)dim, what, (long long)len);
  if (dim > ((int64_t)1 << 24)) return api_fail(SSM_ERR_UNSUPPORTED, "dim=%lld exceeds 2^24", (long long)dim);
  int64_t n;
  if (!product_ok(rows, dim, &n)) return api_fail(SSM_ERR_BAD_SHAPE, "tensors of more than 2^40 elements");
  return SSM_OK;
}

int check_row_stride(const char *name, int64_t stride, int64_t dim, int64_t rows, int io_dtype) {
  if (stride < 0 || (rows > 1 && stride > kMaxElems))
    return api_fail(SSM_ERR_BAD_SHAPE, "%s has row stride %lld", name, (long long)stride);
  if (stride * (io_dtype == SSM_F32 ? 4 : 2) % 16 != 0)
    return api_fail(SSM_ERR_ALIGNMENT, "%s has row stride %lld, not a multiple of 16 bytes", name, (long long)stride);
  (void)dim;
  return SSM_OK;
}

int check_residual_dtype(int io_dtype, int residual_dtype) {
  const int st = check_dtype(io_dtype);
  if (st != SSM_OK) return st;
  if (residual_dtype != SSM_F32 && residual_dtype != io_dtype)
    return api_fail(SSM_ERR_UNSUPPORTED, "residual_dtype=%d with io_dtype=%d", residual_dtype, io_dtype);
  return SSM_OK;
}

}  // namespace

extern "C" {

int ssm_block_abi_version(void) { return SSM_BLOCK_ABI_VERSION; }

int64_t ssm_decay_attn_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads, int64_t key_heads, int64_t dk,
                                           int64_t dv, int io_dtype) {
  if (check_attn(batch, seqlen, heads, key_heads, dk, dv, io_dtype) != SSM_OK) return -1;
  return ssm::decay_attn_fwd_workspace_bytes(attn_args(batch, seqlen, heads, key_heads, dk, dv), io_dtype);
}

int ssm_decay_attn_fwd(int64_t batch, int64_t seqlen, int64_t heads, int64_t key_heads, int64_t dk, int64_t dv,
                       int io_dtype, const ssm_view4 *q, const ssm_view4 *k, const ssm_view4 *v,
                       const float *log_decay, int decay_per_token, float scale, const float *state0,
                       float *state_final, void *o, void *workspace, int64_t workspace_bytes, void *hip_stream) {
  ssm::api_clear_error();
  SSM_TRY(check_attn(batch, seqlen, heads, key_heads, dk, dv, io_dtype));
  SSM_TRY(check_view("q", q, io_dtype));
  SSM_TRY(check_view("k", k, io_dtype));
  SSM_TRY(check_view("v", v, io_dtype));
  const Ptr ps[] = {{"log_decay", log_decay, true, 4}, {"state0", state0, false, 16}, {"state_final", state_final, false, 16}, {"o", o, true, 16}};
  SSM_TRY_PTRS(ps);
  ssm::DecayAttnArgs a = attn_args(batch, seqlen, heads, key_heads, dk, dv);
  SSM_TRY(check_workspace(workspace, workspace_bytes, ssm::decay_attn_fwd_workspace_bytes(a, io_dtype)));
  const int64_t share = heads / key_heads;
  a.q = view(q, share), a.k = view(k, share), a.v = view(v, 1);
  a.g = log_decay, a.g_b = decay_per_token ? seqlen * heads : 0, a.g_t = decay_per_token ? heads : 0;
  a.scale = scale, a.state0 = state0, a.state_final = state_final, a.o = o, a.workspace = workspace;
  return api_hip_status(ssm::launch_decay_attn_fwd(a, io_dtype, (hipStream_t)hip_stream), "ssm_decay_attn_fwd launch");
}

int64_t ssm_decay_attn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads, int64_t key_heads, int64_t dk,
                                           int64_t dv, int io_dtype) {
  if (check_attn(batch, seqlen, heads, key_heads, dk, dv, io_dtype) != SSM_OK) return -1;
  return ssm::decay_attn_bwd_workspace_bytes(attn_args(batch, seqlen, heads, key_heads, dk, dv), io_dtype);
}

int ssm_decay_attn_bwd(int64_t batch, int64_t seqlen, int64_t heads, int64_t key_heads, int64_t dk, int64_t dv,
                       int io_dtype, const ssm_view4 *q, const ssm_view4 *k, const ssm_view4 *v,
                       const float *log_decay, int decay_per_token, float scale, const float *state0,
                       const ssm_view4 *dout, const float *dstate_final, void *dq, void *dk_out, void *dv_out,
                       float *dlog_decay, float *dstate0, void *workspace, int64_t workspace_bytes, void *hip_stream) {
  ssm::api_clear_error();
  SSM_TRY(check_attn(batch, seqlen, heads, key_heads, dk, dv, io_dtype));
  SSM_TRY(check_view("q", q, io_dtype));
  SSM_TRY(check_view("k", k, io_dtype));
  SSM_TRY(check_view("v", v, io_dtype));
  SSM_TRY(check_view("dout", dout, io_dtype));
  const Ptr ps[] = {{"log_decay", log_decay, true, 4}, {"state0", state0, false, 16},       {"dstate_final", dstate_final, false, 16},
                    {"dq", dq, true, 16},              {"dk_out", dk_out, true, 16},        {"dv_out", dv_out, true, 16},
                    {"dlog_decay", dlog_decay, false, 4}, {"dstate0", dstate0, false, 16}};
  SSM_TRY_PTRS(ps);
  ssm::DecayAttnArgs a = attn_args(batch, seqlen, heads, key_heads, dk, dv);
  SSM_TRY(check_workspace(workspace, workspace_bytes, ssm::decay_attn_bwd_workspace_bytes(a, io_dtype)));
  const int64_t share = heads / key_heads;
  a.q = view(q, share), a.k = view(k, share), a.v = view(v, 1), a.dout = view(dout, 1);
  a.g = log_decay, a.g_b = decay_per_token ? seqlen * heads : 0, a.g_t = decay_per_token ? heads : 0;
  a.scale = scale, a.state0 = state0, a.dstate_final = dstate_final;
  a.dq = dq, a.dk_out = dk_out, a.dv_out = dv_out, a.dlog_decay = dlog_decay, a.dstate0 = dstate0, a.workspace = workspace;
  return api_hip_status(ssm::launch_decay_attn_bwd(a, io_dtype, (hipStream_t)hip_stream), "ssm_decay_attn_bwd launch");
}

int ssm_decay_attn_update(int64_t batch, int64_t heads, int64_t key_heads, int64_t dk, int64_t dv, int io_dtype,
                          float *state, const ssm_view4 *q, const ssm_view4 *k, const ssm_view4 *v,
                          const float *log_decay, int decay_per_token, float scale, void *o, void *hip_stream) {
  ssm::api_clear_error();
  SSM_TRY(check_attn(batch, 1, heads, key_heads, dk, dv, io_dtype));
  SSM_TRY(check_view("q", q, io_dtype, true));
  SSM_TRY(check_view("k", k, io_dtype, true));
  SSM_TRY(check_view("v", v, io_dtype, true));
  const Ptr ps[] = {{"state", state, true, 16}, {"log_decay", log_decay, true, 4}, {"o", o, true, 16}};
  SSM_TRY_PTRS(ps);
  ssm::DecayUpdateArgs a{};
  const int64_t share = heads / key_heads;
  a.B = batch, a.H = heads, a.G = key_heads, a.dk = dk, a.dv = dv, a.state = state;
  a.q = view(q, share), a.k = view(k, share), a.v = view(v, 1);
  a.g = log_decay, a.g_b = decay_per_token ? heads : 0, a.scale = scale, a.o = o;
  return api_hip_status(ssm::launch_decay_update(a, io_dtype, (hipStream_t)hip_stream), "ssm_decay_attn_update launch");
}

int ssm_residual_norm_fwd(int64_t rows, int64_t dim, int io_dtype, int residual_dtype, const void *x,
                          int64_t x_row_stride, const void *residual, const float *weight, const float *scale,
                          float eps, void *y, void *h, float *rstd, void *hip_stream) {
  ssm::api_clear_error();
  SSM_TRY(check_row(rows, dim, dim, "dim"));
  SSM_TRY(check_residual_dtype(io_dtype, residual_dtype));
  SSM_TRY(check_row_stride("x", x_row_stride, dim, rows, io_dtype));
  const Ptr ps[] = {{"x", x, true, 16},       {"residual", residual, true, 16}, {"weight", weight, true, 16},
                    {"scale", scale, false, 16}, {"y", y, true, 16},            {"h", h, true, 16},
                    {"rstd", rstd, false, 4}};
  SSM_TRY_PTRS(ps);
  ssm::ResidualNormArgs a{};
  a.rows = rows, a.dim = dim, a.x_stride = x_row_stride, a.x = x, a.residual = residual, a.weight = weight, a.scale = scale;
  a.eps = eps, a.y = y, a.h_out = h, a.rstd_out = rstd;
  return api_hip_status(ssm::launch_residual_norm_fwd(a, io_dtype, residual_dtype, (hipStream_t)hip_stream), "ssm_residual_norm_fwd launch");
}

int64_t ssm_residual_norm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
  if (check_row(rows, dim, dim, "dim") != SSM_OK) return -1;
  return ssm::residual_norm_bwd_workspace_bytes(rows, dim);
}

int ssm_residual_norm_bwd(int64_t rows, int64_t dim, int io_dtype, int residual_dtype, const void *dy, const void *dh,
                          const void *h, const float *rstd, const float *weight, const void *x, int64_t x_row_stride,
                          const float *scale, void *dx, void *dresidual, float *dweight, float *dscale,
                          void *workspace, int64_t workspace_bytes, void *hip_stream) {
  ssm::api_clear_error();
  SSM_TRY(check_row(rows, dim, dim, "dim"));
  SSM_TRY(check_residual_dtype(io_dtype, residual_dtype));
  const Ptr ps[] = {{"dy", dy, true, 16},        {"dh", dh, false, 16},     {"h", h, true, 16},
                    {"rstd", rstd, true, 4},     {"weight", weight, true, 16}, {"x", x, dscale != nullptr, 16},
                    {"scale", scale, false, 16}, {"dx", dx, false, 16},     {"dresidual", dresidual, true, 16},
                    {"dweight", dweight, true, 4}, {"dscale", dscale, false, 4}};
  SSM_TRY_PTRS(ps);
  if (dscale) SSM_TRY(check_row_stride("x", x_row_stride, dim, rows, io_dtype));
  if (dscale && !scale) return api_fail(SSM_ERR_NULL_ARG, "dscale is given without scale");
  SSM_TRY(check_workspace(workspace, workspace_bytes, ssm::residual_norm_bwd_workspace_bytes(rows, dim)));
  ssm::ResidualNormArgs a{};
  a.rows = rows, a.dim = dim, a.x_stride = x_row_stride, a.x = x, a.dy = dy, a.dh = dh, a.h = h, a.rstd = rstd;
  a.weight = weight, a.scale = scale, a.dx = dx, a.dresidual = dresidual, a.dweight = dweight, a.dscale = dscale;
  a.workspace = workspace;
  return api_hip_status(ssm::launch_residual_norm_bwd(a, io_dtype, residual_dtype, (hipStream_t)hip_stream), "ssm_residual_norm_bwd launch");
}

int ssm_gated_norm_fwd(int64_t rows, int64_t dim, int64_t group, int io_dtype, const void *x, int64_t x_row_stride,
                       const void *z, int64_t z_row_stride, const float *weight, float eps, int gate_first, void *y,
                       float *rstd, void *hip_stream) {
  ssm::api_clear_error();
  SSM_TRY(check_row(rows, dim, group, "group"));
  SSM_TRY(check_dtype(io_dtype));
  const Ptr ps[] = {{"x", x, true, 16}, {"z", z, false, 16}, {"weight", weight, true, 16}, {"y", y, true, 16}, {"rstd", rstd, false, 4}};
  SSM_TRY_PTRS(ps);
  SSM_TRY(check_row_stride("x", x_row_stride, dim, rows, io_dtype));
  if (z) SSM_TRY(check_row_stride("z", z_row_stride, dim, rows, io_dtype));
  ssm::GatedNormArgs a{};
  a.rows = rows, a.dim = dim, a.group = group, a.x = x, a.x_stride = x_row_stride, a.z = z, a.z_stride = z_row_stride;
  a.weight = weight, a.eps = eps, a.gate_first = gate_first != 0, a.y = y, a.rstd_out = rstd;
  return api_hip_status(ssm::launch_gated_norm_fwd(a, io_dtype, (hipStream_t)hip_stream), "ssm_gated_norm_fwd launch");
}

int64_t ssm_gated_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, int64_t group) {
  if (check_row(rows, dim, group, "group") != SSM_OK) return -1;
  return ssm::gated_norm_bwd_workspace_bytes(rows, dim, group);
}

int ssm_gated_norm_bwd(int64_t rows, int64_t dim, int64_t group, int io_dtype, const void *dy, const void *x,
                       int64_t x_row_stride, const void *z, int64_t z_row_stride, const float *weight,
                       const float *rstd, int gate_first, void *dx, void *dz, float *dweight, void *workspace,
                       int64_t workspace_bytes, void *hip_stream) {
  ssm::api_clear_error();
  SSM_TRY(check_row(rows, dim, group, "group"));
  SSM_TRY(check_dtype(io_dtype));
  const Ptr ps[] = {{"dy", dy, true, 16},    {"x", x, true, 16},  {"z", z, false, 16},  {"weight", weight, true, 16},
                    {"rstd", rstd, true, 4}, {"dx", dx, true, 16}, {"dz", dz, false, 16}, {"dweight", dweight, true, 4}};
  SSM_TRY_PTRS(ps);
  if ((z == nullptr) != (dz == nullptr)) return api_fail(SSM_ERR_NULL_ARG, "dz must be given if and only if z is");
  SSM_TRY(check_row_stride("x", x_row_stride, dim, rows, io_dtype));
  if (z) SSM_TRY(check_row_stride("z", z_row_stride, dim, rows, io_dtype));
  SSM_TRY(check_workspace(workspace, workspace_bytes, ssm::gated_norm_bwd_workspace_bytes(rows, dim, group)));
  ssm::GatedNormArgs a{};
  a.rows = rows, a.dim = dim, a.group = group, a.x = x, a.x_stride = x_row_stride, a.z = z, a.z_stride = z_row_stride;
  a.dy = dy, a.weight = weight, a.rstd = rstd, a.gate_first = gate_first != 0, a.dx = dx, a.dz = dz, a.dweight = dweight;
  a.workspace = workspace;
  return api_hip_status(ssm::launch_gated_norm_bwd(a, io_dtype, (hipStream_t)hip_stream), "ssm_gated_norm_bwd launch");
}

}  // extern "C"
