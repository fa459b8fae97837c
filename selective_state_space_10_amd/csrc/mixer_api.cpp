// mixer_api.cpp -- the extern "C" entry points of the gated recurrence, the
// causal convolution and the norm and rotation of heads (include/ssm_block.h):
// argument validation (before anything is enqueued), size queries and dispatch
// to the HIP launchers.  No device code lives here.
#include <math.h>

#include "api_checks.hpp"
#include "mixer_kernels.hpp"

using ssm::api_fail;
using ssm::api_hip_status;
using ssm::check_dtype;
using ssm::check_workspace;
using ssm::Ptr;

static_assert(SSM_RECURRENCE_CHUNK == ssm::kRecurrenceChunk, "chunk length of the header and the kernels");

namespace {

int check_seq(int64_t batch, int64_t seqlen, int64_t dim) {
  if (batch < 1 || seqlen < 1 || dim < 1)
    return api_fail(SSM_ERR_BAD_SHAPE, "sizes must be >= 1 (batch=%lld seqlen=%lld dim=%lld)", (long long)batch, (long long)seqlen, (long long)dim);
  if (dim % 8 != 0 || dim > ssm::kMaxStep)
    return api_fail(SSM_ERR_UNSUPPORTED, "dim=%lld must be a multiple of 8 up to 2^23", (long long)dim);
  if (batch > 65536) return api_fail(SSM_ERR_UNSUPPORTED, "batch=%lld exceeds 2^16", (long long)batch);
  int64_t n;
  if (!ssm::product_ok(batch * dim, seqlen, &n)) return api_fail(SSM_ERR_BAD_SHAPE, "tensors of more than 2^40 elements");
  return SSM_OK;
}

// Tensors of at most 2^40 elements, in workgroups for 64 channels of a chunk: a
// launch has fewer than 2^32 threads.
int check_recurrence(int64_t batch, int64_t seqlen, int64_t dim) {
  SSM_TRY(check_seq(batch, seqlen, dim));
  if (batch * ((dim + 63) / 64) > ((int64_t)1 << 22) / ((seqlen + SSM_RECURRENCE_CHUNK - 1) / SSM_RECURRENCE_CHUNK))
    return api_fail(SSM_ERR_UNSUPPORTED, "batch * ceil(dim / 64) * ceil(seqlen / 128) exceeds 2^22");
  return SSM_OK;
}

// The same for threads of 4 channels and up to 32 steps, and of 4 channels of a last state.
int check_conv(int64_t batch, int64_t seqlen, int64_t dim) {
  SSM_TRY(check_seq(batch, seqlen, dim));
  if (seqlen > ((int64_t)1 << 30)) return api_fail(SSM_ERR_UNSUPPORTED, "seqlen=%lld exceeds 2^30", (long long)seqlen);
  if (batch * (dim / 8) > ((int64_t)1 << 30) / ((seqlen + 31) / 32 + 1))
    return api_fail(SSM_ERR_UNSUPPORTED, "batch * dim / 8 * (ceil(seqlen / 32) + 1) exceeds 2^30");
  return SSM_OK;
}

// one_step: stride_step is not used.  optional: the view may be NULL.
int check_view3(const char *name, const ssm_view3 *v, int io_dtype, bool optional = false, bool one_step = false) {
  if (optional && v == nullptr) return SSM_OK;
  SSM_TRY(ssm::check_view_ptr(name, v, v ? v->ptr : nullptr));
  const int64_t step = one_step ? 0 : v->stride_step;
  SSM_TRY(ssm::check_stride(name, v->stride_batch, io_dtype));
  SSM_TRY(ssm::check_stride(name, step, io_dtype));
  if (step > ssm::kMaxStep) return api_fail(SSM_ERR_UNSUPPORTED, "%s has a step stride over 2^23 elements", name);
  return SSM_OK;
}

int check_view4(const char *name, const ssm_view4 *v, int io_dtype) {
  SSM_TRY(ssm::check_view_ptr(name, v, v ? v->ptr : nullptr));
  SSM_TRY(ssm::check_stride(name, v->stride_batch, io_dtype));
  SSM_TRY(ssm::check_stride(name, v->stride_step, io_dtype));
  SSM_TRY(ssm::check_stride(name, v->stride_head, io_dtype));
  return SSM_OK;
}

int check_sharpness(const float *decay, float sharpness) {
  if (decay != nullptr && !(sharpness > 0.0f && isfinite(sharpness)))
    return api_fail(SSM_ERR_UNSUPPORTED, "sharpness=%g must be positive and finite", (double)sharpness);
  return SSM_OK;
}

int check_width(int width) {
  if (width < 1 || width > 4) return api_fail(SSM_ERR_UNSUPPORTED, "width=%d not in 1..4", width);
  return SSM_OK;
}

int check_heads(int64_t batch, int64_t seqlen, int64_t q_heads, int64_t k_heads, int64_t dim) {
  if (batch < 1 || seqlen < 1 || q_heads < 1 || k_heads < 0 || dim < 1)
    return api_fail(SSM_ERR_BAD_SHAPE, "sizes must be >= 1 (batch=%lld seqlen=%lld q_heads=%lld k_heads=%lld dim=%lld)", (long long)batch,
                    (long long)seqlen, (long long)q_heads, (long long)k_heads, (long long)dim);
  if (dim % 8 != 0 || dim > 256) return api_fail(SSM_ERR_UNSUPPORTED, "dim=%lld must be a multiple of 8 up to 256", (long long)dim);
  if (q_heads > 65536 || k_heads > 65536 || q_heads + k_heads > 65536)
    return api_fail(SSM_ERR_UNSUPPORTED, "q_heads=%lld and k_heads=%lld exceed 65536 together", (long long)q_heads, (long long)k_heads);
  int64_t n;
  if (!ssm::product_ok(batch, seqlen, &n) || !ssm::product_ok(n, (q_heads + k_heads) * dim, &n))
    return api_fail(SSM_ERR_BAD_SHAPE, "tensors of more than 2^40 elements");
  return SSM_OK;
}

int check_rotary(int64_t rotary, int64_t dim, const int64_t *positions, const double *inv_freq) {
  if (rotary < 0 || rotary > dim || rotary % 8 != 0)
    return api_fail(SSM_ERR_UNSUPPORTED, "rotary=%lld must be a multiple of 8 up to dim=%lld", (long long)rotary, (long long)dim);
  if ((positions != nullptr) != (rotary > 0) || (inv_freq != nullptr) != (rotary > 0))
    return api_fail(SSM_ERR_NULL_ARG, "positions and inv_freq must be given if and only if rotary is not 0");
  return SSM_OK;
}

int check_weights(int64_t k_heads, const float *q_weight, const float *k_weight, int norm, float eps) {
  if (!norm && (q_weight || k_weight)) return api_fail(SSM_ERR_NULL_ARG, "weights are given without a norm");
  if (k_heads > 0 && (q_weight == nullptr) != (k_weight == nullptr))
    return api_fail(SSM_ERR_NULL_ARG, "q_weight and k_weight must be given both or neither");
  if (k_heads == 0 && k_weight) return api_fail(SSM_ERR_NULL_ARG, "k_weight is given without k");
  if (norm && !(eps >= 0.0f)) return api_fail(SSM_ERR_UNSUPPORTED, "eps=%g must not be negative", (double)eps);
  return SSM_OK;
}

ssm::View3 view(const ssm_view3 *v) { return v ? ssm::View3{v->ptr, v->stride_batch, v->stride_step} : ssm::View3{nullptr, 0, 0}; }
ssm::HeadView view(const ssm_view4 *v) {
  return v ? ssm::HeadView{v->ptr, v->stride_batch, v->stride_step, v->stride_head} : ssm::HeadView{nullptr, 0, 0, 0};
}

}  // namespace

extern "C" {

int64_t ssm_gated_recurrence_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype) {
  if (check_recurrence(batch, seqlen, dim) != SSM_OK || check_dtype(io_dtype) != SSM_OK) return -1;
  return ssm::recurrence_fwd_workspace_bytes(batch, seqlen, dim, io_dtype);
}

int ssm_gated_recurrence_fwd(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype, const ssm_view3 *x,
                             const ssm_view3 *decay_gate, const ssm_view3 *input_gate, const ssm_view3 *z, const float *decay,
                             float sharpness, const float *state0, const uint8_t *starts, const int32_t *lengths, void *y,
                             float *state_final, float *states, void *workspace, int64_t workspace_bytes, void *hip_stream) {
  ssm::api_clear_error();
  SSM_TRY(check_recurrence(batch, seqlen, dim));
  SSM_TRY(check_dtype(io_dtype));
  SSM_TRY(check_sharpness(decay, sharpness));
  SSM_TRY(check_view3("x", x, io_dtype));
  SSM_TRY(check_view3("decay_gate", decay_gate, io_dtype));
  SSM_TRY(check_view3("input_gate", input_gate, io_dtype, true));
  SSM_TRY(check_view3("z", z, io_dtype, true));
  const Ptr ps[] = {{"decay", decay, false, 16}, {"state0", state0, false, 16},           {"lengths", lengths, false, 4},
                    {"y", y, true, 16},          {"state_final", state_final, false, 16}, {"states", states, false, 16}};
  SSM_TRY_PTRS(ps);
  SSM_TRY(check_workspace(workspace, workspace_bytes, ssm::recurrence_fwd_workspace_bytes(batch, seqlen, dim, io_dtype)));
  ssm::RecurrenceArgs a{};
  a.B = batch, a.L = seqlen, a.D = dim, a.x = view(x), a.g = view(decay_gate), a.ig = view(input_gate), a.z = view(z);
  a.decay = decay, a.sharpness = sharpness, a.state0 = state0, a.starts = starts, a.lengths = lengths;
  a.y = y, a.state_final = state_final, a.states = states, a.workspace = workspace;
  return api_hip_status(ssm::launch_recurrence_fwd(a, io_dtype, (hipStream_t)hip_stream), "ssm_gated_recurrence_fwd launch");
}

int64_t ssm_gated_recurrence_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype) {
  if (check_recurrence(batch, seqlen, dim) != SSM_OK || check_dtype(io_dtype) != SSM_OK) return -1;
  return ssm::recurrence_bwd_workspace_bytes(batch, seqlen, dim, io_dtype);
}

int ssm_gated_recurrence_bwd(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype, const ssm_view3 *dy, const ssm_view3 *x,
                             const ssm_view3 *decay_gate, const ssm_view3 *input_gate, const ssm_view3 *z, const float *decay,
                             float sharpness, const float *states, const uint8_t *starts, const int32_t *lengths,
                             const float *dstate_final, void *dx, void *ddecay_gate, void *dinput_gate, void *dz, float *ddecay,
                             float *dstate0, void *workspace, int64_t workspace_bytes, void *hip_stream) {
  ssm::api_clear_error();
  SSM_TRY(check_recurrence(batch, seqlen, dim));
  SSM_TRY(check_dtype(io_dtype));
  SSM_TRY(check_sharpness(decay, sharpness));
  SSM_TRY(check_view3("dy", dy, io_dtype));
  SSM_TRY(check_view3("x", x, io_dtype));
  SSM_TRY(check_view3("decay_gate", decay_gate, io_dtype));
  SSM_TRY(check_view3("input_gate", input_gate, io_dtype, true));
  SSM_TRY(check_view3("z", z, io_dtype, true));
  const Ptr ps[] = {{"decay", decay, false, 16},   {"states", states, true, 16},          {"lengths", lengths, false, 4},
                    {"dstate_final", dstate_final, false, 16}, {"dx", dx, true, 16},      {"ddecay_gate", ddecay_gate, true, 16},
                    {"dinput_gate", dinput_gate, false, 16},   {"dz", dz, false, 16},     {"ddecay", ddecay, false, 16},
                    {"dstate0", dstate0, false, 16}};
  SSM_TRY_PTRS(ps);
  if ((input_gate == nullptr) != (dinput_gate == nullptr)) return api_fail(SSM_ERR_NULL_ARG, "dinput_gate must be given if and only if input_gate is");
  if ((z == nullptr) != (dz == nullptr)) return api_fail(SSM_ERR_NULL_ARG, "dz must be given if and only if z is");
  if ((decay == nullptr) != (ddecay == nullptr)) return api_fail(SSM_ERR_NULL_ARG, "ddecay must be given if and only if decay is");
  SSM_TRY(check_workspace(workspace, workspace_bytes, ssm::recurrence_bwd_workspace_bytes(batch, seqlen, dim, io_dtype)));
  ssm::RecurrenceArgs a{};
  a.B = batch, a.L = seqlen, a.D = dim, a.x = view(x), a.g = view(decay_gate), a.ig = view(input_gate), a.z = view(z), a.dy = view(dy);
  a.decay = decay, a.sharpness = sharpness, a.states = const_cast<float *>(states), a.starts = starts, a.lengths = lengths;
  a.dstate_final = dstate_final, a.dx = dx, a.dg = ddecay_gate, a.dig = dinput_gate, a.dz = dz, a.ddecay = ddecay;
  a.dstate0 = dstate0, a.workspace = workspace;
  return api_hip_status(ssm::launch_recurrence_bwd(a, io_dtype, (hipStream_t)hip_stream), "ssm_gated_recurrence_bwd launch");
}

int ssm_gated_recurrence_update(int64_t batch, int64_t dim, int io_dtype, float *state, const ssm_view3 *x,
                                const ssm_view3 *decay_gate, const ssm_view3 *input_gate, const ssm_view3 *z, const float *decay,
                                float sharpness, void *y, void *hip_stream) {
  ssm::api_clear_error();
  SSM_TRY(check_conv(batch, 1, dim));
  SSM_TRY(check_dtype(io_dtype));
  SSM_TRY(check_sharpness(decay, sharpness));
  SSM_TRY(check_view3("x", x, io_dtype, false, true));
  SSM_TRY(check_view3("decay_gate", decay_gate, io_dtype, false, true));
  SSM_TRY(check_view3("input_gate", input_gate, io_dtype, true, true));
  SSM_TRY(check_view3("z", z, io_dtype, true, true));
  const Ptr ps[] = {{"state", state, true, 16}, {"decay", decay, false, 16}, {"y", y, true, 16}};
  SSM_TRY_PTRS(ps);
  ssm::RecurrenceUpdateArgs a{};
  a.B = batch, a.D = dim, a.x = view(x), a.g = view(decay_gate), a.ig = view(input_gate), a.z = view(z);
  a.decay = decay, a.sharpness = sharpness, a.state = state, a.y = y;
  return api_hip_status(ssm::launch_recurrence_update(a, io_dtype, (hipStream_t)hip_stream), "ssm_gated_recurrence_update launch");
}

int ssm_causal_conv_fwd(int64_t batch, int64_t seqlen, int64_t dim, int width, int io_dtype, const ssm_view3 *x,
                        const float *weight, const float *bias, const void *state0, const uint8_t *starts, const int32_t *lengths,
                        int silu, void *y, void *state_final, void *hip_stream) {
  ssm::api_clear_error();
  SSM_TRY(check_conv(batch, seqlen, dim));
  SSM_TRY(check_width(width));
  SSM_TRY(check_dtype(io_dtype));
  SSM_TRY(check_view3("x", x, io_dtype));
  const Ptr ps[] = {{"weight", weight, true, 16},   {"bias", bias, false, 16}, {"state0", state0, false, 16},
                    {"lengths", lengths, false, 4}, {"y", y, true, 16},        {"state_final", state_final, false, 16}};
  SSM_TRY_PTRS(ps);
  if (width == 1 && (state0 || state_final)) return api_fail(SSM_ERR_NULL_ARG, "a convolution of width 1 has no state");
  ssm::ConvArgs a{};
  a.B = batch, a.L = seqlen, a.D = dim, a.width = width, a.silu = silu != 0, a.x = view(x), a.weight = weight, a.bias = bias;
  a.state0 = state0, a.starts = starts, a.lengths = lengths, a.y = y, a.state_final = state_final;
  return api_hip_status(ssm::launch_conv_fwd(a, io_dtype, (hipStream_t)hip_stream), "ssm_causal_conv_fwd launch");
}

int64_t ssm_causal_conv_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int width) {
  if (check_conv(batch, seqlen, dim) != SSM_OK || check_width(width) != SSM_OK) return -1;
  return ssm::conv_bwd_workspace_bytes(batch, seqlen, dim, width);
}

int ssm_causal_conv_bwd(int64_t batch, int64_t seqlen, int64_t dim, int width, int io_dtype, const ssm_view3 *dy,
                        const ssm_view3 *x, const float *weight, const float *bias, const void *state0, const uint8_t *starts,
                        const int32_t *lengths, int silu, const void *dstate_final, void *dx, float *dweight, float *dbias,
                        void *dstate0, void *workspace, int64_t workspace_bytes, void *hip_stream) {
  ssm::api_clear_error();
  SSM_TRY(check_conv(batch, seqlen, dim));
  SSM_TRY(check_width(width));
  SSM_TRY(check_dtype(io_dtype));
  SSM_TRY(check_view3("dy", dy, io_dtype));
  SSM_TRY(check_view3("x", x, io_dtype));
  const Ptr ps[] = {{"weight", weight, true, 16},   {"bias", bias, false, 16}, {"state0", state0, false, 16},
                    {"lengths", lengths, false, 4}, {"dstate_final", dstate_final, false, 16}, {"dx", dx, true, 16},
                    {"dweight", dweight, true, 16}, {"dbias", dbias, false, 16}, {"dstate0", dstate0, false, 16}};
  SSM_TRY_PTRS(ps);
  if (width == 1 && (state0 || dstate_final || dstate0)) return api_fail(SSM_ERR_NULL_ARG, "a convolution of width 1 has no state");
  SSM_TRY(check_workspace(workspace, workspace_bytes, ssm::conv_bwd_workspace_bytes(batch, seqlen, dim, width)));
  ssm::ConvArgs a{};
  a.B = batch, a.L = seqlen, a.D = dim, a.width = width, a.silu = silu != 0, a.x = view(x), a.dy = view(dy), a.weight = weight;
  a.bias = bias, a.state0 = state0, a.starts = starts, a.lengths = lengths, a.dstate_final = dstate_final;
  a.dx = dx, a.dweight = dweight, a.dbias = dbias, a.dstate0 = dstate0, a.workspace = workspace;
  return api_hip_status(ssm::launch_conv_bwd(a, io_dtype, (hipStream_t)hip_stream), "ssm_causal_conv_bwd launch");
}

int ssm_causal_conv_update(int64_t batch, int64_t dim, int width, int io_dtype, void *state, const ssm_view3 *x,
                           const float *weight, const float *bias, int silu, void *y, void *hip_stream) {
  ssm::api_clear_error();
  SSM_TRY(check_conv(batch, 1, dim));
  SSM_TRY(check_width(width));
  SSM_TRY(check_dtype(io_dtype));
  SSM_TRY(check_view3("x", x, io_dtype, false, true));
  const Ptr ps[] = {{"state", state, width > 1, 16}, {"weight", weight, true, 16}, {"bias", bias, false, 16}, {"y", y, true, 16}};
  SSM_TRY_PTRS(ps);
  if (width == 1 && state) return api_fail(SSM_ERR_NULL_ARG, "a convolution of width 1 has no state");
  ssm::ConvArgs a{};
  a.B = batch, a.L = 1, a.D = dim, a.width = width, a.silu = silu != 0, a.x = view(x), a.weight = weight, a.bias = bias;
  a.state = state, a.y = y;
  return api_hip_status(ssm::launch_conv_update(a, io_dtype, (hipStream_t)hip_stream), "ssm_causal_conv_update launch");
}

int ssm_head_norm_rotary_fwd(int64_t batch, int64_t seqlen, int64_t q_heads, int64_t k_heads, int64_t dim, int64_t rotary,
                             int io_dtype, const ssm_view4 *q, const ssm_view4 *k, const float *q_weight, const float *k_weight,
                             int weight_per_head, const int64_t *positions, int positions_per_batch, const double *inv_freq,
                             float eps, int norm, int interleaved, void *q_out, void *k_out, void *hip_stream) {
  ssm::api_clear_error();
  SSM_TRY(check_heads(batch, seqlen, q_heads, k_heads, dim));
  SSM_TRY(check_dtype(io_dtype));
  SSM_TRY(check_rotary(rotary, dim, positions, inv_freq));
  SSM_TRY(check_weights(k_heads, q_weight, k_weight, norm, eps));
  SSM_TRY(check_view4("q", q, io_dtype));
  if (k_heads > 0) SSM_TRY(check_view4("k", k, io_dtype));
  const Ptr ps[] = {{"q_weight", q_weight, false, 16}, {"k_weight", k_weight, false, 16}, {"positions", positions, false, 8},
                    {"inv_freq", inv_freq, false, 8},  {"q_out", q_out, true, 16},        {"k_out", k_out, k_heads > 0, 16}};
  SSM_TRY_PTRS(ps);
  ssm::HeadNormArgs a{};
  a.B = batch, a.L = seqlen, a.Hq = (int)q_heads, a.Hk = (int)k_heads, a.d = (int)dim, a.rot = (int)rotary;
  a.q = view(q), a.k = view(k_heads ? k : nullptr), a.wq = q_weight, a.wk = k_weight, a.w_h = weight_per_head ? dim : 0;
  a.pos = positions, a.pos_b = positions_per_batch ? seqlen : 0, a.inv_freq = inv_freq, a.eps = eps, a.norm = norm != 0;
  a.interleaved = interleaved != 0, a.q_out = q_out, a.k_out = k_out;
  return api_hip_status(ssm::launch_head_norm_fwd(a, io_dtype, (hipStream_t)hip_stream), "ssm_head_norm_rotary_fwd launch");
}

int64_t ssm_head_norm_rotary_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t q_heads, int64_t k_heads, int64_t dim) {
  if (check_heads(batch, seqlen, q_heads, k_heads, dim) != SSM_OK) return -1;
  return ssm::head_norm_bwd_workspace_bytes(batch, seqlen, q_heads, k_heads, dim);
}

int ssm_head_norm_rotary_bwd(int64_t batch, int64_t seqlen, int64_t q_heads, int64_t k_heads, int64_t dim, int64_t rotary,
                             int io_dtype, const ssm_view4 *dq_out, const ssm_view4 *dk_out, const ssm_view4 *q,
                             const ssm_view4 *k, const float *q_weight, const float *k_weight, int weight_per_head,
                             const int64_t *positions, int positions_per_batch, const double *inv_freq, float eps, int norm,
                             int interleaved, void *dq, void *dk, float *dq_weight, float *dk_weight, void *workspace,
                             int64_t workspace_bytes, void *hip_stream) {
  ssm::api_clear_error();
  SSM_TRY(check_heads(batch, seqlen, q_heads, k_heads, dim));
  SSM_TRY(check_dtype(io_dtype));
  SSM_TRY(check_rotary(rotary, dim, positions, inv_freq));
  SSM_TRY(check_weights(k_heads, q_weight, k_weight, norm, eps));
  SSM_TRY(check_view4("dq_out", dq_out, io_dtype));
  SSM_TRY(check_view4("q", q, io_dtype));
  if (k_heads > 0) SSM_TRY(check_view4("dk_out", dk_out, io_dtype));
  if (k_heads > 0) SSM_TRY(check_view4("k", k, io_dtype));
  const Ptr ps[] = {{"q_weight", q_weight, false, 16}, {"k_weight", k_weight, false, 16}, {"positions", positions, false, 8},
                    {"inv_freq", inv_freq, false, 8},  {"dq", dq, true, 16},              {"dk", dk, k_heads > 0, 16},
                    {"dq_weight", dq_weight, false, 16}, {"dk_weight", dk_weight, false, 16}};
  SSM_TRY_PTRS(ps);
  if ((q_weight == nullptr) != (dq_weight == nullptr) || (k_weight == nullptr) != (dk_weight == nullptr))
    return api_fail(SSM_ERR_NULL_ARG, "dq_weight and dk_weight must be given if and only if their weights are");
  if (q_weight) SSM_TRY(check_workspace(workspace, workspace_bytes, ssm::head_norm_bwd_workspace_bytes(batch, seqlen, q_heads, k_heads, dim)));
  ssm::HeadNormArgs a{};
  a.B = batch, a.L = seqlen, a.Hq = (int)q_heads, a.Hk = (int)k_heads, a.d = (int)dim, a.rot = (int)rotary;
  a.q = view(q), a.k = view(k_heads ? k : nullptr), a.dq_out = view(dq_out), a.dk_out = view(k_heads ? dk_out : nullptr);
  a.wq = q_weight, a.wk = k_weight, a.w_h = weight_per_head ? dim : 0;
  a.pos = positions, a.pos_b = positions_per_batch ? seqlen : 0, a.inv_freq = inv_freq, a.eps = eps, a.norm = norm != 0;
  a.interleaved = interleaved != 0, a.dq = dq, a.dk = dk, a.dwq = dq_weight, a.dwk = dk_weight, a.workspace = workspace;
  return api_hip_status(ssm::launch_head_norm_bwd(a, io_dtype, (hipStream_t)hip_stream), "ssm_head_norm_rotary_bwd launch");
}

}  // extern "C"
