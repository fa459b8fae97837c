// mixer_kernels.hpp -- argument blocks and launchers of the gated recurrence,
// the causal convolution and the norm and rotation of heads (ssm_block.h), shared
// by the C-ABI layer (mixer_api.cpp) and the HIP kernel files.  Sizes here are
// already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mixer_plans.hpp"

namespace ssm {

// (batch, step, channel) tensor, strides in elements, channels adjacent.
struct View3 {
  const void *p;
  int64_t sb, st;
};

struct RecurrenceArgs {
  int64_t B, L, D;
  View3 x, g, ig, z, dy;  // g: the decay's gate, ig: the input's (p NULL = none)
  const float *decay;     // NULL: the logistic form
  float sharpness;
  const float *state0, *dstate_final;
  const uint8_t *starts;
  const int32_t *lengths;
  void *y;
  float *state_final, *states;  // states: written by the forward, read by the backward
  void *dx, *dg, *dig, *dz;
  float *ddecay, *dstate0;
  void *workspace;
};

struct RecurrenceUpdateArgs {
  int64_t B, D;
  View3 x, g, ig, z;
  const float *decay;
  float sharpness;
  float *state;
  void *y;
};

struct ConvArgs {
  int64_t B, L, D;
  int width, silu;
  View3 x, dy;
  const float *weight, *bias;
  const void *state0, *dstate_final;
  const uint8_t *starts;
  const int32_t *lengths;
  void *y, *state_final, *dx, *dstate0;
  float *dweight, *dbias;
  void *state;  // of the single token, in place
  void *workspace;
};

// (batch, step, head, element) tensor, strides in elements, elements adjacent.
struct HeadView {
  const void *p;
  int64_t sb, st, sh;
};

struct HeadNormArgs {
  int64_t B, L;
  int Hq, Hk, d, rot;
  HeadView q, k, dq_out, dk_out;
  const float *wq, *wk;
  int64_t w_h;  // elements from one head's weight to the next, 0 if they share one
  const int64_t *pos;
  int64_t pos_b;  // elements from one batch row's positions to the next
  const double *inv_freq;
  float eps;
  int norm, interleaved;
  void *q_out, *k_out, *dq, *dk;
  float *dwq, *dwk;
  void *workspace;
};

int64_t recurrence_fwd_workspace_bytes(int64_t B, int64_t L, int64_t D, int io_dtype);
int64_t recurrence_bwd_workspace_bytes(int64_t B, int64_t L, int64_t D, int io_dtype);
int64_t conv_bwd_workspace_bytes(int64_t B, int64_t L, int64_t D, int width);
int64_t head_norm_bwd_workspace_bytes(int64_t B, int64_t L, int64_t Hq, int64_t Hk, int64_t d);

// Each launcher enqueues its kernels on `stream` and returns the first HIP
// error reported while enqueuing (hipSuccess otherwise).
hipError_t launch_recurrence_fwd(const RecurrenceArgs &a, int io_dtype, hipStream_t stream);
hipError_t launch_recurrence_bwd(const RecurrenceArgs &a, int io_dtype, hipStream_t stream);
hipError_t launch_recurrence_update(const RecurrenceUpdateArgs &a, int io_dtype, hipStream_t stream);
hipError_t launch_conv_fwd(const ConvArgs &a, int io_dtype, hipStream_t stream);
hipError_t launch_conv_bwd(const ConvArgs &a, int io_dtype, hipStream_t stream);
hipError_t launch_conv_update(const ConvArgs &a, int io_dtype, hipStream_t stream);
hipError_t launch_head_norm_fwd(const HeadNormArgs &a, int io_dtype, hipStream_t stream);
hipError_t launch_head_norm_bwd(const HeadNormArgs &a, int io_dtype, hipStream_t stream);

// out[c] = sum over rows of part[row][c] in a fixed order, c < n; columns from
// `split` on go to out2 (NULL = dropped).
hipError_t launch_sum_rows(const float *part, int64_t rows, int64_t n, int64_t split, float *out, float *out2, hipStream_t stream);

}  // namespace ssm
