// block_kernels.hpp -- argument blocks and launchers of the block operators
// (ssm_block.h), shared by the C-ABI layer (block_api.cpp) and the HIP kernel
// files.  Sizes here are already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm {

// (batch, step, head, element) tensor, strides in elements, elements adjacent;
// head h of the kernel reads head h / share.
struct View4 {
  const void *p;
  int64_t sb, st, sh;
  int share;
};

struct DecayAttnArgs {
  int64_t B, L, H, G, dk, dv;
  View4 q, k, v, dout;
  const float *g;     // log decays
  int64_t g_b, g_t;   // their strides (elements); both 0 for one decay per head
  float scale;
  const float *state0, *dstate_final;
  float *state_final, *dstate0, *dlog_decay;
  void *o, *dq, *dk_out, *dv_out;
  void *workspace;
};

struct DecayUpdateArgs {
  int64_t B, H, G, dk, dv;
  float *state;
  View4 q, k, v;
  const float *g;
  int64_t g_b;
  float scale;
  void *o;
};

struct ResidualNormArgs {
  int64_t rows, dim, x_stride;
  const void *x, *residual, *dy, *dh, *h;
  const float *weight, *scale, *rstd;
  float eps;
  void *y, *h_out, *dx, *dresidual;
  float *rstd_out, *dweight, *dscale;
  void *workspace;
};

struct GatedNormArgs {
  int64_t rows, dim, group, x_stride, z_stride;
  const void *x, *z, *dy;
  const float *weight, *rstd;
  float eps;
  int gate_first;
  void *y, *dx, *dz;
  float *rstd_out, *dweight;
  void *workspace;
};

int64_t decay_attn_fwd_workspace_bytes(const DecayAttnArgs &a, int io_dtype);
int64_t decay_attn_bwd_workspace_bytes(const DecayAttnArgs &a, int io_dtype);
int64_t residual_norm_bwd_workspace_bytes(int64_t rows, int64_t dim);
int64_t gated_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, int64_t group);

// Each launcher enqueues its kernels on `stream` and returns the first HIP
// error reported while enqueuing (hipSuccess otherwise).
hipError_t launch_decay_attn_fwd(const DecayAttnArgs &a, int io_dtype, hipStream_t stream);
hipError_t launch_decay_attn_bwd(const DecayAttnArgs &a, int io_dtype, hipStream_t stream);
hipError_t launch_decay_update(const DecayUpdateArgs &a, int io_dtype, hipStream_t stream);
hipError_t launch_residual_norm_fwd(const ResidualNormArgs &a, int io_dtype, int res_dtype, hipStream_t stream);
hipError_t launch_residual_norm_bwd(const ResidualNormArgs &a, int io_dtype, int res_dtype, hipStream_t stream);
hipError_t launch_gated_norm_fwd(const GatedNormArgs &a, int io_dtype, hipStream_t stream);
hipError_t launch_gated_norm_bwd(const GatedNormArgs &a, int io_dtype, hipStream_t stream);

}  // namespace ssm
