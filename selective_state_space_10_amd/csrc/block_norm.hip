// block_norm.hip -- the RMS norms around a block, each fused with what is next
// to it: the residual sum and its scale before a block, the gate after its
// mixing.  Every tensor is read and written once, 8 elements per lane and access,
// a row stays in registers between its sum of squares and its result, and weights
// stay in registers over the rows that a workgroup takes: rows and groups of 128
// and more are bound by HBM (below).
//
// Mapping: TPR lanes share a row (of one group of channels), each with V
// pieces of 8 elements, piece i at (i TPR + lane) 8.  A workgroup stays in one
// group of channels, so that the gradients of weights and scales are sums in
// registers over its rows; workgroups' sums are added in order by a second
// small kernel.
//
// Measured: residual norm forward, 16384 x 2048, bf16 with fp32 stream (403 MB): 78 us;
// residual norm backward, 16384 x 2048, bf16 with fp32 stream (604 MB):
// 115 us and 7 for the second kernel; gated norm forward, 32768 x 5120 in groups of
// 128, bf16 (1.0 GB): 213 us; gated norm backward, 4099 x 5120 fp32 (420 MB): 82 us
// and 6; 5.1, 5.3, 4.7 and 5.1 TB/s, a large copy 5.0.  One row of 5120: 4 us, latency.
// Groups of 32768 x 5120, bf16, forward and backward: 128 in 215 and 364 us, 64 in 264
// and 426, 32 in 437 and 668, 16 in 846 and 1236, 8 in 1628 and 2950: at least 8
// lanes share a row, so that below 64 most of them idle and a workgroup's reads are
// parts of lines.  A group of 5120 backward takes 524 us, 3.2 TB/s.
#include "block_kernels.hpp"
#include "device_common.hpp"

namespace ssm {

namespace {

struct F8 {
  float v[8];
};

__device__ __forceinline__ F8 load8(const float *p) {
  const float4 a = ((const float4 *)p)[0], b = ((const float4 *)p)[1];
  return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ F8 load8(const bf16 *p) {
  const uint4 a = *(const uint4 *)p;
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[2 * i] = __uint_as_float(w[i] << 16), r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  return r;
}
__device__ __forceinline__ void store8(float *p, const F8 &x) {
  ((float4 *)p)[0] = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
  ((float4 *)p)[1] = make_float4(x.v[4], x.v[5], x.v[6], x.v[7]);
}
__device__ __forceinline__ void store8(bf16 *p, const F8 &x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (uint32_t)f32_to_bf16_bits(x.v[2 * i]) | ((uint32_t)f32_to_bf16_bits(x.v[2 * i + 1]) << 16);
  *(uint4 *)p = make_uint4(w[0], w[1], w[2], w[3]);
}

// Sum over the TPR lanes of a row, on all of them.  More than a wave's 64:
// over LDS, `slot` alternating between calls so that one barrier is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*lds)[16], int slot) {
#pragma unroll
  for (int d = (TPR < 64 ? TPR : 64) / 2; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  if constexpr (TPR > 64) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[slot][w] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) v += lds[slot][threadIdx.x / TPR * (TPR / 64) + i];
  }
  return v;
}

// Adds the workgroup's sums over its rows (acc, per lane and piece) in row
// order and writes one row of partial sums.
template <int TPR, int V, int NT>
__device__ __forceinline__ void put_partial(const F8 (&acc)[V], int n8, float *out, float *lds) {
  constexpr int GR = NT / TPR;
  const int l = threadIdx.x % TPR, r = threadIdx.x / TPR;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int p = i * TPR + l;
    F8 a = acc[i];
    if constexpr (GR > 1) {
      __syncthreads();
      store8(lds + threadIdx.x * 8, a);
      __syncthreads();
      if (r == 0)
        for (int k = 1; k < GR; ++k) {
          const F8 o = load8(lds + (k * TPR + l) * 8);
#pragma unroll
          for (int j = 0; j < 8; ++j) a.v[j] += o.v[j];
        }
    }
    if (r == 0 && p < n8) store8(out + p * 8, a);
  }
}

// out[c] = sum over rows of part[row][c], in a fixed order; blockIdx.y: the
// first or the second of two such sums, whose partial sums lie one after the other.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *part, int rows, int64_t dim, float *out, float *out2) {
  __shared__ float s[64][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int64_t col = (int64_t)blockIdx.x * 16 + c;
  part += blockIdx.y * rows * dim;
  if (blockIdx.y) out = out2;
  float v = 0.0f;
  if (col < dim) {
    constexpr int U = 4;  // loads under way
    int i = r;
    for (; i + 64 * (U - 1) < rows; i += 64 * U) {
      float x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) x[u] = part[(int64_t)(i + 64 * u) * dim + col];
#pragma unroll
      for (int u = 0; u < U; ++u) v += x[u];
    }
    for (; i < rows; i += 64) v += part[(int64_t)i * dim + col];
  }
  s[r][c] = v;
  __syncthreads();
  for (int n = 32; n >= 1; n >>= 1) {
    if (r < n) s[r][c] += s[r + n][c];
    __syncthreads();
  }
  if (r == 0 && col < dim) out[col] = s[0][c];
}

template <typename T, typename R, int TPR, int V, int NT>
__global__ void __launch_bounds__(NT) residual_norm_fwd_kernel(ResidualNormArgs a) {
  __shared__ float red[2][16];
  constexpr int GR = NT / TPR;
  const int l = threadIdx.x % TPR, n8 = (int)(a.dim / 8);
  F8 wt[V], sc[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i * TPR + l < n8) {
      wt[i] = load8(a.weight + (i * TPR + l) * 8);
      if (a.scale) sc[i] = load8(a.scale + (i * TPR + l) * 8);
    }
  int slot = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * GR; r0 < a.rows; r0 += (int64_t)gridDim.x * GR, slot ^= 1) {
    const int64_t row = r0 + threadIdx.x / TPR;
    const bool on = row < a.rows;
    const T *x = (const T *)a.x + row * a.x_stride;
    const R *res = (const R *)a.residual + row * a.dim;
    F8 h[V];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = i * TPR + l;
      if (on && p < n8) {
        const F8 u = load8(x + p * 8);
        h[i] = load8(res + p * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[i].v[j] = a.scale ? fmaf(sc[i].v[j], u.v[j], h[i].v[j]) : h[i].v[j] + u.v[j];
          ss = fmaf(h[i].v[j], h[i].v[j], ss);
        }
      }
    }
    ss = row_sum<TPR>(ss, red, slot);
    const float rstd = rsqrtf(ss / (float)a.dim + a.eps);
    if (on && l == 0 && a.rstd_out) a.rstd_out[row] = rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = i * TPR + l;
      if (on && p < n8) {
        store8((R *)a.h_out + row * a.dim + p * 8, h[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i].v[j] = h[i].v[j] * rstd * wt[i].v[j];
        store8((T *)a.y + row * a.dim + p * 8, h[i]);
      }
    }
  }
}

// With hat = h rstd and u = dy weight:  dresidual = dh + rstd (u - hat mean(u hat)).
template <typename T, typename R, int TPR, int V, int NT>
__global__ void __launch_bounds__(NT) residual_norm_bwd_kernel(ResidualNormArgs a, float *part_w, float *part_s) {
  __shared__ float red[2][16];
  __shared__ alignas(16) float lds[NT / TPR > 1 ? NT * 8 : 8];
  constexpr int GR = NT / TPR;
  const int l = threadIdx.x % TPR, n8 = (int)(a.dim / 8);
  F8 wt[V], sc[V], aw[V], as[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) aw[i].v[j] = as[i].v[j] = 0.0f;
    if (i * TPR + l < n8) {
      wt[i] = load8(a.weight + (i * TPR + l) * 8);
      if (a.scale) sc[i] = load8(a.scale + (i * TPR + l) * 8);
    }
  }
  int slot = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * GR; r0 < a.rows; r0 += (int64_t)gridDim.x * GR, slot ^= 1) {
    const int64_t row = r0 + threadIdx.x / TPR;
    const bool on = row < a.rows;
    const float rstd = on ? a.rstd[row] : 0.0f;
    F8 hat[V], u[V], d[V], x[V];
    float s = 0.0f;
    // Everything of the row is on its way before the sum needs the first of it
    // (16384 x 2048, bf16 and fp32: 127 us against 156 us), where registers hold it.
    constexpr bool kEarly = V <= 3;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = i * TPR + l;
      if (on && p < n8) {
        hat[i] = load8((const R *)a.h + row * a.dim + p * 8);
        u[i] = load8((const T *)a.dy + row * a.dim + p * 8);
        if (kEarly && a.dh) d[i] = load8((const R *)a.dh + row * a.dim + p * 8);
        if (kEarly && a.dscale) x[i] = load8((const T *)a.x + row * a.x_stride + p * 8);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = i * TPR + l;
      if (on && p < n8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          hat[i].v[j] *= rstd;
          aw[i].v[j] = fmaf(u[i].v[j], hat[i].v[j], aw[i].v[j]);
          u[i].v[j] *= wt[i].v[j];
          s = fmaf(u[i].v[j], hat[i].v[j], s);
        }
      }
    }
    s = row_sum<TPR>(s, red, slot) / (float)a.dim;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = i * TPR + l;
      if (on && p < n8) {
        const int64_t o = row * a.dim + p * 8;
        if (!kEarly && a.dh) d[i] = load8((const R *)a.dh + o);
        if (!kEarly && a.dscale) x[i] = load8((const T *)a.x + row * a.x_stride + p * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[i].v[j] = fmaf(rstd, u[i].v[j] - hat[i].v[j] * s, a.dh ? d[i].v[j] : 0.0f);
        store8((R *)a.dresidual + o, d[i]);
        if (a.dscale)
#pragma unroll
          for (int j = 0; j < 8; ++j) as[i].v[j] = fmaf(d[i].v[j], x[i].v[j], as[i].v[j]);
        if (a.dx) {
          if (a.scale)
#pragma unroll
            for (int j = 0; j < 8; ++j) d[i].v[j] *= sc[i].v[j];
          store8((T *)a.dx + o, d[i]);
        }
      }
    }
  }
  put_partial<TPR, V, NT>(aw, n8, part_w + (int64_t)blockIdx.x * a.dim, lds);
  if (a.dscale) put_partial<TPR, V, NT>(as, n8, part_s + (int64_t)blockIdx.x * a.dim, lds);
}

// Workgroup blockIdx.x: group blockIdx.x % ngroups of rows from blockIdx.x / ngroups on.
template <typename T, int TPR, int V, int NT>
__global__ void __launch_bounds__(NT) gated_norm_fwd_kernel(GatedNormArgs a, int ngroups, int nrow) {
  __shared__ float red[2][16];
  constexpr int GR = NT / TPR;
  const int l = threadIdx.x % TPR, n8 = (int)(a.group / 8);
  const int gi = blockIdx.x % ngroups, rb = blockIdx.x / ngroups;
  const int64_t c0 = gi * a.group;
  F8 wt[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i * TPR + l < n8) wt[i] = load8(a.weight + c0 + (i * TPR + l) * 8);
  int slot = 0;
  for (int64_t r0 = (int64_t)rb * GR; r0 < a.rows; r0 += (int64_t)nrow * GR, slot ^= 1) {
    const int64_t row = r0 + threadIdx.x / TPR;
    const bool on = row < a.rows;
    const T *x = (const T *)a.x + row * a.x_stride + c0, *z = (const T *)a.z + row * a.z_stride + c0;
    F8 t[V], f[V];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = i * TPR + l;
      if (on && p < n8) {
        t[i] = load8(x + p * 8);
        f[i] = wt[i];
        if (a.z) {
          const F8 zz = load8(z + p * 8);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float g = silu_f(zz.v[j]);
            if (a.gate_first)
              t[i].v[j] *= g;
            else
              f[i].v[j] *= g;
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(t[i].v[j], t[i].v[j], ss);
      }
    }
    ss = row_sum<TPR>(ss, red, slot);
    const float rstd = rsqrtf(ss / (float)a.group + a.eps);
    if (on && l == 0 && a.rstd_out) a.rstd_out[row * ngroups + gi] = rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = i * TPR + l;
      if (on && p < n8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) t[i].v[j] = t[i].v[j] * rstd * f[i].v[j];
        store8((T *)a.y + row * a.dim + c0 + p * 8, t[i]);
      }
    }
  }
}

// With s = sigmoid(z), gate = z s, gate' = s + gate (1 - s), hat = t rstd, and
// n = the gradient of hat weight (dy if the gate comes first, else dy gate):
//   dt = rstd (u - hat mean(u hat)), u = n weight;  dweight = sum n hat;
//   dx = dt (gate);  dz = (dt x, or dy hat weight) gate'.
template <typename T, int TPR, int V, int NT>
__global__ void __launch_bounds__(NT) gated_norm_bwd_kernel(GatedNormArgs a, int ngroups, int nrow, float *part_w) {
  __shared__ float red[2][16];
  __shared__ alignas(16) float lds[NT / TPR > 1 ? NT * 8 : 8];
  constexpr int GR = NT / TPR;
  const int l = threadIdx.x % TPR, n8 = (int)(a.group / 8);
  const int gi = blockIdx.x % ngroups, rb = blockIdx.x / ngroups;
  const int64_t c0 = gi * a.group;
  F8 wt[V], aw[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) aw[i].v[j] = 0.0f;
    if (i * TPR + l < n8) wt[i] = load8(a.weight + c0 + (i * TPR + l) * 8);
  }
  int slot = 0;
  for (int64_t r0 = (int64_t)rb * GR; r0 < a.rows; r0 += (int64_t)nrow * GR, slot ^= 1) {
    const int64_t row = r0 + threadIdx.x / TPR;
    const bool on = row < a.rows;
    const T *x = (const T *)a.x + row * a.x_stride + c0, *z = (const T *)a.z + row * a.z_stride + c0;
    const int64_t o0 = row * a.dim + c0;
    const float rstd = on ? a.rstd[row * ngroups + gi] : 0.0f;
    F8 xs[V], zs[V], ds[V];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = i * TPR + l;
      if (on && p < n8) {
        xs[i] = load8(x + p * 8);
        ds[i] = load8((const T *)a.dy + o0 + p * 8);
        if (a.z) zs[i] = load8(z + p * 8);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = i * TPR + l;
      if (on && p < n8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float gate = a.z ? silu_f(zs[i].v[j]) : 1.0f;
          const float hat = (a.gate_first ? xs[i].v[j] * gate : xs[i].v[j]) * rstd;
          const float n = a.gate_first ? ds[i].v[j] : ds[i].v[j] * gate;
          aw[i].v[j] = fmaf(n, hat, aw[i].v[j]);
          s = fmaf(n * wt[i].v[j], hat, s);
        }
      }
    }
    s = row_sum<TPR>(s, red, slot) / (float)a.group;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = i * TPR + l;
      if (on && p < n8) {
        F8 dz;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float sg = a.z ? sigmoid_f(zs[i].v[j]) : 1.0f;
          const float gate = a.z ? zs[i].v[j] * sg : 1.0f;
          const float hat = (a.gate_first ? xs[i].v[j] * gate : xs[i].v[j]) * rstd;
          const float uw = ds[i].v[j] * wt[i].v[j];
          const float u = a.gate_first ? uw : uw * gate;
          const float dt = rstd * (u - hat * s);
          dz.v[j] = (a.gate_first ? dt * xs[i].v[j] : uw * hat) * (sg + gate * (1.0f - sg));
          xs[i].v[j] = a.gate_first ? dt * gate : dt;
        }
        store8((T *)a.dx + o0 + p * 8, xs[i]);
        if (a.z) store8((T *)a.dz + o0 + p * 8, dz);
      }
    }
  }
  put_partial<TPR, V, NT>(aw, n8, part_w + (int64_t)rb * a.dim + c0, lds);
}

// Lanes per row and pieces per lane: few pieces, so that many waves share a CU,
// and few lanes without one.  Calls f with (TPR, V, NT) as integral constants.
template <int X>
struct Int {
  static constexpr int v = X;
};
template <typename F>
hipError_t by_row_length(int64_t n, F f) {
  if (n <= 64) return f(Int<8>{}, Int<1>{}, Int<256>{});
  if (n <= 128) return f(Int<16>{}, Int<1>{}, Int<256>{});
  if (n <= 256) return f(Int<32>{}, Int<1>{}, Int<256>{});
  if (n <= 512) return f(Int<64>{}, Int<1>{}, Int<256>{});
  if (n <= 1024) return f(Int<128>{}, Int<1>{}, Int<256>{});
  if (n <= 2048) return f(Int<256>{}, Int<1>{}, Int<256>{});
  if (n <= 4096) return f(Int<256>{}, Int<2>{}, Int<256>{});
  if (n <= 6144) return f(Int<256>{}, Int<3>{}, Int<256>{});
  if (n <= 8192) return f(Int<512>{}, Int<2>{}, Int<512>{});
  if (n <= 12288) return f(Int<512>{}, Int<3>{}, Int<512>{});
  return f(Int<512>{}, Int<4>{}, Int<512>{});
}
int rows_per_workgroup(int64_t n) { return n <= 64 ? 32 : n <= 128 ? 16 : n <= 256 ? 8 : n <= 512 ? 4 : n <= 1024 ? 2 : 1; }

// Workgroups that share the rows of one group of channels, `most` over all groups.
int64_t row_workgroups(int64_t rows, int64_t row_len, int64_t ngroups, int64_t most) {
  const int64_t need = (rows + rows_per_workgroup(row_len) - 1) / rows_per_workgroup(row_len);
  int64_t n = most / ngroups;
  if (n < 1) n = 1;
  return need < n ? need : n;
}
constexpr int64_t kFwdWorkgroups = 2048;
// With gradients of weights: as many as are resident at once (registers grow
// with the pieces per lane), since each writes a row of partial sums
// (2000 x 16384: 262 us with 1024, 212 us with 256; 4096 x 8192: 151 and 127 us).
int64_t bwd_workgroups(int64_t n) { return n <= 2048 ? 1024 : n <= 4096 ? 768 : n <= 6144 ? 512 : 256; }

hipError_t column_sum(const float *part, int64_t rows, int64_t dim, float *out, float *out2, hipStream_t s) {
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((dim + 15) / 16), out2 ? 2 : 1), dim3(1024), 0, s, part, (int)rows, dim, out, out2);
  return hipGetLastError();
}

template <typename T, typename R>
hipError_t residual_fwd(const ResidualNormArgs &a, hipStream_t s) {
  const unsigned grid = (unsigned)row_workgroups(a.rows, a.dim, 1, kFwdWorkgroups);
  return by_row_length(a.dim, [&](auto tpr, auto v, auto nt) {
    hipLaunchKernelGGL((residual_norm_fwd_kernel<T, R, decltype(tpr)::v, decltype(v)::v, decltype(nt)::v>), dim3(grid), dim3(decltype(nt)::v), 0, s, a);
    return hipGetLastError();
  });
}

template <typename T, typename R>
hipError_t residual_bwd(const ResidualNormArgs &a, hipStream_t s) {
  const int64_t grid = row_workgroups(a.rows, a.dim, 1, bwd_workgroups(a.dim));
  float *pw = (float *)a.workspace, *ps = pw + grid * a.dim;
  hipError_t e = by_row_length(a.dim, [&](auto tpr, auto v, auto nt) {
    hipLaunchKernelGGL((residual_norm_bwd_kernel<T, R, decltype(tpr)::v, decltype(v)::v, decltype(nt)::v>), dim3((unsigned)grid), dim3(decltype(nt)::v), 0, s, a, pw, ps);
    return hipGetLastError();
  });
  return e == hipSuccess ? column_sum(pw, grid, a.dim, a.dweight, a.dscale, s) : e;
}

template <typename T>
hipError_t gated_fwd(const GatedNormArgs &a, hipStream_t s) {
  const int64_t ng = a.dim / a.group, nrow = row_workgroups(a.rows, a.group, ng, kFwdWorkgroups);
  return by_row_length(a.group, [&](auto tpr, auto v, auto nt) {
    hipLaunchKernelGGL((gated_norm_fwd_kernel<T, decltype(tpr)::v, decltype(v)::v, decltype(nt)::v>), dim3((unsigned)(ng * nrow)), dim3(decltype(nt)::v), 0, s, a, (int)ng, (int)nrow);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t gated_bwd(const GatedNormArgs &a, hipStream_t s) {
  const int64_t ng = a.dim / a.group, nrow = row_workgroups(a.rows, a.group, ng, bwd_workgroups(a.group));
  float *pw = (float *)a.workspace;
  const hipError_t e = by_row_length(a.group, [&](auto tpr, auto v, auto nt) {
    hipLaunchKernelGGL((gated_norm_bwd_kernel<T, decltype(tpr)::v, decltype(v)::v, decltype(nt)::v>), dim3((unsigned)(ng * nrow)), dim3(decltype(nt)::v), 0, s, a, (int)ng, (int)nrow, pw);
    return hipGetLastError();
  });
  return e == hipSuccess ? column_sum(pw, nrow, a.dim, a.dweight, nullptr, s) : e;
}

}  // namespace

int64_t residual_norm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
  return 2 * row_workgroups(rows, dim, 1, bwd_workgroups(dim)) * dim * 4;
}
int64_t gated_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, int64_t group) {
  return row_workgroups(rows, group, dim / group, bwd_workgroups(group)) * dim * 4;
}

hipError_t launch_residual_norm_fwd(const ResidualNormArgs &a, int io_dtype, int res_dtype, hipStream_t s) {
  return io_dtype == 0 ? residual_fwd<float, float>(a, s) : res_dtype == 0 ? residual_fwd<bf16, float>(a, s) : residual_fwd<bf16, bf16>(a, s);
}
hipError_t launch_residual_norm_bwd(const ResidualNormArgs &a, int io_dtype, int res_dtype, hipStream_t s) {
  return io_dtype == 0 ? residual_bwd<float, float>(a, s) : res_dtype == 0 ? residual_bwd<bf16, float>(a, s) : residual_bwd<bf16, bf16>(a, s);
}
hipError_t launch_gated_norm_fwd(const GatedNormArgs &a, int io_dtype, hipStream_t s) {
  return io_dtype == 0 ? gated_fwd<float>(a, s) : gated_fwd<bf16>(a, s);
}
hipError_t launch_gated_norm_bwd(const GatedNormArgs &a, int io_dtype, hipStream_t s) {
  return io_dtype == 0 ? gated_bwd<float>(a, s) : gated_bwd<bf16>(a, s);
}

}  // namespace ssm
