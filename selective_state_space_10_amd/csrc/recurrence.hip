// recurrence.hip -- the gated recurrence h_t = a_t h_{t-1} + s_t i_t x_t.
#include "mixer_device.hpp"
#include "mixer_kernels.hpp"

namespace ssm {

namespace {

// The decay's gate.  Power form: r = sigmoid(g), log2 a = rate2 r, s^2 = 1 - a^2,
// by the series of -expm1(2 log a) where a is near 1: four terms up to 1/8 leave
// (1/8)^5 / 720 < 2^-24 relative, beyond it 1 - a^2 loses 2^-24 / (1 - e^-1/8) of
// itself, half of that in s.  Logistic form: a = r, s = 1 - r.
struct Gate {
  float a, s, r, o, la2;  // o = 1 - r
};
template <bool POWER>
__device__ __forceinline__ Gate gate_of(float g, float rate2) {
  Gate q;
  sigmoid_both(g, q.r, q.o);
  if constexpr (POWER) {
    q.la2 = rate2 * q.r;
    q.a = fast_exp2(q.la2);
    const float v = 2.0f * kLn2 * q.la2;
    const float p = fmaf(v, fmaf(v, fmaf(v, fmaf(v, 1.0f / 120, 1.0f / 24), 1.0f / 6), 0.5f), 1.0f);
    const float m = fabsf(v) < 0.125f ? -v * p : fmaf(-q.a, q.a, 1.0f);
    q.s = __builtin_amdgcn_sqrtf(m);
  } else {
    q.la2 = 0.0f;
    q.a = q.r;
    q.s = q.o;
  }
  return q;
}

__device__ __forceinline__ float softplus_exact(float v) { return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))); }
// log2 of the smallest decay
template <bool POWER>
__device__ __forceinline__ float rate_of(const RecurrenceArgs &a, int64_t c) {
  return POWER ? -a.sharpness * softplus_exact(a.decay[c]) * kLog2e : 0.0f;
}

template <typename T, bool POWER>
__global__ void __launch_bounds__(64) recurrence_fwd_kernel(RecurrenceArgs a) {
  const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
  if (c >= a.D) return;
  const float rate2 = rate_of<POWER>(a, c);
  const int len = row_length(a.lengths, b, a.L);
  const int64_t K = (a.L + kRecurrenceChunk - 1) / kRecurrenceChunk;
  float h = a.state0 ? a.state0[b * a.D + c] : 0.0f;
  for (int64_t t = 0; t < a.L; ++t) {
    if (a.states && t % kRecurrenceChunk == 0) a.states[(b * K + t / kRecurrenceChunk) * a.D + c] = h;
    float y = 0.0f;
    if (t < len) {
      const Gate q = gate_of<POWER>(load_io((const T *)a.g.p, b * a.g.sb + t * a.g.st + c), rate2);
      float u = load_io((const T *)a.x.p, b * a.x.sb + t * a.x.st + c), o;
      if (a.ig.p) {
        float i;
        sigmoid_both(load_io((const T *)a.ig.p, b * a.ig.sb + t * a.ig.st + c), i, o);
        u *= i;
      }
      h = a.starts && a.starts[b * a.L + t] ? u : fmaf(q.a, h, q.s * u);
      y = h;
      if (a.z.p) y *= silu_f(load_io((const T *)a.z.p, b * a.z.sb + t * a.z.st + c));
    }
    store_one((T *)a.y + (b * a.L + t) * a.D + c, y);
  }
  if (a.state_final) a.state_final[b * a.D + c] = h;
}

template <typename T, bool POWER>
__global__ void __launch_bounds__(64) recurrence_bwd_kernel(RecurrenceArgs a) {
  __shared__ float before[kRecurrenceChunk][64];
  const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
  if (c >= a.D) return;
  const float rate2 = rate_of<POWER>(a, c);
  const int len = row_length(a.lengths, b, a.L);
  const int64_t K = (a.L + kRecurrenceChunk - 1) / kRecurrenceChunk;
  float w = a.dstate_final ? a.dstate_final[b * a.D + c] : 0.0f, acc = 0.0f;
  for (int64_t k = K - 1; k >= 0; --k) {
    const int64_t t0 = k * kRecurrenceChunk, t1 = t0 + kRecurrenceChunk < a.L ? t0 + kRecurrenceChunk : a.L;
    float h = a.states[(b * K + k) * a.D + c];
    for (int64_t t = t0; t < t1; ++t) {
      before[t - t0][threadIdx.x] = h;
      if (t < len) {
        const Gate q = gate_of<POWER>(load_io((const T *)a.g.p, b * a.g.sb + t * a.g.st + c), rate2);
        float u = load_io((const T *)a.x.p, b * a.x.sb + t * a.x.st + c), i, o;
        if (a.ig.p) {
          sigmoid_both(load_io((const T *)a.ig.p, b * a.ig.sb + t * a.ig.st + c), i, o);
          u *= i;
        }
        h = a.starts && a.starts[b * a.L + t] ? u : fmaf(q.a, h, q.s * u);
      }
    }
    for (int64_t t = t1 - 1; t >= t0; --t) {
      const int64_t out = (b * a.L + t) * a.D + c;
      float dx = 0.0f, dg = 0.0f, dig = 0.0f, dz = 0.0f;
      if (t < len) {
        Gate q = gate_of<POWER>(load_io((const T *)a.g.p, b * a.g.sb + t * a.g.st + c), rate2);
        const float x = load_io((const T *)a.x.p, b * a.x.sb + t * a.x.st + c);
        float i = 1.0f, o = 0.0f;
        if (a.ig.p) sigmoid_both(load_io((const T *)a.ig.p, b * a.ig.sb + t * a.ig.st + c), i, o);
        const bool first = a.starts && a.starts[b * a.L + t];
        if (first) q.a = 0.0f, q.s = 1.0f;
        const float u = i * x, hp = before[t - t0][threadIdx.x];
        float e = load_io((const T *)a.dy.p, b * a.dy.sb + t * a.dy.st + c);
        if (a.z.p) {
          float f, df;
          silu_both(load_io((const T *)a.z.p, b * a.z.sb + t * a.z.st + c), f, df);
          dz = e * (first ? u : fmaf(q.a, hp, q.s * u)) * df;
          e *= f;
        }
        w += e;
        const float ws = w * q.s;
        dx = ws * i;
        dig = ws * u * o;
        if (!first) {
          if constexpr (POWER) {
            const float la = kLn2 * q.la2;
            const float f = w * q.a * (la * hp - u * q.a * (q.s > 0.0f ? la * fast_rcp(q.s) : 0.0f));
            acc += f;
            dg = f * q.o;
          } else {
            dg = w * q.a * q.s * (hp - u);
          }
        }
        w = first ? 0.0f : q.a * w;
      }
      store_one((T *)a.dx + out, dx);
      store_one((T *)a.dg + out, dg);
      if (a.dig) store_one((T *)a.dig + out, dig);
      if (a.dz) store_one((T *)a.dz + out, dz);
    }
  }
  if (a.dstate0) a.dstate0[b * a.D + c] = w;
  if constexpr (POWER) {
    const float v = a.decay[c], sp = softplus_exact(v);  // sigmoid / softplus goes to 1 where both vanish
    ((float *)a.workspace)[b * a.D + c] = acc * (v < -40.0f ? 1.0f : sigmoid_f(v) / sp);
  }
}

// One token: 8 channels per lane.
template <typename T, bool POWER>
__global__ void __launch_bounds__(256) recurrence_update_kernel(RecurrenceUpdateArgs a) {
  const int64_t n8 = a.D / 8, i8 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i8 >= a.B * n8) return;
  const int64_t b = i8 / n8, c = i8 % n8 * 8;
  float x[8], g[8], i[8], z[8], h[8], l[8];
  load_vec((const T *)a.x.p + b * a.x.sb + c, x);
  load_vec((const T *)a.g.p + b * a.g.sb + c, g);
  if (a.ig.p) load_vec((const T *)a.ig.p + b * a.ig.sb + c, i);
  if (a.z.p) load_vec((const T *)a.z.p + b * a.z.sb + c, z);
  if (POWER) load_vec(a.decay + c, l);
  load_vec(a.state + b * a.D + c, h);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const Gate q = gate_of<POWER>(g[j], POWER ? -a.sharpness * softplus_f(l[j]) * kLog2e : 0.0f);
    h[j] = fmaf(q.a, h[j], q.s * (a.ig.p ? x[j] * sigmoid_f(i[j]) : x[j]));
    x[j] = a.z.p ? h[j] * silu_f(z[j]) : h[j];
  }
  store_vec(a.state + b * a.D + c, h);
  store_vec((T *)a.y + b * a.D + c, x);
}

template <typename T>
hipError_t fwd(const RecurrenceArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.D + 63) / 64), (unsigned)a.B);
  if (a.decay)
    hipLaunchKernelGGL((recurrence_fwd_kernel<T, true>), grid, dim3(64), 0, s, a);
  else
    hipLaunchKernelGGL((recurrence_fwd_kernel<T, false>), grid, dim3(64), 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t bwd(const RecurrenceArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.D + 63) / 64), (unsigned)a.B);
  if (a.decay)
    hipLaunchKernelGGL((recurrence_bwd_kernel<T, true>), grid, dim3(64), 0, s, a);
  else
    hipLaunchKernelGGL((recurrence_bwd_kernel<T, false>), grid, dim3(64), 0, s, a);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess && a.decay ? launch_sum_rows((const float *)a.workspace, a.B, a.D, a.D, a.ddecay, nullptr, s) : e;
}

template <typename T>
hipError_t update(const RecurrenceUpdateArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.B * (a.D / 8) + 255) / 256));
  if (a.decay)
    hipLaunchKernelGGL((recurrence_update_kernel<T, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((recurrence_update_kernel<T, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

int64_t recurrence_fwd_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }
int64_t recurrence_bwd_workspace_bytes(int64_t B, int64_t, int64_t D) { return B * D * 4; }

hipError_t launch_recurrence_fwd(const RecurrenceArgs &a, int io_dtype, hipStream_t s) {
  return io_dtype == 0 ? fwd<float>(a, s) : fwd<bf16>(a, s);
}
hipError_t launch_recurrence_bwd(const RecurrenceArgs &a, int io_dtype, hipStream_t s) {
  return io_dtype == 0 ? bwd<float>(a, s) : bwd<bf16>(a, s);
}
hipError_t launch_recurrence_update(const RecurrenceUpdateArgs &a, int io_dtype, hipStream_t s) {
  return io_dtype == 0 ? update<float>(a, s) : update<bf16>(a, s);
}

// ---- sums over rows of partial sums

namespace {

// A workgroup takes 16 columns, 64 lanes' worth of rows each in turn; sums in a
// fixed order.
__global__ void __launch_bounds__(1024) sum_rows_kernel(const float *part, int64_t rows, int64_t n, int64_t split, float *out, float *out2) {
  __shared__ float s[64][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int64_t col = (int64_t)blockIdx.x * 16 + c;
  float v = 0.0f;
  if (col < n) {
    constexpr int U = 4;  // loads under way
    int64_t i = r;
    for (; i + 64 * (U - 1) < rows; i += 64 * U) {
      float x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) x[u] = part[(i + 64 * u) * n + col];
#pragma unroll
      for (int u = 0; u < U; ++u) v += x[u];
    }
    for (; i < rows; i += 64) v += part[i * n + col];
  }
  s[r][c] = v;
  __syncthreads();
  for (int m = 32; m >= 1; m >>= 1) {
    if (r < m) s[r][c] += s[r + m][c];
    __syncthreads();
  }
  if (r == 0 && col < n) {
    if (col < split)
      out[col] = s[0][c];
    else if (out2)
      out2[col - split] = s[0][c];
  }
}

}  // namespace

hipError_t launch_sum_rows(const float *part, int64_t rows, int64_t n, int64_t split, float *out, float *out2, hipStream_t stream) {
  hipLaunchKernelGGL(sum_rows_kernel, dim3((unsigned)((n + 15) / 16)), dim3(1024), 0, stream, part, rows, n, split, out, out2);
  return hipGetLastError();
}

}  // namespace ssm
