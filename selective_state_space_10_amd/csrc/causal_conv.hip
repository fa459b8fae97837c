// causal_conv.hip -- the short causal depthwise convolution by itself: forward
// with a state of the last inputs, gradients, one token.
//
// Every tensor is read and written once but for the rows that chunks share: a
// lane owns 8 adjacent channels and walks over a chunk of steps with the last
// width - 1 inputs in registers; the rows before its chunk (and in the backward
// those after it, whose outputs its inputs reach) are read again, mostly from L2.
#include "mixer_device.hpp"
#include "mixer_kernels.hpp"

namespace ssm {

namespace {

constexpr int kRows = 8;  // rows whose loads are under way together

// 8 channels of a row as they lie in memory.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) { a = ((const float4 *)p)[0], b = ((const float4 *)p)[1]; }
  __device__ __forceinline__ void get(float (&v)[8]) const { v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w; }
};
template <>
struct Raw<bf16> {
  uint4 a;
  __device__ __forceinline__ void load(const bf16 *p) { a = *(const uint4 *)p; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
};

// weights of 8 channels, w[k][j], and their bias
template <int K>
__device__ __forceinline__ void load_weights(const ConvArgs &a, int64_t c, float (&w)[K][8], float (&bias)[8]) {
  float flat[8 * K];
  load_vec(a.weight + c * K, flat);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    bias[j] = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][j] = flat[j * K + k];
  }
  if (a.bias) load_vec(a.bias + c, bias);
}

// The input at step t < 0 of the state, zero without one and at other steps.
template <typename T, int K>
__device__ __forceinline__ void load_before(const ConvArgs &a, int64_t b, int64_t t, int64_t c, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  if (K > 1 && t < 0 && a.state0) load_vec((const T *)a.state0 + (b * (K - 1) + t + (K - 1)) * a.D + c, v);
}

// win[0 .. K-2] are the inputs before a step, oldest first; at a document's
// start they are nothing.
template <int K>
__device__ __forceinline__ void clear(float (&win)[K][8]) {
#pragma unroll
  for (int k = 0; k + 1 < K; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) win[k][j] = 0.0f;
}
template <int K>
__device__ __forceinline__ void shift(float (&win)[K][8]) {
#pragma unroll
  for (int k = 0; k + 1 < K; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) win[k][j] = win[k + 1][j];
}

// The inputs before step t0, into win[0 .. K-2]; none behind the row's length.
template <typename T, int K>
__device__ __forceinline__ void load_window(const ConvArgs &a, int64_t b, int64_t t0, int len, int64_t c, float (&win)[K][8]) {
#pragma unroll
  for (int k = 0; k + 1 < K; ++k) {
    const int64_t t = t0 - (K - 1) + k;
    if (t < 0 || t >= len)
      load_before<T, K>(a, b, t, c, win[k]);
    else
      load_vec((const T *)a.x.p + b * a.x.sb + t * a.x.st + c, win[k]);
  }
  if (a.starts)
#pragma unroll
    for (int k = 1; k < K; ++k) {  // a start at t0 - (K - 1) + k leaves nothing of what is before it
      const int64_t t = t0 - (K - 1) + k;
      if (k + 1 < K && t >= 0 && a.starts[b * a.L + t])
#pragma unroll
        for (int m = 0; m < k; ++m)
#pragma unroll
          for (int j = 0; j < 8; ++j) win[m][j] = 0.0f;
    }
}

// Threads: (batch row, chunk, 8 channels), channels fastest; behind them one for
// every 8 channels of the last states.
template <typename T, int K>
__global__ void __launch_bounds__(256) conv_fwd_kernel(ConvArgs a, int64_t nchunk, int steps, int64_t main_threads) {
  const int64_t n8 = a.D / 8;
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < main_threads) {
    const int64_t c = i % n8 * 8, bc = i / n8, b = bc / nchunk, t0 = bc % nchunk * steps;
    const int len = row_length(a.lengths, b, a.L);
    const int64_t t1 = t0 + steps < a.L ? t0 + steps : a.L;
    float w[K][8], bias[8], win[K][8];
    load_weights<K>(a, c, w, bias);
    load_window<T, K>(a, b, t0, len, c, win);
    const T *x = (const T *)a.x.p + b * a.x.sb + c;
    T *y = (T *)a.y + b * a.L * a.D + c;
    for (int64_t t = t0; t < t1; t += kRows) {
      Raw<T> raw[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) raw[r].load(x + (t + r < a.L ? t + r : a.L - 1) * a.x.st);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (t + r >= t1) break;
        if (a.starts && a.starts[b * a.L + t + r]) clear<K>(win);
        raw[r].get(win[K - 1]);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = bias[j];
#pragma unroll
          for (int k = 0; k < K; ++k) v[j] = fmaf(w[k][j], win[k][j], v[j]);
          if (a.silu) v[j] = silu_f(v[j]);
          if (t + r >= len) v[j] = 0.0f;
        }
        store_vec(y + (t + r) * a.D, v);
        shift<K>(win);
      }
    }
    return;
  }
  if constexpr (K > 1) {
    i -= main_threads;
    if (!a.state_final || i >= a.B * n8) return;
    const int64_t b = i / n8, c = i % n8 * 8;
    const int len = row_length(a.lengths, b, a.L);
    float win[K][8];
    load_window<T, K>(a, b, len, len, c, win);
#pragma unroll
    for (int k = 0; k + 1 < K; ++k) store_vec((T *)a.state_final + (b * (K - 1) + k) * a.D + c, win[k]);
  }
}

// dpre_s = dy_s act'(pre_s);  dx_t = sum over taps `back` of w[K-1-back] dpre_{t+back}
// where no document starts in (t, t+back];  dweight[k] = sum dpre_s x_{s-(K-1)+k}.
// A workgroup takes CG groups of 8 channels and 256 / CG chunks at once; a chunk
// of nrow steps s yields dx of nrow - (K-1) steps t and as much of the weights' sums.
template <typename T, int K, int CG>
__global__ void __launch_bounds__(256) conv_bwd_kernel(ConvArgs a, int64_t nchunk, int nrow, int ctiles, int64_t nruns, float *part) {
  constexpr int R = 256 / CG;
  __shared__ alignas(16) float lds[256 * 8];
  const int64_t ct = blockIdx.x % ctiles, run = blockIdx.x / ctiles;
  const int slot = threadIdx.x / CG;
  const int64_t c = (ct * CG + threadIdx.x % CG) * 8;
  const bool on = c < a.D;
  const int own = nrow - (K - 1);
  float w[K][8], bias[8], dw[K + 1][8];
#pragma unroll
  for (int k = 0; k <= K; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[k][j] = 0.0f;
  if (on) {
    load_weights<K>(a, c, w, bias);
    for (int64_t it = run * R + slot; it < a.B * nchunk; it += nruns * R) {
      const int64_t b = it / nchunk, t0 = it % nchunk * own;
      const int len = row_length(a.lengths, b, a.L);
      float win[K][8], d[K][8];
      load_window<T, K>(a, b, t0, len, c, win);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) d[k][j] = 0.0f;
      const T *x = (const T *)a.x.p + b * a.x.sb + c, *dy = (const T *)a.dy.p + b * a.dy.sb + c;
      int age = K - 1;  // steps of this document before step s, as far as taps reach
      if (a.starts)
#pragma unroll
        for (int k = 1; k < K; ++k) {
          const int64_t t = t0 - K + k;
          if (t >= 0 && a.starts[b * a.L + t]) age = K - 1 - k;
        }
      for (int m0 = 0; m0 < nrow && t0 + m0 - (K - 1) < a.L; m0 += kRows) {
        Raw<T> rx[kRows], ry[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const int64_t s = t0 + m0 + r < a.L ? t0 + m0 + r : a.L - 1;
          rx[r].load(x + s * a.x.st);
          ry[r].load(dy + s * a.dy.st);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const int64_t s = t0 + m0 + r, t = s - (K - 1);
          const bool live = s < len;
          if (a.starts) {
            age = age + 1 < K - 1 ? age + 1 : K - 1;
            if (s < a.L && a.starts[b * a.L + s]) {
              clear<K>(win);
              age = 0;
            }
          }
          float g[8];
          rx[r].get(win[K - 1]);
          ry[r].get(g);
#pragma unroll
          for (int k = K - 1; k > 0; --k)
#pragma unroll
            for (int j = 0; j < 8; ++j) d[k][j] = d[k - 1][j];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (!live) win[K - 1][j] = 0.0f;
            if (a.silu) {
              float pre = bias[j], f, df;
#pragma unroll
              for (int k = 0; k < K; ++k) pre = fmaf(w[k][j], win[k][j], pre);
              silu_both(pre, f, df);
              g[j] *= df;
            }
            if (!live) g[j] = 0.0f;
            d[0][j] = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k)
              if (!a.starts || k <= age) d[k][j] = fmaf(w[K - 1 - k][j], g[j], d[k][j]);
            if (m0 + r < own) {
#pragma unroll
              for (int k = 0; k < K; ++k) dw[k][j] = fmaf(g[j], win[k][j], dw[k][j]);
              dw[K][j] += g[j];
            }
          }
          if (m0 + r >= K - 1 ? t < a.L : t < 0) {
            if (K > 1 && a.dstate_final && t >= len - (K - 1) && t < len) {  // an input of the last state
              bool kept = true;
              if (a.starts)
                for (int64_t u = t < 0 ? 0 : t + 1; u < len; ++u) kept = kept && !a.starts[b * a.L + u];
              if (kept) {
                float f[8];
                load_vec((const T *)a.dstate_final + (b * (K - 1) + t - len + (K - 1)) * a.D + c, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[K - 1][j] += f[j];
              }
            }
            if (t >= 0)
              store_vec((T *)a.dx + (b * a.L + t) * a.D + c, d[K - 1]);
            else if (a.dstate0)
              store_vec((T *)a.dstate0 + (b * (K - 1) + t + (K - 1)) * a.D + c, d[K - 1]);
          }
          shift<K>(win);
        }
      }
    }
  }
  part += run * a.D * (K + 1);
#pragma unroll
  for (int k = 0; k <= K; ++k) {
    __syncthreads();
    store_vec(lds + threadIdx.x * 8, dw[k]);
    __syncthreads();
    if (slot == 0)
      for (int r = 1; r < R; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[k][j] += lds[(r * CG + threadIdx.x) * 8 + j];
    if (slot == 0 && on) {
      if (k == K)
        store_vec(part + a.D * K + c, dw[k]);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j) part[(c + j) * K + k] = dw[k][j];
    }
  }
}

template <typename T, int K>
__global__ void __launch_bounds__(256) conv_update_kernel(ConvArgs a) {
  const int64_t n8 = a.D / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.B * n8) return;
  const int64_t b = i / n8, c = i % n8 * 8;
  T *state = (T *)a.state + b * (K - 1) * a.D + c;
  float w[K][8], bias[8], win[K][8], v[8];
#pragma unroll
  for (int k = 0; k + 1 < K; ++k) load_vec(state + k * a.D, win[k]);
  load_vec((const T *)a.x.p + b * a.x.sb + c, win[K - 1]);
  load_weights<K>(a, c, w, bias);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = bias[j];
#pragma unroll
    for (int k = 0; k < K; ++k) v[j] = fmaf(w[k][j], win[k][j], v[j]);
    if (a.silu) v[j] = silu_f(v[j]);
  }
  store_vec((T *)a.y + b * a.D + c, v);
#pragma unroll
  for (int k = 0; k + 1 < K; ++k) store_vec(state + k * a.D, win[k + 1]);
}

template <int X>
struct Int {
  static constexpr int v = X;
};
template <typename F>
hipError_t by_width(int width, F f) {
  return width == 1 ? f(Int<1>{}) : width == 2 ? f(Int<2>{}) : width == 3 ? f(Int<3>{}) : f(Int<4>{});
}

constexpr int kFwdSteps = 32, kBwdRows = 64;

struct BwdPlan {
  int cg;            // groups of 8 channels per workgroup
  int64_t ctiles, nchunk, nruns;
};
BwdPlan bwd_plan(int64_t B, int64_t L, int64_t D, int width) {
  BwdPlan p;
  const int64_t n8 = D / 8;
  p.cg = n8 >= 64 ? 64 : n8 >= 32 ? 32 : n8 >= 16 ? 16 : 8;
  p.ctiles = (n8 + p.cg - 1) / p.cg;
  const int own = kBwdRows - (width - 1);
  p.nchunk = (L + own - 1) / own;
  const int64_t need = (B * p.nchunk + 256 / p.cg - 1) / (256 / p.cg), most = p.ctiles < 1024 ? 1024 / p.ctiles : 1;
  p.nruns = need < most ? need : most;
  return p;
}

template <typename T>
hipError_t fwd(const ConvArgs &a, hipStream_t s) {
  const int64_t nchunk = (a.L + kFwdSteps - 1) / kFwdSteps, n8 = a.D / 8, main = a.B * nchunk * n8;
  const int64_t threads = main + (a.state_final ? a.B * n8 : 0);
  return by_width(a.width, [&](auto k) {
    hipLaunchKernelGGL((conv_fwd_kernel<T, decltype(k)::v>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, a, nchunk, kFwdSteps, main);
    return hipGetLastError();
  });
}

template <typename T, int CG>
hipError_t bwd_cg(const ConvArgs &a, const BwdPlan &p, hipStream_t s) {
  return by_width(a.width, [&](auto k) {
    hipLaunchKernelGGL((conv_bwd_kernel<T, decltype(k)::v, CG>), dim3((unsigned)(p.ctiles * p.nruns)), dim3(256), 0, s, a, p.nchunk, kBwdRows,
                       (int)p.ctiles, p.nruns, (float *)a.workspace);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t bwd(const ConvArgs &a, hipStream_t s) {
  const BwdPlan p = bwd_plan(a.B, a.L, a.D, a.width);
  const hipError_t e = p.cg == 64 ? bwd_cg<T, 64>(a, p, s) : p.cg == 32 ? bwd_cg<T, 32>(a, p, s) : p.cg == 16 ? bwd_cg<T, 16>(a, p, s) : bwd_cg<T, 8>(a, p, s);
  if (e != hipSuccess) return e;
  return launch_sum_rows((const float *)a.workspace, p.nruns, a.D * (a.width + 1), a.D * a.width, a.dweight, a.dbias, s);
}

template <typename T>
hipError_t update(const ConvArgs &a, hipStream_t s) {
  return by_width(a.width, [&](auto k) {
    hipLaunchKernelGGL((conv_update_kernel<T, decltype(k)::v>), dim3((unsigned)((a.B * (a.D / 8) + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace

int64_t conv_bwd_workspace_bytes(int64_t B, int64_t L, int64_t D, int width) { return bwd_plan(B, L, D, width).nruns * D * (width + 1) * 4; }

hipError_t launch_conv_fwd(const ConvArgs &a, int io_dtype, hipStream_t s) { return io_dtype == 0 ? fwd<float>(a, s) : fwd<bf16>(a, s); }
hipError_t launch_conv_bwd(const ConvArgs &a, int io_dtype, hipStream_t s) { return io_dtype == 0 ? bwd<float>(a, s) : bwd<bf16>(a, s); }
hipError_t launch_conv_update(const ConvArgs &a, int io_dtype, hipStream_t s) { return io_dtype == 0 ? update<float>(a, s) : update<bf16>(a, s); }

}  // namespace ssm
