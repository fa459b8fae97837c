// causal_conv.hip -- the short causal depthwise convolution by itself: forward
// with a state of the last inputs, gradients, one token.
//
// Every tensor is read and written once but for the rows that chunks share: a
// lane owns a few adjacent channels and walks over a chunk of steps with the last
// width - 1 inputs in registers; the rows before its chunk (and in the backward
// those after it, whose outputs its inputs reach) are read again, mostly from L2.
//
// Measured, width 4, per call: forward 4 x 4096 x 5120 bf16 (336 MB) 69 us, 4.9 TB/s, a
// large copy 5.1; 8 x 2048 x 2048 fp32 (268 MB) 46 us; 1 x 2048 x 2048 bf16 (17 MB) 13 us, four loads'
// latency of 32 steps in 130 workgroups; backward 8 x 2048 x 2048 bf16
// (201 MB) on packed documents 50 us with 4 for the second kernel, 4.0 TB/s: one round of
// four waves per SIMD, whose start and end nothing overlaps; 4 x 4096 x 5120 (503 MB) 107 us.
// One token of 2048 channels takes 2.4 us, latency.
#include "mixer_device.hpp"
#include "mixer_kernels.hpp"

namespace ssm {

using namespace conv;

namespace {

template <int X>
struct Int {
  static constexpr int v = X;
};

// 4 channels of a row as they lie in memory.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 a;
  __device__ __forceinline__ void load(const float *p) { a = load_once((const float4 *)p); }
  __device__ __forceinline__ void get(float (&v)[4]) const { v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w; }
};
template <>
struct Raw<bf16> {
  uint2 a;
  __device__ __forceinline__ void load(const bf16 *p) { a = load_once((const uint2 *)p); }
  __device__ __forceinline__ void get(float (&v)[4]) const {
    const uint32_t w[2] = {a.x, a.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
};

// weights of 4 channels, w[k][j], and their bias
template <int K>
__device__ __forceinline__ void load_weights(const ConvArgs &a, int64_t c, float (&w)[K][4], float (&bias)[4]) {
  float flat[4 * K];
  load_vec(a.weight + c * K, flat);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    bias[j] = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][j] = flat[j * K + k];
  }
  if (a.bias) load_vec(a.bias + c, bias);
}

// The input at step t < 0 of the state, zero without one and at other steps.
template <typename T, int K>
__device__ __forceinline__ void load_before(const ConvArgs &a, int64_t b, int64_t t, int64_t c, float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = 0.0f;
  if (K > 1 && t < 0 && a.state0) load_vec((const T *)a.state0 + (b * (K - 1) + t + (K - 1)) * a.D + c, v);
}

// win[0 .. K-2] are the inputs before a step, oldest first; at a document's
// start they are nothing.
template <int K, int V>
__device__ __forceinline__ void clear(float (&win)[K][V]) {
#pragma unroll
  for (int k = 0; k + 1 < K; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) win[k][j] = 0.0f;
}
template <int K, int V>
__device__ __forceinline__ void shift(float (&win)[K][V]) {
#pragma unroll
  for (int k = 0; k + 1 < K; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) win[k][j] = win[k + 1][j];
}

// The inputs before step t0, into win[0 .. K-2]; none behind the row's length.
template <typename T, int K>
__device__ __forceinline__ void load_window(const ConvArgs &a, int64_t b, int64_t t0, int len, int64_t c, float (&win)[K][4]) {
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
          for (int j = 0; j < 4; ++j) win[m][j] = 0.0f;
    }
}

// Threads: (batch row, chunk, 4 channels), channels fastest; behind them one for
// every 4 channels of the last states.
template <typename T, int K>
__global__ void __launch_bounds__(256) conv_fwd_kernel(ConvArgs a, uint32_t nchunk, int steps, uint32_t main_threads) {
  const uint32_t n4 = (uint32_t)(a.D / 4);
  uint32_t i = blockIdx.x * 256 + threadIdx.x;  // (a launch has fewer than 2^32 threads)
  if (i < main_threads) {
    const uint32_t bc = i / n4, b32 = bc / nchunk;
    const int64_t c = (i - bc * n4) * 4, b = b32, t0 = (int64_t)(bc - b32 * nchunk) * steps;
    const int len = row_length(a.lengths, b, a.L);
    const int64_t t1 = t0 + steps < a.L ? t0 + steps : a.L;
    float w[K][4], bias[4], win[K][4];
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
        if (a.starts && a.starts[b * a.L + t + r]) clear<K, 4>(win);
        raw[r].get(win[K - 1]);
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = bias[j];
#pragma unroll
          for (int k = 0; k < K; ++k) v[j] = fmaf(w[k][j], win[k][j], v[j]);
          if (a.silu) v[j] = silu_f(v[j]);
          if (t + r >= len) v[j] = 0.0f;
        }
        store_vec(y + (t + r) * a.D, v);
        shift<K, 4>(win);
      }
    }
    return;
  }
  if constexpr (K > 1) {
    i -= main_threads;
    if (!a.state_final || i >= a.B * n4) return;
    const int64_t b = i / n4, c = i % n4 * 4;
    const int len = row_length(a.lengths, b, a.L);
    float win[K][4];
    load_window<T, K>(a, b, len, len, c, win);
#pragma unroll
    for (int k = 0; k + 1 < K; ++k) store_vec((T *)a.state_final + (b * (K - 1) + k) * a.D + c, win[k]);
  }
}

// Backward.  dpre_s = dy_s act'(pre_s);  dx_t = sum over taps `back` of w[K-1-back]
// dpre_{t+back} where no document starts in (t, t+back];  dweight[k] = sum dpre_s x_{s-(K-1)+k}.
//
// A wave takes two channels per lane and walks over nrow steps s with the inputs
// under the taps and the unfinished dx of the last K steps in registers: it yields
// dx of nrow - (K-1) steps t and as much of the weights' sums, which stay in registers
// over its chunks; a workgroup adds its waves' sums and a second kernel the workgroups', in order.
// All of a wave is at the same step, so that steps, starts and lengths are scalar work.
// Two channels and not eight: 74 registers' worth of sums and windows less, four waves per
// SIMD in bf16 (three in fp32) instead of two (8 x 2048 x 2048 bf16: 101 us with eight).
template <typename T>
struct Raw2;
template <>
struct Raw2<float> {
  uint32_t a, b;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t p, uint32_t lane, uint32_t step) {
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    const u2 v = __builtin_bit_cast(u2, __builtin_amdgcn_raw_buffer_load_b64(p, lane, step, kStream));
    a = v.x, b = v.y;
  }
  __device__ __forceinline__ void get(float (&v)[2]) const { v[0] = __uint_as_float(a), v[1] = __uint_as_float(b); }
};
template <>
struct Raw2<bf16> {
  uint32_t a;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t p, uint32_t lane, uint32_t step) { a = __builtin_amdgcn_raw_buffer_load_b32(p, lane, step, kStream); }
  __device__ __forceinline__ void get(float (&v)[2]) const { v[0] = __uint_as_float(a << 16), v[1] = __uint_as_float(a & 0xffff0000u); }
};
__device__ __forceinline__ void load2(const float *p, float (&v)[2]) { v[0] = ((const float2 *)p)->x, v[1] = ((const float2 *)p)->y; }
__device__ __forceinline__ void load2(const bf16 *p, float (&v)[2]) {
  const uint32_t w = *(const uint32_t *)p;
  v[0] = __uint_as_float(w << 16), v[1] = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void store2(float *p, const float (&v)[2]) { *(float2 *)p = make_float2(v[0], v[1]); }
__device__ __forceinline__ void store2(bf16 *p, const float (&v)[2]) { *(uint32_t *)p = pack_bf16(v[0], v[1]); }

__device__ __forceinline__ int uniform(int64_t v) { return __builtin_amdgcn_readfirstlane((int)v); }
// Bit i: a document starts at step t0 + i, of the steps from 0 to L.
__device__ __forceinline__ uint64_t start_bits(const uint8_t *starts, int64_t b, int t0, int L) {
  if (!starts) return 0;
  const int t = t0 + (int)(threadIdx.x & 63);
  return __ballot(t >= 0 && t < L && starts[b * L + t] != 0);
}

template <typename T, int K, bool MARKS>
__global__ void __launch_bounds__(256) conv_bwd_kernel(ConvArgs a, int nrow, int nchunk, int ctiles, int nruns, float *part) {
  constexpr int N = 2 * (K + 1);
  const int own = nrow - (K - 1);
  __shared__ float sums[4][N][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int ct = uniform(blockIdx.x % ctiles), run = uniform(blockIdx.x / ctiles);
  const int D = (int)a.D, L = (int)a.L;
  const int c_lane = (ct * 64 + lane) * 2, c = c_lane < D ? c_lane : D - 2;
  const bool on = c_lane < D;
  const uint32_t lane_bytes = (uint32_t)(c * sizeof(T));
  float w[K][2], bias[2] = {0.0f, 0.0f}, dw[K + 1][2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][j] = a.weight[(int64_t)(c + j) * K + k];
  if (a.bias) load2(a.bias + c, bias);
#pragma unroll
  for (int k = 0; k <= K; ++k) dw[k][0] = dw[k][1] = 0.0f;
  const int items = (int)a.B * nchunk;
  for (int it = run * 4 + wave; it < items; it += nruns * 4) {
    const int b32 = uniform(it / nchunk), t0 = uniform(it - b32 * nchunk) * own;
    const int64_t b = b32;
    const int len = MARKS ? uniform(row_length(a.lengths, b, L)) : L;
    const int rows = L - t0 < nrow ? L - t0 : nrow;
    const uint64_t first = MARKS ? start_bits(a.starts, b, t0, L) : 0, first2 = MARKS ? start_bits(a.starts, b, t0 + 64, L) : 0;
    const uint32_t xstep = (uint32_t)a.x.st * sizeof(T), ystep = (uint32_t)a.dy.st * sizeof(T);
    auto buffer = [&](const View3 &v, uint32_t step) {
      return __builtin_amdgcn_make_buffer_rsrc((char *)v.p + (b * v.sb + t0 * v.st) * (int64_t)sizeof(T), 0, (int)((rows - 1) * step + D * (uint32_t)sizeof(T)),
                                               0x00027000);
    };
    const auto bx = buffer(a.x, xstep), by = buffer(a.dy, ystep);
    float win[K][2], d[K][2];
#pragma unroll
    for (int k = 0; k < K; ++k) win[k][0] = win[k][1] = d[k][0] = d[k][1] = 0.0f;
    int age = K - 1;  // steps of this document before step s, as far as taps reach
    if constexpr (K > 1) {
      const uint64_t ahead = MARKS ? start_bits(a.starts, b, t0 - (K - 1), L) : 0;
#pragma unroll
      for (int k = 0; k + 1 < K; ++k) {
        const int t = t0 - (K - 1) + k;
        if (MARKS && (ahead >> k & 1)) {
          clear<K, 2>(win);
          age = K - 2 - k;
        }
        if (t >= 0 && t < len)
          load2((const T *)a.x.p + b * a.x.sb + t * a.x.st + c, win[k]);
        else if (t < 0 && a.state0)
          load2((const T *)a.state0 + (b * (K - 1) + t + (K - 1)) * a.D + c, win[k]);
      }
    }
    T *dx = (T *)a.dx + (b * L + t0 - (K - 1)) * a.D + c;
    Raw2<T> rx[kRows], ry[kRows], nx[kRows], ny[kRows];
    auto load = [&](int m0) {  // the last row again behind it
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const uint32_t m = m0 + r < rows ? m0 + r : rows - 1;
        nx[r].load(bx, lane_bytes, m * xstep);
        ny[r].load(by, lane_bytes, m * ystep);
      }
    };
    load(0);
    for (int m0 = 0; m0 < nrow && m0 - (K - 1) < rows; m0 += kRows) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) rx[r] = nx[r], ry[r] = ny[r];
      if (m0 + kRows < nrow) load(m0 + kRows);  // on its way while these rows are walked over
      const uint32_t firsts = MARKS ? (uint32_t)((m0 < 64 ? first >> m0 : first2 >> (m0 - 64)) & ((1 << kRows) - 1)) : 0;
      // EDGE: a document starts among these steps or just before, or the row ends
      auto walk = [&](auto edge) {
        constexpr bool EDGE = decltype(edge)::v;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const int m = m0 + r, t = t0 + m - (K - 1);
          if constexpr (EDGE && MARKS && K > 1) {
            age = age + 1 < K - 1 ? age + 1 : K - 1;
            if (firsts >> r & 1) {
              clear<K, 2>(win);
              age = 0;
            }
          }
          float g[2];
          rx[r].get(win[K - 1]);
          ry[r].get(g);
          if (a.silu)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float z = bias[j];
#pragma unroll
              for (int k = 0; k < K; ++k) z = fmaf(w[k][j], win[k][j], z);
              const float s = sigmoid_f(z);
              g[j] *= fmaf(s, fmaf(-z, s, z), s);  // silu' = s + s z (1 - s)
            }
          if (EDGE && t0 + m >= len) win[K - 1][0] = win[K - 1][1] = g[0] = g[1] = 0.0f;
#pragma unroll
          for (int k = K - 1; k > 0; --k) d[k][0] = d[k - 1][0], d[k][1] = d[k - 1][1];
          d[0][0] = w[K - 1][0] * g[0], d[0][1] = w[K - 1][1] * g[1];
#pragma unroll
          for (int k = 1; k < K; ++k)
            if (!EDGE || k <= age)
#pragma unroll
              for (int j = 0; j < 2; ++j) d[k][j] = fmaf(w[K - 1 - k][j], g[j], d[k][j]);
          // (a step behind the row's length has no part in the sums, not even 0 times an unused state that is not finite)
          if (m < own && !(EDGE && t0 + m >= len))
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
              for (int k = 0; k < K; ++k) dw[k][j] = fmaf(g[j], win[k][j], dw[k][j]);
              dw[K][j] += g[j];
            }
          if constexpr (EDGE)
            if (K > 1 && a.dstate_final && t >= len - (K - 1) && t < len && (m >= K - 1 || t < 0)) {  // an input of the last state
              bool kept = true;
              if (MARKS && a.starts)
                for (int u = t < 0 ? 0 : t + 1; u < len; ++u) kept = kept && !a.starts[b * L + u];
              if (kept) {
                float f[2];
                load2((const T *)a.dstate_final + (b * (K - 1) + t - len + (K - 1)) * a.D + c, f);
                d[K - 1][0] += f[0], d[K - 1][1] += f[1];
              }
            }
          if (m >= K - 1) {
            if (on && (!EDGE || t < L)) store2(dx + m * a.D, d[K - 1]);
          } else if (K > 1 && t < 0 && a.dstate0) {
            if (on) store2((T *)a.dstate0 + (b * (K - 1) + t + (K - 1)) * a.D + c, d[K - 1]);
          }
          shift<K, 2>(win);
        }
      };
      if ((MARKS && K > 1 && (age < K - 1 || firsts)) || t0 + m0 + kRows > len)
        walk(Int<1>{});
      else
        walk(Int<0>{});
    }
  }
#pragma unroll
  for (int k = 0; k <= K; ++k) sums[wave][2 * k][lane] = dw[k][0], sums[wave][2 * k + 1][lane] = dw[k][1];
  __syncthreads();
  part += (int64_t)run * a.D * (K + 1);
  for (int i = threadIdx.x; i < N * 64; i += 256) {
    const int q = i >> 6, l = i & 63, k = q >> 1;
    const int64_t ch = (ct * 64 + l) * 2 + (q & 1);
    if (ch >= D) continue;
    const float v = (sums[0][q][l] + sums[1][q][l]) + (sums[2][q][l] + sums[3][q][l]);
    part[k == K ? (int64_t)D * K + ch : ch * K + k] = v;
  }
}

template <typename T, int K>
__global__ void __launch_bounds__(256) conv_update_kernel(ConvArgs a) {
  const uint32_t n4 = (uint32_t)(a.D / 4), i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.B * n4) return;
  const int64_t b = i / n4, c = i % n4 * 4;
  T *state = (T *)a.state + b * (K - 1) * a.D + c;
  float w[K][4], bias[4], win[K][4], v[4];
#pragma unroll
  for (int k = 0; k + 1 < K; ++k) load_vec(state + k * a.D, win[k]);
  load_vec((const T *)a.x.p + b * a.x.sb + c, win[K - 1]);
  load_weights<K>(a, c, w, bias);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = bias[j];
#pragma unroll
    for (int k = 0; k < K; ++k) v[j] = fmaf(w[k][j], win[k][j], v[j]);
    if (a.silu) v[j] = silu_f(v[j]);
  }
  store_vec((T *)a.y + b * a.D + c, v);
#pragma unroll
  for (int k = 0; k + 1 < K; ++k) store_vec(state + k * a.D, win[k + 1]);
}

template <typename F>
hipError_t by_width(int width, F f) {
  return width == 1 ? f(Int<1>{}) : width == 2 ? f(Int<2>{}) : width == 3 ? f(Int<3>{}) : f(Int<4>{});
}

constexpr int kFwdSteps = 32;

template <typename T>
hipError_t fwd(const ConvArgs &a, hipStream_t s) {
  const int64_t nchunk = (a.L + kFwdSteps - 1) / kFwdSteps, n4 = a.D / 4, main = a.B * nchunk * n4;
  const int64_t threads = main + (a.state_final ? a.B * n4 : 0);
  return by_width(a.width, [&](auto k) {
    hipLaunchKernelGGL((conv_fwd_kernel<T, decltype(k)::v>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, a, (uint32_t)nchunk, kFwdSteps, (uint32_t)main);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t bwd(const ConvArgs &a, hipStream_t s) {
  const BwdPlan p = bwd_plan(a.B, a.L, a.D, a.width, sizeof(T));
  const hipError_t e = by_width(a.width, [&](auto k) {
    constexpr int K = decltype(k)::v;
    const dim3 grid((unsigned)(p.ctiles * p.nruns));
    if (a.starts || a.lengths)
      hipLaunchKernelGGL((conv_bwd_kernel<T, K, true>), grid, dim3(256), 0, s, a, p.nrow, (int)p.nchunk, (int)p.ctiles, (int)p.nruns, (float *)a.workspace);
    else
      hipLaunchKernelGGL((conv_bwd_kernel<T, K, false>), grid, dim3(256), 0, s, a, p.nrow, (int)p.nchunk, (int)p.ctiles, (int)p.nruns, (float *)a.workspace);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  return launch_sum_rows((const float *)a.workspace, p.nruns, a.D * (a.width + 1), a.D * a.width, a.dweight, a.dbias, s);
}

template <typename T>
hipError_t update(const ConvArgs &a, hipStream_t s) {
  return by_width(a.width, [&](auto k) {
    hipLaunchKernelGGL((conv_update_kernel<T, decltype(k)::v>), dim3((unsigned)((a.B * (a.D / 4) + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace

int64_t conv_bwd_workspace_bytes(int64_t B, int64_t L, int64_t D, int width) {
  const int64_t a = bwd_plan(B, L, D, width, 2).nruns, b = bwd_plan(B, L, D, width, 4).nruns;
  return (a > b ? a : b) * D * (width + 1) * 4;
}

hipError_t launch_conv_fwd(const ConvArgs &a, int io_dtype, hipStream_t s) { return io_dtype == 0 ? fwd<float>(a, s) : fwd<bf16>(a, s); }
hipError_t launch_conv_bwd(const ConvArgs &a, int io_dtype, hipStream_t s) { return io_dtype == 0 ? bwd<float>(a, s) : bwd<bf16>(a, s); }
hipError_t launch_conv_update(const ConvArgs &a, int io_dtype, hipStream_t s) { return io_dtype == 0 ? update<float>(a, s) : update<bf16>(a, s); }

}  // namespace ssm
