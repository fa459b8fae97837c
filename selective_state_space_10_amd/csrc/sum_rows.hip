// sum_rows.hip -- the sums over rows of partial sums that end the backward passes of the
// gated recurrence, the causal convolution and the norm of heads: a workgroup takes
// 16 columns, 64 lanes' worth of rows each in turn, all in a fixed order.  A launch
// of its own takes about 4 us, latency for the most part (128 rows x 2048 and 60 rows x 10240).
#include "mixer_kernels.hpp"

namespace ssm {

namespace {

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
