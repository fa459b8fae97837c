// decay_update.hip -- one token of the decay attention: S <- exp(g) S + k v^T,
// o = scale S^T q, with S (B, H, dk, dv) fp32 updated in place.  The state is
// streamed once in and once out with 16-byte accesses and everything else is
// small, so the kernel is bound by HBM: 256 requests of 40 heads of 128 x 128
// (1.35 GB) take 264 us, 5.1 TB/s, where a large copy reaches 5.0; of 128 x 64 143 us
// (4.7 TB/s), of 128 x 32 67 us (from caches, 5.1).  Columns are taken 128 at a time: of 128
// x 8, 62 us (1.5 TB/s, 30 of 32 lanes idle), of 128 x 136, 381 us (3.8 TB/s).  One
// request of 16 heads takes 7 us, which is latency.
//
// Mapping: a workgroup owns a slab of columns of one (batch row, head); LPR
// lanes cover a row of the slab, 4 columns each, and the other lanes and the
// four waves take further rows.  A lane's columns are the same in every row,
// so o is a sum in registers, then over lanes and waves.
#include "block_kernels.hpp"
#include "device_common.hpp"

namespace ssm {

template <typename T, int LPR>
__global__ void __launch_bounds__(256) decay_update_kernel(DecayUpdateArgs a, int nslab) {
  constexpr int RPP = 256 / LPR;  // rows per pass
  constexpr int U = 4;            // passes in flight
  __shared__ float qs[256], ks[256];
  __shared__ float4 part[4][LPR];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t bh = blockIdx.x / nslab;
  const int slab = blockIdx.x % nslab;
  const int64_t b = bh / a.H, h = bh % a.H;
  const int dk = (int)a.dk, dv = (int)a.dv;
  const int col = (slab * LPR + tid % LPR) * 4;
  const int row0 = tid / LPR;
  if (tid < dk) {
    qs[tid] = load_io((const T *)a.q.p, b * a.q.sb + (h / a.q.share) * a.q.sh + tid);
    ks[tid] = load_io((const T *)a.k.p, b * a.k.sb + (h / a.k.share) * a.k.sh + tid);
  }
  const bool on = col < dv;
  float4 v = make_float4(0, 0, 0, 0), o = v;
  if (on) v = Vec4<T>::cvt(Vec4<T>::load((const T *)a.v.p + b * a.v.sb + h * a.v.sh, col));
  const float e = fast_exp2(a.g[b * a.g_b + h] * kLog2e);
  float *s = a.state + bh * dk * dv + col;
  __syncthreads();
  for (int r0 = row0; r0 < dk; r0 += RPP * U) {
    float4 x[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (on && r0 + i * RPP < dk) x[i] = *(const float4 *)(s + (int64_t)(r0 + i * RPP) * dv);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int r = r0 + i * RPP;
      if (on && r < dk) {
        const float k = ks[r], q = qs[r];
        x[i].x = fmaf(e, x[i].x, k * v.x), x[i].y = fmaf(e, x[i].y, k * v.y);
        x[i].z = fmaf(e, x[i].z, k * v.z), x[i].w = fmaf(e, x[i].w, k * v.w);
        *(float4 *)(s + (int64_t)r * dv) = x[i];
        o.x = fmaf(q, x[i].x, o.x), o.y = fmaf(q, x[i].y, o.y);
        o.z = fmaf(q, x[i].z, o.z), o.w = fmaf(q, x[i].w, o.w);
      }
    }
  }
#pragma unroll
  for (int d = LPR; d < 64; d <<= 1) {
    o.x += __shfl_xor(o.x, d, 64), o.y += __shfl_xor(o.y, d, 64);
    o.z += __shfl_xor(o.z, d, 64), o.w += __shfl_xor(o.w, d, 64);
  }
  if (lane < LPR) part[w][lane] = o;
  __syncthreads();
  if (tid < LPR && on) {
    float4 r = part[0][tid];
    for (int i = 1; i < 4; ++i) r.x += part[i][tid].x, r.y += part[i][tid].y, r.z += part[i][tid].z, r.w += part[i][tid].w;
    r.x *= a.scale, r.y *= a.scale, r.z *= a.scale, r.w *= a.scale;
    Vec4<T>::store((T *)a.o, bh * dv + col, r);
  }
}

template <typename T>
static hipError_t launch_update_t(const DecayUpdateArgs &a, hipStream_t s) {
  const int64_t bh = a.B * a.H;
  constexpr int LPR = 32;
  const int nslab = (int)((a.dv + 4 * LPR - 1) / (4 * LPR));
  hipLaunchKernelGGL((decay_update_kernel<T, LPR>), dim3((unsigned)(bh * nslab)), dim3(256), 0, s, a, nslab);
  return hipGetLastError();
}

hipError_t launch_decay_update(const DecayUpdateArgs &a, int io_dtype, hipStream_t s) {
  return io_dtype == 0 ? launch_update_t<float>(a, s) : launch_update_t<bf16>(a, s);
}

}  // namespace ssm
