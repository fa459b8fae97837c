// head_norm.hip -- the RMS norm of every head of queries and keys and the
// rotation of its elements by position, in one pass, and its gradients.
//
// A group of TPR lanes owns one head: 8 elements per lane in two pieces of 4, so
// that both elements of a rotated pair are in one lane (pieces p and p + rotary / 8
// where pairs are half a rotation apart, 8 adjacent elements where they are
// interleaved).  A workgroup takes up to 256 / TPR heads, all heads of as many
// tokens as fit, over a run of tokens; it stays with its heads, so that their
// weights are in registers, and so are the sums for the weights' gradients.  The
// cosines and sines of a few tokens are formed once per workgroup, into LDS, while
// the tokens' rows are on their way.
//
// Bound by HBM.  Measured, per call, bf16 (a large copy moves 5.1 TB/s): forward 1 x
// 32768, 40 and 8 heads of 128 (806 MB) 161 us, 5.0 TB/s; backward 8 x 2048, 16 and 16
// heads of 128 (403 MB) 80 us with 4 for the second kernel, 5.0 TB/s; the same in fp32 85 and
// 130 us (537 and 805 MB; outputs stay in the last-level cache).  Heads of 64 (8 x 2048, 32
// and 4: 151 and 227 MB) 39 and 56 us, 3.9 and 4.0 TB/s: blocks of 8 heads form the angles five times.  Heads of
// 80 and 160, which leave 6 of 16 and 12 of 32 lanes idle (8 x 2048, 16 and 16): 50 and 100 us forward, 72 and 141
// backward, 3.4 to 3.6 TB/s.  Single tokens, 40 and 8 heads of 128: 3.4 us for one, 8.4 for 256 (6 MB in 96
// workgroups), since a group of lanes takes its rows one after the other however few there are.  The forward
// runs six waves per SIMD (with five the first takes 7% longer).
#include "mixer_device.hpp"
#include "mixer_kernels.hpp"

namespace ssm {

using namespace heads;

namespace {

// cos and sin of 2 pi turns, |turns| <= 1/2: to the nearest quarter, then the
// series of an angle up to pi / 4; what they leave out is below 2^-28.
__device__ __forceinline__ float2 cos_sin(double turns) {
  const double q = rint(4.0 * turns);
  const float x = (float)((turns - 0.25 * q) * 6.283185307179586), x2 = x * x;
  const float s = x * fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), 1.0f);
  const float c = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
  const int n = (int)q & 3;
  const float u = n & 1 ? s : c, v = n & 1 ? c : s;
  return make_float2(n == 1 || n == 2 ? -u : u, n >= 2 ? -v : v);
}

// A lane's two pieces of a head as they lie in memory; the elements one[i], two[i]
// are a pair.
template <typename T>
struct Pieces {
  typename Vec4<T>::raw lo, hi;
  __device__ __forceinline__ void load(const T *p, int o1, int o2) { lo = Vec4<T>::load(p, o1), hi = Vec4<T>::load(p, o2); }
  template <bool ONCE>
  __device__ __forceinline__ void load_row(const T *p, int o1, int o2) {
    using R = typename Vec4<T>::raw;
    if constexpr (ONCE)
      lo = load_once((const R *)(p + o1)), hi = load_once((const R *)(p + o2));
    else
      load(p, o1, o2);
  }
  template <bool INTER>
  __device__ __forceinline__ void get(float (&one)[4], float (&two)[4]) const {
    const float4 a = Vec4<T>::cvt(lo), b = Vec4<T>::cvt(hi);
    const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) one[i] = x[INTER ? 2 * i : i], two[i] = x[INTER ? 2 * i + 1 : 4 + i];
  }
};
template <bool INTER>
__device__ __forceinline__ void split(const float (&one)[4], const float (&two)[4], float (&lo)[4], float (&hi)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = INTER ? (i & 1 ? two[i / 2] : one[i / 2]) : one[i];
    hi[i] = INTER ? (i & 1 ? two[2 + i / 2] : one[2 + i / 2]) : two[i];
  }
}

template <int TPR>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int d = TPR / 2; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// One thread's angles of a chunk of tokens: one frequency, every `step`-th token.
struct Angles {
  int p, tok, step;
  double turns;  // per position
  __device__ __forceinline__ explicit Angles(const HeadNormArgs &a) {
    const int half = a.rot / 2;
    step = half ? kThreads / half : 0;
    p = half ? threadIdx.x % half : 0, tok = half ? threadIdx.x / half : 0;
    if (tok >= step) step = 0;  // (threads left over, or nothing to rotate)
    turns = step ? a.inv_freq[p] * 0.15915494309189535 : 0.0;
  }
  // cosines and sines of tokens t0 .. t0 + n of a batch row
  __device__ __forceinline__ void fill(const HeadNormArgs &a, int64_t b, int64_t t0, int n, float2 *table) const {
    if (step == 0) return;
    for (int t = tok; t < n; t += step) {
      const double x = (double)a.pos[b * a.pos_b + t0 + t] * turns;
      table[t * (a.rot / 2) + p] = cos_sin(x - rint(x));
    }
  }
};

template <typename T, int TPR, bool BWD, bool INTER>
__global__ void __launch_bounds__(kThreads, BWD ? 1 : 6) head_norm_kernel(HeadNormArgs a, Plan plan, float *part) {
  __shared__ alignas(16) float2 table[kMaxTable];
  const int half = a.rot / 2, HT = a.Hq + a.Hk;
  const int blk = (int)(blockIdx.x % plan.nblk), grp = threadIdx.x / TPR, p = threadIdx.x % TPR;
  const int64_t run = blockIdx.x / plan.nblk;
  const int hl = grp % plan.hb, sub = grp / plan.hb, h = blk * plan.hb + hl;
  const bool mine = sub < plan.tsub && h < HT, on = mine && p < a.d / 8;
  const bool is_q = h < a.Hq, rotated = p < a.rot / 8;
  const int hh = is_q ? h : h - a.Hq, nh = is_q ? a.Hq : a.Hk;
  const HeadView &src = is_q ? a.q : a.k, &up = is_q ? a.dq_out : a.dk_out;
  T *dst = (T *)(BWD ? (is_q ? a.dq : a.dk) : (is_q ? a.q_out : a.k_out));
  // where the lane's two pieces begin
  const int o1 = rotated && !INTER ? 4 * p : 8 * p, o2 = rotated && !INTER ? 4 * p + half : 8 * p + 4;
  float w1[4], w2[4], acc1[4], acc2[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w1[i] = w2[i] = 1.0f, acc1[i] = acc2[i] = 0.0f;
  const float *wp = is_q ? a.wq : a.wk;
  if (on && wp) {
    Pieces<float> w;
    w.load(wp + hh * a.w_h, o1, o2);
    w.template get<INTER>(w1, w2);
  }
  // Rows past the caches' order where a piece's loads are whole 128-byte lines, and not in
  // the bf16 forward: 8 x 2048, 16 and 16 heads of 128, fp32 forward 104 -> 85 us, backward 161 ->
  // 135, bf16 88 -> 81; heads of 64 fp32 backward 102 -> 86.  Elsewhere it loses: heads of 64 bf16 41 -> 45 and
  // 63 -> 67, the forward of heads of 128 in bf16 of which 32 are rotated 53 -> 59, of 64 in fp32 60 -> 67.
  constexpr bool ONCE = sizeof(T) == 4 ? TPR >= (BWD ? 8 : 16) : BWD && TPR >= 16;
  const float over_d = 1.0f / (float)a.d;
  const Angles angles(a);
  const int tt = plan.tsub * plan.rows;  // tokens of a chunk
  const int64_t row_chunks = (a.L + tt - 1) / tt;
  for (int64_t ch = run; ch < plan.nchunk; ch += plan.nruns) {
    const int64_t b = ch / row_chunks, t0 = ch % row_chunks * tt;
    const int n = (int)(a.L - t0 < tt ? a.L - t0 : tt);
    const T *xp = (const T *)src.p + b * src.sb + (t0 + sub) * src.st + hh * src.sh;
    const T *gp = BWD ? (const T *)up.p + b * up.sb + (t0 + sub) * up.st + hh * up.sh : nullptr;
    T *out = dst + ((b * a.L + t0 + sub) * nh + hh) * a.d;
    // a row is loaded while the one before it is worked on, the first while the angles are
    Pieces<T> next, next_g;
    const int mine_n = on ? n : 0;
    if (sub < mine_n) {
      next.template load_row<ONCE>(xp, o1, o2);
      if (BWD) next_g.template load_row<ONCE>(gp, o1, o2);
    }
    __syncthreads();  // the table's last readers are done
    angles.fill(a, b, t0, n, table);
    __syncthreads();
    for (int tok = sub; mine && tok < n; tok += plan.tsub) {
      float one[4] = {}, two[4] = {}, g1[4] = {}, g2[4] = {};
      if (on) {
        next.template get<INTER>(one, two);
        if (BWD) next_g.template get<INTER>(g1, g2);
      }
      if (tok + plan.tsub < mine_n) {
        xp += plan.tsub * src.st;
        next.template load_row<ONCE>(xp, o1, o2);
        if (BWD) {
          gp += plan.tsub * up.st;
          next_g.template load_row<ONCE>(gp, o1, o2);
        }
      }
      float rstd = 1.0f;
      if (a.norm) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fmaf(one[i], one[i], fmaf(two[i], two[i], ss));
        rstd = rsqrtf(head_sum<TPR>(ss) * over_d + a.eps);
      }
      float2 cs[4];
      if (rotated)
#pragma unroll
        for (int i = 0; i < 4; ++i) cs[i] = table[tok * half + 4 * p + i];
      if constexpr (!BWD) {
#pragma unroll
        for (int i = 0; i < 4; ++i) one[i] *= rstd * w1[i], two[i] *= rstd * w2[i];
        if (rotated)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float n1 = one[i], n2 = two[i];
            one[i] = fmaf(n1, cs[i].x, -n2 * cs[i].y);
            two[i] = fmaf(n2, cs[i].x, n1 * cs[i].y);
          }
      } else {
        // u = the gradient of n, turned back; with hat = x rstd: dx = rstd (u w - hat mean(u w hat))
        float s = 0.0f;
        if (rotated)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u1 = fmaf(g1[i], cs[i].x, g2[i] * cs[i].y), u2 = fmaf(g2[i], cs[i].x, -g1[i] * cs[i].y);
            g1[i] = u1, g2[i] = u2;
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          one[i] *= rstd, two[i] *= rstd;
          acc1[i] = fmaf(g1[i], one[i], acc1[i]), acc2[i] = fmaf(g2[i], two[i], acc2[i]);
          g1[i] *= w1[i], g2[i] *= w2[i];
          s = fmaf(g1[i], one[i], fmaf(g2[i], two[i], s));
        }
        if (a.norm) {
          s = head_sum<TPR>(s) * over_d;
#pragma unroll
          for (int i = 0; i < 4; ++i) one[i] = rstd * fmaf(-one[i], s, g1[i]), two[i] = rstd * fmaf(-two[i], s, g2[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) one[i] = g1[i], two[i] = g2[i];
        }
      }
      if (on) {
        float lo[4], hi[4];
        split<INTER>(one, two, lo, hi);
        store_vec(out + o1, lo);
        store_vec(out + o2, hi);
      }
      out += (int64_t)plan.tsub * nh * a.d;
    }
  }
  if constexpr (BWD) {
    if (!a.dwq) return;
    // sums over the workgroup's groups, in their order: for a head's own weight
    // over its tokens at once, for a shared one over the heads too (rows: one per
    // workgroup, columns: q's elements, then k's)
    float *lds = (float *)table;
    static_assert(sizeof(table) >= kThreads * 8 * sizeof(float), "the sums fit where the angles were");
    __syncthreads();
    float lo[4], hi[4];
    split<INTER>(acc1, acc2, lo, hi);
    if (on) {
#pragma unroll
      for (int i = 0; i < 4; ++i) lds[grp * a.d + o1 + i] = lo[i], lds[grp * a.d + o2 + i] = hi[i];
    }
    __syncthreads();
    if (a.w_h) {
      for (int i = threadIdx.x; i < plan.hb * a.d; i += kThreads) {
        const int head = blk * plan.hb + i / a.d;
        if (head >= HT) break;
        float v = lds[i];
        for (int k = 1; k < plan.tsub; ++k) v += lds[k * plan.hb * a.d + i];
        part[(run * HT + head) * a.d + i % a.d] = v;
      }
    } else {
      for (int i = threadIdx.x; i < 2 * a.d; i += kThreads) {
        float v = 0.0f;
        for (int k = 0; k < plan.hb * plan.tsub; ++k) {
          const int head = blk * plan.hb + k % plan.hb;
          if (head < HT && (head < a.Hq) == (i < a.d)) v += lds[k * a.d + i % a.d];
        }
        part[(int64_t)blockIdx.x * 2 * a.d + i] = v;
      }
    }
  }
}

// Batch rows that follow each other evenly are one row; so are rows of one token.
HeadNormArgs merged(HeadNormArgs a, bool bwd) {
  auto even = [&](const HeadView &v) { return a.L == 1 || v.sb == v.st * a.L; };
  const bool all = even(a.q) && (a.Hk == 0 || even(a.k)) && (!bwd || (even(a.dq_out) && (a.Hk == 0 || even(a.dk_out))));
  if (a.B == 1 || !all || (a.pos && a.pos_b != a.L)) return a;
  if (a.L == 1) a.q.st = a.q.sb, a.k.st = a.k.sb, a.dq_out.st = a.dq_out.sb, a.dk_out.st = a.dk_out.sb;
  a.L *= a.B, a.B = 1;
  return a;
}

template <typename T, int TPR, bool BWD>
void launch_tpr(const HeadNormArgs &a, const Plan &p, hipStream_t s) {
  const dim3 grid((unsigned)(p.nblk * p.nruns));
  if (a.interleaved)
    hipLaunchKernelGGL((head_norm_kernel<T, TPR, BWD, true>), grid, dim3(kThreads), 0, s, a, p, (float *)a.workspace);
  else
    hipLaunchKernelGGL((head_norm_kernel<T, TPR, BWD, false>), grid, dim3(kThreads), 0, s, a, p, (float *)a.workspace);
}

template <typename T, bool BWD>
hipError_t launch(const HeadNormArgs &given, hipStream_t s) {
  const HeadNormArgs a = merged(given, BWD);
  const Plan p = plan_of(a.B, a.L, a.Hq + a.Hk, a.d, a.rot, BWD, sizeof(T));
  const float *part = (const float *)a.workspace;
  if (p.tpr == 4)
    launch_tpr<T, 4, BWD>(a, p, s);
  else if (p.tpr == 8)
    launch_tpr<T, 8, BWD>(a, p, s);
  else if (p.tpr == 16)
    launch_tpr<T, 16, BWD>(a, p, s);
  else
    launch_tpr<T, 32, BWD>(a, p, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !BWD || !a.dwq) return e;
  return a.w_h ? launch_sum_rows(part, p.nruns, (int64_t)(a.Hq + a.Hk) * a.d, (int64_t)a.Hq * a.d, a.dwq, a.dwk, s)
               : launch_sum_rows(part, p.nruns * p.nblk, 2 * a.d, a.d, a.dwq, a.dwk, s);
}

}  // namespace

int64_t head_norm_bwd_workspace_bytes(int64_t B, int64_t L, int64_t Hq, int64_t Hk, int64_t d) { return bwd_workspace_bytes(B, L, Hq, Hk, d); }

hipError_t launch_head_norm_fwd(const HeadNormArgs &a, int io_dtype, hipStream_t s) { return io_dtype == 0 ? launch<float, false>(a, s) : launch<bf16, false>(a, s); }
hipError_t launch_head_norm_bwd(const HeadNormArgs &a, int io_dtype, hipStream_t s) { return io_dtype == 0 ? launch<float, true>(a, s) : launch<bf16, true>(a, s); }

}  // namespace ssm
