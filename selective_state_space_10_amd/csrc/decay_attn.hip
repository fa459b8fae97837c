// decay_attn.hip -- host side of the decay attention (roles, segments,
// workspace) and the small kernels that finish its gradients.
#include "decay_attn.hpp"

namespace ssm {

namespace {

constexpr int64_t kAlign = 256;

struct Carve {
  char *p;
  int64_t used = 0;
  template <typename T>
  T *take(int64_t count) {
    T *r = p ? (T *)(p + used) : nullptr;
    used += (count * (int64_t)sizeof(T) + kAlign - 1) / kAlign * kAlign;
    return r;
  }
};

int padded(int64_t d) { return d <= 32 ? 32 : d <= 64 ? 64 : d <= 128 ? 128 : 256; }

// How a call splits the sequence: nseg segments of seg_len steps.
struct Split {
  int nseg;
  int64_t seg_len;
};

Split split_of(int64_t L) { return {1, L}; }

struct FwdPlanDa {
  Split sp;
  int64_t nslice, tile;
};

}  // namespace

// The decays' gradient from the dot products of the main pass:
//   dg_t = sum_{r >= t in the segment} (q_r . dq_r - k_r . dk_r) + <exp(g) S, R> at the segment's end,
// where S and R are the states that both directions carry over that boundary:
// what crosses t is the products of pairs around t, and starting the sum at
// every segment's end keeps rounding from adding up over the sequence.  (The
// dot products leave out pairs with no decay between, decay_attn.hpp.)  One
// workgroup per segment; the running sum is fp64.
struct DaDecayGrad {
  const float *dots_q, *dots_k;   // (parts, BH, L)
  const float *edge_q, *edge_k;   // NULL = no boundary terms
  const float *g;
  int64_t g_b, g_t, L, seg_len, edge_size;
  int H, BH, nseg, parts, last_edge;
  float *out;       // (B, L, H), or NULL
  float *sums;      // (BH, nseg) sums over the segment, or NULL
};

__global__ void __launch_bounds__(256) decay_grad_kernel(DaDecayGrad a) {
  __shared__ double wsum[4];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int bh = blockIdx.x / a.nseg, seg = blockIdx.x % a.nseg;
  const int h = bh % a.H;
  const int64_t b = bh / a.H;
  const int64_t t0 = seg * a.seg_len, t1 = min(a.L, t0 + a.seg_len);
  const float *pg = a.g + b * a.g_b + h;
  auto block_sum = [&](double v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
    __syncthreads();
    if (lane == 0) wsum[w] = v;
    __syncthreads();
    return wsum[0] + wsum[1] + wsum[2] + wsum[3];
  };
  double carry = 0.0;
  if (a.edge_q && (seg + 1 < a.nseg || a.last_edge)) {
    const int64_t o = ((int64_t)bh * (a.nseg + 1) + seg + 1) * a.edge_size;
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < a.edge_size; i += 256) v += (double)a.edge_q[o + i] * a.edge_k[o + i];
    carry = block_sum(v);
    if (t1 < a.L) carry *= fast_exp2(decay_log2(pg[t1 * a.g_t]));
  }
  double total = 0.0;
  // from the last step to the first, 256 at a time
  for (int64_t hi = t1; hi > t0; hi -= 256) {
    const int64_t t = hi - 1 - threadIdx.x;
    double v = 0.0;
    if (t >= t0)
      for (int p = 0; p < a.parts; ++p) {
        const int64_t o = ((int64_t)p * a.BH + bh) * a.L + t;
        v += (double)a.dots_q[o] - (double)a.dots_k[o];
      }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double o = __shfl_up(v, d, 64);
      if (lane >= d) v += o;
    }
    __syncthreads();
    if (lane == 63) wsum[w] = v;
    __syncthreads();
    for (int i = 0; i < w; ++i) v += wsum[i];
    v += carry;
    carry += wsum[0] + wsum[1] + wsum[2] + wsum[3];
    if (t >= t0) {
      // a cleared state passes nothing on (what the sums leave there is rounding)
      if (pg[t * a.g_t] < kMinLog2Decay * kLn2) v = 0.0;
      total += v;
      if (a.out) a.out[(b * a.L + t) * a.H + h] = (float)v;
    }
  }
  if (a.sums) {
    total = block_sum(total);
    if (threadIdx.x == 0) a.sums[blockIdx.x] = (float)total;
  }
}

// One decay per head: the sum over batch rows and segments.
__global__ void __launch_bounds__(64) decay_grad_heads_kernel(const float *sums, int B, int H, int nseg, float *out) {
  const int h = blockIdx.x * 64 + threadIdx.x;
  if (h >= H) return;
  double v = 0.0;
  for (int b = 0; b < B; ++b)
    for (int s = 0; s < nseg; ++s) v += sums[((int64_t)b * H + h) * nseg + s];
  out[h] = (float)v;
}

// Gradients of shared heads: (rows, G, share, d) fp32 -> (rows, G, d), summed in order.
template <typename T>
__global__ void __launch_bounds__(256) shared_heads_kernel(const float *part, int64_t n4, int d4, int share, T *out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  const int64_t rg = i / d4, x = i % d4;
  const float4 *p = (const float4 *)part + rg * share * d4 + x;
  float4 v = p[0];
  for (int s = 1; s < share; ++s) {
    const float4 q = p[(int64_t)s * d4];
    v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
  }
  Vec4<T>::store(out, i * 4, v);
}

namespace {

hipError_t launch_kernel(const DaArgs &a, int io_dtype, bool precise, bool state_only, hipStream_t s) {
  return io_dtype == 0 ? launch_decay_attn_f32(a, padded(a.da), precise, state_only, s)
                       : launch_decay_attn_bf16(a, padded(a.da), precise, state_only, s);
}

DaArgs base_args(const DecayAttnArgs &a, int64_t da, int64_t dc, Split sp) {
  DaArgs r{};
  r.L = a.L, r.da = da, r.dc = dc, r.g = a.g, r.g_b = a.g_b, r.g_t = a.g_t;
  r.H = (int)a.H, r.BH = (int)(a.B * a.H), r.nseg = sp.nseg, r.seg_len = sp.seg_len;
  r.nslice = (int)((dc + kDaCols - 1) / kDaCols);
  return r;
}

int64_t edge_size(int64_t da, int64_t dc) { return (int64_t)padded(da) * kDaCols * ((dc + kDaCols - 1) / kDaCols); }

void take_segments(Carve &c, DaRole &r, const DaArgs &a) {
  if (a.nseg == 1) return;
  r.loc = c.take<float>((int64_t)a.BH * a.nseg * edge_size(a.da, a.dc));
  r.tot = c.take<float>((int64_t)a.BH * a.nseg);
}

DaArgs fwd_args(const DecayAttnArgs &a, Carve &c) {
  DaArgs r = base_args(a, a.dk, a.dv, split_of(a.L));
  r.nroles = 1;
  DaRole &o = r.role[0];
  o.a = a.q, o.b = a.k, o.c = a.v;
  o.out = a.o;
  o.pscale = o.iscale = a.scale, o.sscale = 1.0f;
  o.state_in = a.state0, o.state_out = a.state_final;
  take_segments(c, o, r);
  return r;
}

struct BwdSet {
  DaArgs qk, v;          // dq and dk (state dv x dk), dv (state dk x dv)
  float *dq_part, *dk_part, *sums;
  bool want_g, edges;
};

BwdSet bwd_args(const DecayAttnArgs &a, bool want_g, Carve &c) {
  BwdSet r{};
  const Split sp = split_of(a.L);
  r.want_g = want_g;
  r.qk = base_args(a, a.dv, a.dk, sp), r.v = base_args(a, a.dk, a.dv, sp);
  r.qk.nroles = 2, r.v.nroles = 1;
  DaRole &q = r.qk.role[0], &k = r.qk.role[1], &v = r.v.role[0];
  q.a = a.dout, q.b = a.v, q.c = a.k, q.e = a.q;
  k.a = a.v, k.b = a.dout, k.c = a.q, k.e = a.k;
  v.a = a.k, v.b = a.q, v.c = a.dout;
  q.pscale = q.iscale = a.scale, q.sscale = 1.0f;
  for (DaRole *x : {&k, &v}) x->pscale = a.scale, x->iscale = 1.0f, x->sscale = a.scale, x->reverse = 1, x->state_in = a.dstate_final;
  q.state_in = a.state0, q.state_in_t = 1, k.state_in_t = 1;
  v.state_out = a.dstate0;
  q.out = a.dq, k.out = a.dk_out, v.out = a.dv_out;
  take_segments(c, q, r.qk), take_segments(c, k, r.qk), take_segments(c, v, r.v);
  if (a.G < a.H) {
    const int64_t n = a.B * a.L * a.H * a.dk;
    q.out = r.dq_part = c.take<float>(n), k.out = r.dk_part = c.take<float>(n);
    q.out_f32 = k.out_f32 = 1;
  }
  if (want_g) {
    const int64_t n = a.B * a.H * a.L * r.qk.nslice * kDaWaves;
    q.dots = c.take<float>(n), k.dots = c.take<float>(n);
    // taken whether dstate_final is given or not: the workspace's size goes by the shape
    const int64_t m = a.B * a.H * (sp.nseg + 1) * edge_size(a.dv, a.dk);
    float *eq = c.take<float>(m), *ek = c.take<float>(m);
    r.edges = sp.nseg > 1 || a.dstate_final;
    if (r.edges) q.edge = eq, k.edge = ek;
    r.sums = c.take<float>(a.B * a.H * sp.nseg);
  }
  return r;
}

}  // namespace

int64_t decay_attn_fwd_workspace_bytes(const DecayAttnArgs &a, int) {
  Carve c{nullptr};
  fwd_args(a, c);
  return c.used;
}

int64_t decay_attn_bwd_workspace_bytes(const DecayAttnArgs &a, int) {
  Carve c{nullptr};
  bwd_args(a, true, c);
  return c.used;
}

hipError_t launch_decay_attn_fwd(const DecayAttnArgs &a, int io_dtype, hipStream_t s) {
  Carve c{(char *)a.workspace};
  const DaArgs r = fwd_args(a, c);
  if (r.nseg > 1) {
    const hipError_t e = launch_kernel(r, io_dtype, false, true, s);
    if (e != hipSuccess) return e;
  }
  return launch_kernel(r, io_dtype, false, false, s);
}

hipError_t launch_decay_attn_bwd(const DecayAttnArgs &a, int io_dtype, hipStream_t s) {
  Carve c{(char *)a.workspace};
  const BwdSet r = bwd_args(a, a.dlog_decay != nullptr, c);
  hipError_t e;
  if (r.qk.nseg > 1) {
    if ((e = launch_kernel(r.qk, io_dtype, false, true, s)) != hipSuccess) return e;
    if ((e = launch_kernel(r.v, io_dtype, false, true, s)) != hipSuccess) return e;
  }
  if ((e = launch_kernel(r.qk, io_dtype, r.want_g, false, s)) != hipSuccess) return e;
  if ((e = launch_kernel(r.v, io_dtype, false, false, s)) != hipSuccess) return e;
  if (r.want_g) {
    DaDecayGrad d{};
    d.dots_q = r.qk.role[0].dots, d.dots_k = r.qk.role[1].dots;
    d.edge_q = r.qk.role[0].edge, d.edge_k = r.qk.role[1].edge;
    d.g = a.g, d.g_b = a.g_b, d.g_t = a.g_t, d.L = a.L, d.seg_len = r.qk.seg_len, d.edge_size = edge_size(a.dv, a.dk);
    d.H = (int)a.H, d.BH = (int)(a.B * a.H), d.nseg = r.qk.nseg, d.parts = r.qk.nslice * kDaWaves, d.last_edge = a.dstate_final != nullptr;
    const bool heads = a.g_t == 0;
    d.out = heads ? nullptr : a.dlog_decay, d.sums = heads ? r.sums : nullptr;
    hipLaunchKernelGGL(decay_grad_kernel, dim3((unsigned)(d.BH * d.nseg)), dim3(256), 0, s, d);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (heads) {
      hipLaunchKernelGGL(decay_grad_heads_kernel, dim3((unsigned)((a.H + 63) / 64)), dim3(64), 0, s, r.sums, (int)a.B, (int)a.H, d.nseg, a.dlog_decay);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  if (r.dq_part) {
    const int64_t n4 = a.B * a.L * a.G * a.dk / 4;
    const dim3 grid((unsigned)((n4 + 255) / 256));
    for (int i = 0; i < 2; ++i) {
      const float *p = i ? r.dk_part : r.dq_part;
      void *o = i ? a.dk_out : a.dq;
      if (io_dtype == 0)
        hipLaunchKernelGGL(shared_heads_kernel<float>, grid, dim3(256), 0, s, p, n4, (int)(a.dk / 4), (int)(a.H / a.G), (float *)o);
      else
        hipLaunchKernelGGL(shared_heads_kernel<bf16>, grid, dim3(256), 0, s, p, n4, (int)(a.dk / 4), (int)(a.H / a.G), (bf16 *)o);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace ssm
