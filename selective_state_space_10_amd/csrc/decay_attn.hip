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

int cols_of(int64_t dc) { return da_waves(dc) * 16; }
int64_t slices_of(int64_t dc) { return (dc + cols_of(dc) - 1) / cols_of(dc); }

int64_t compute_units() {
  static const int n = [] {
    int dev = 0, v = 0;
    if (hipGetDevice(&dev) != hipSuccess || hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v < 1) v = 256;
    return v;
  }();
  return n;
}

// Into how many segments a sequence is split: the estimate below is least.
// Workgroups run `slots` to a CU (as LDS and registers hold them); a CU takes
// about chunk_us for a chunk of all of them, and 0.3 more of it for a round
// that is not full.  A first pass costs 0.4 of a main pass of its segments and a
// launch, combining another, folding what the last segment reads.  Measured,
// forward and backward, in us of GPU time (* the split taken):
//   segments                              1           2 to 6             more
//   8 x 2048, 16 heads of 128, bf16       165, 617    2: 130, 387        8: 143, 475
//                                                     4*: 120, 379
//   1 x 32768, 40 heads of 128, bf16      2522, 9735  6: 642, 2314       12*: 574, 2116  32: 598, 2184  64: 656, 2348
//   3 x 1111, 8 heads of 72 x 96, fp32    169, 576    6: 54, 154         9*: 43, 129     18: 53, 156
//   2 x 1537, 32 heads of 64, fp32        148, 554    4: 71, 215         9*: 53, 161     13: 56, 185
//   1 x 512, 8 heads of 64, bf16          33, 120     4: 17, 51          8*: 13.1, 40.6
//   1 x 512, 32 heads of 64, bf16         33, 122     4: 17.4, 52        8*: 14.0, 42.9
constexpr int64_t kMinSegment = 64;
// From how many segments on the states before them are computed once, by a
// kernel of its own, and not by every workgroup from the end states before it:
// earlier for wider states, and backward in time, where dv folds transposed
// states and there are more passes to one combining.  Folded and combined, us:
//   wider of dk, dv           forward                                backward
//   64 (1 x 2048, 16 heads)   16: 28.6, 34.5   32: 29.3, 34.8        8: 137, 135   11: 119, 111
//      (2 x 1537, 32 heads)   13: 55.5, 58.5   25: 65.3, 61.8        9: 162, 168   13: 191, 185
//   128 (3 x 1111, 8 heads)   9: 42.5, 46.5    18: 53.4, 52.9        6: 153.6, 153.7   9: 129.6, 128.0
//      (2 x 1500, 16 heads)   12: 32.2, 35.8   24: 42.8, 42.1        6: 108, 109   8: 95.6, 94.6
//      (1 x 16384, 4 heads)   16: 128, 128     24: 98, 94            6: 881, 876   9: 617, 603
//   256 (1 x 1500, 4 heads)   8: 78.7, 81.3    12: 63.3, 61.3        4: 391, 374   5: 345, 318
//      (2 x 2048, 8 heads)    8: 67.8, 74.6    16: 98.8, 101         5: 259, 261   8: 214, 216
// (64: fp32; 128: fp32, bf16 with dv 64, bf16; 256: fp32, bf16.)
int combine_from(int64_t dk, int64_t dv, bool backward) {
  const int wide = padded(dk > dv ? dk : dv);
  return wide <= 64 ? (backward ? 10 : 24) : wide == 128 ? (backward ? 8 : 20) : (backward ? 5 : 12);
}
Split split_of(int64_t L, int64_t bh, int64_t da, int64_t dc, int es, int combine) {
  const bool wide = da_waves(dc) == 8;
  const int64_t cus = compute_units(), wgs = bh * slices_of(dc), chunk = es == 2 ? 64 : 32;
  const int64_t slots = padded(da) > 128 ? 1 : es == 4 && padded(da) == 128 ? (wide ? 1 : 2) : wide ? 2 : 3;
  const double chunk_us = wide ? 10.0 : 6.0, launch_us = 5.0;
  // a segment's states go out and in about four times, at 5 TB/s
  const double tile = padded(da) * cols_of(dc) * 4, state_us = 4.0 * tile / 5e6;
  auto rounds = [&](int64_t n) {
    const int64_t q = (n + cus - 1) / cus;
    return (double)q / slots + (q % slots ? 0.3 : 0.0);
  };
  Split best{1, L};
  double least = 0.0;
  for (int64_t n = 1; n <= 128 && n <= (L + kMinSegment - 1) / kMinSegment; ++n) {
    const int64_t len = n == 1 ? L : ((L + n - 1) / n + 63) / 64 * 64, segs = (L + len - 1) / len;
    if (segs != n) continue;
    const double chunks = (double)((len + chunk - 1) / chunk);
    double us = rounds(wgs * n) * chunks * chunk_us;
    if (n > 1) us += 0.4 * rounds(wgs * (n - 1)) * chunks * chunk_us + launch_us;
    if (n >= combine)
      us += launch_us;
    else
      us += (n - 1) * tile / 2e5;  // a workgroup folds at most that many, at 0.2 TB/s
    if (n > 1) us += n * wgs * state_us;
    if (n == 1 || us < least) best = {(int)n, len}, least = us;
  }
  return best;
}

}  // namespace

// The decays' gradient from the dot products of the main passes:
//   dg_t = sum_{r >= t up to the next edge} (q_r . dq_r - k_r . dk_r) + <exp(g) S, R> at that edge,
// where S and R are the states that both directions carry over it: what crosses
// t is the products of pairs around t.  (The dot products leave out pairs with
// no decay between, decay_attn.hpp.)  The edge before t gives it as well,
//   dg_t = <exp(g) S, R> there - sum_{r < t from there on} (q_r . dq_r - k_r . dk_r),
// and the two are averaged with weights linear in t: the rounding of the dot
// products, which adds up with the distance from an edge, is then zero at both
// ends of a block, and in a sum over its steps a dot product counts at most half
// the block (from one edge: all of it).
// One workgroup per block between edges; the running sum is fp64.  A few MB and chains
// of dependent sums: latency (7 to 9 us for 8 x 2048 steps of 16 heads, 1024
// workgroups; 2% of the backward).
struct DaDecayGrad {
  const float *dots_q, *dots_k;   // (slices, BH, L)
  const float *edge_dot;          // (parts, BH, nblock)
  const float *g;
  int64_t g_b, g_t, L;
  int H, BH, nblock, edge_len, last_edge, state0, slices, parts;
  float *out;       // (B, L, H), or NULL
  float *sums;      // (BH, nblock) sums over the steps before an edge, or NULL
};

__global__ void __launch_bounds__(256) decay_grad_kernel(DaDecayGrad a) {
  __shared__ double wsum[4];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int bh = blockIdx.x / a.nblock, blk = blockIdx.x % a.nblock;
  const int h = bh % a.H;
  const int64_t b = bh / a.H;
  const int64_t t0 = (int64_t)blk * a.edge_len, t1 = min(a.L, t0 + a.edge_len);
  const float *pg = a.g + b * a.g_b + h;
  auto at_edge = [&](int i) {
    double v = 0.0;
    for (int p = 0; p < a.parts; ++p) v += a.edge_dot[((int64_t)p * a.BH + bh) * a.nblock + i];
    return v;
  };
  auto dots = [&](int64_t t) {
    double v = 0.0;
    for (int p = 0; p < a.slices; ++p) {
      const int64_t o = ((int64_t)p * a.BH + bh) * a.L + t;
      v += (double)a.dots_q[o] - (double)a.dots_k[o];
    }
    return v;
  };
  double carry = blk + 1 < a.nblock || a.last_edge ? at_edge(blk) : 0.0;
  // what the edge before the block gives more than the one after it: 0 but for
  // rounding, and not known at a given first state
  double more = 0.0;
  if (blk > 0 || !a.state0) {
    for (int64_t t = t0 + threadIdx.x; t < t1; t += 256) more -= dots(t);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) more += __shfl_xor(more, d, 64);
    if (lane == 0) wsum[w] = more;
    __syncthreads();
    more = wsum[0] + wsum[1] + wsum[2] + wsum[3] - carry;
    if (blk > 0) more += at_edge(blk - 1);
    if (!(fabs(more) < INFINITY)) more = 0.0;  // a NaN or an infinity before a step is no reason for one at it
    __syncthreads();
  }
  const double slope = more / (double)(t1 - t0);
  double total = 0.0;
  // from the last step to the first, 256 at a time
  for (int64_t hi = t1; hi > t0; hi -= 256) {
    const int64_t t = hi - 1 - threadIdx.x;
    double v = t >= t0 ? dots(t) : 0.0;
    v = wave_sum_scan(v);
    __syncthreads();
    if (lane == 63) wsum[w] = v;
    __syncthreads();
    for (int i = 0; i < w; ++i) v += wsum[i];
    v += carry + (t1 - t) * slope;
    carry += wsum[0] + wsum[1] + wsum[2] + wsum[3];
    if (t >= t0) {
      // a cleared state passes nothing on (what the sums leave there is rounding)
      if (pg[t * a.g_t] < kMinLog2Decay * kLn2) v = 0.0;
      total += v;
      if (a.out) a.out[(b * a.L + t) * a.H + h] = (float)v;
    }
  }
  if (a.sums) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) total += __shfl_xor(total, d, 64);
    __syncthreads();
    if (lane == 0) wsum[w] = total;
    __syncthreads();
    if (threadIdx.x == 0) a.sums[blockIdx.x] = (float)(wsum[0] + wsum[1] + wsum[2] + wsum[3]);
  }
}

// The states before every segment from the end states of the ones before it
// (in place): one thread per 4 elements, in the order of the recurrence, 8
// segments' loads under way (10 us for 32 segments of 16 heads of 64 x 64, fp32, in
// two roles, 16 MB in and 17 out: latency of the chain).
__global__ void __launch_bounds__(256) combine_kernel(DaArgs a, int da_padded, int cols) {
  const DaRole &R = a.role[blockIdx.y];
  const int64_t tile4 = (int64_t)da_padded * cols / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= tile4 * a.nslice * a.BH) return;
  const int64_t bh = i / (tile4 * a.nslice), x = i % (tile4 * a.nslice);
  f32x4 cur = {0, 0, 0, 0};
  if (R.state_in) {
    // element of the tile as decay_attn_kernel lays it out: waves, row tiles, lanes
    const int slice = (int)(x / tile4), y = (int)(x % tile4), lane = y & 63, dt = (y >> 6) % (da_padded / 16), w = (y >> 6) / (da_padded / 16);
    const int row = dt * 16 + (lane >> 4) * 4, col = slice * cols + w * 16 + (lane & 15), da = (int)a.da, dc = (int)a.dc;
    const float *s = R.state_in + bh * da * dc;
    for (int r = 0; r < 4; ++r)
      if (row + r < da && col < dc) cur[r] = s[R.state_in_t ? col * da + row + r : (row + r) * dc + col];
  }
  const int64_t step = tile4 * a.nslice;
  f32x4 *p = (f32x4 *)R.loc + bh * a.nseg * step + x;
  const float2 *tot = R.tot + bh * a.nseg;
  const int first = R.reverse ? a.nseg - 1 : 0, dir = R.reverse ? -1 : 1;
  int j = 0;
  constexpr int U = 8;  // loads under way
  for (; j + U < a.nseg; j += U) {
    f32x4 l[U];
    float2 e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) l[u] = p[(first + dir * (j + u)) * step], e[u] = tot[first + dir * (j + u)];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      p[(first + dir * (j + u)) * step] = cur;
      cur = cur * e[u].x * e[u].y + l[u];
    }
  }
  for (; j < a.nseg; ++j) {
    f32x4 l = cur;
    float2 e = make_float2(0.0f, 0.0f);
    if (j + 1 < a.nseg) l = p[(first + dir * j) * step], e = tot[first + dir * j];
    p[(first + dir * j) * step] = cur;
    cur = cur * e.x * e.y + l;
  }
}

// One decay per head: the sum over batch rows and steps.
__global__ void __launch_bounds__(64) decay_grad_heads_kernel(const float *sums, int B, int H, int nblock, float *out) {
  const int h = blockIdx.x * 64 + threadIdx.x;
  if (h >= H) return;
  double v = 0.0;
  for (int b = 0; b < B; ++b)
    for (int s = 0; s < nblock; ++s) v += sums[((int64_t)b * H + h) * nblock + s];
  out[h] = (float)v;
}

// Gradients of shared heads, dq (blockIdx.y 0) and dk: (rows, G, share, d) fp32
// -> (rows, G, d), summed in order.  Bound by HBM and caches (57 MB in 9 us at 3074
// rows, 4 x 8 heads of 64).
template <typename T>
__global__ void __launch_bounds__(256) shared_heads_kernel(const float *part, const float *part2, int64_t n4, int d4, int share, T *out, T *out2) {
  if (blockIdx.y) part = part2, out = out2;
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

hipError_t launch_kernel(const DaArgs &a, int io_dtype, bool dots, bool state_only, hipStream_t s) {
  return io_dtype == 0 ? launch_decay_attn_f32(a, padded(a.da), dots, state_only, s)
                       : launch_decay_attn_bf16(a, padded(a.da), dots, state_only, s);
}

// The states before all segments (or what they are folded from) of a set of roles.
hipError_t launch_first_pass(const DaArgs &a, int io_dtype, hipStream_t s) {
  if (a.nseg == 1) return hipSuccess;
  hipError_t e = launch_kernel(a, io_dtype, false, true, s);
  if (e == hipSuccess && a.combined) {
    const int64_t n = (int64_t)padded(a.da) * cols_of(a.dc) / 4 * a.nslice * a.BH;
    hipLaunchKernelGGL(combine_kernel, dim3((unsigned)((n + 255) / 256), a.nroles), dim3(256), 0, s, a, padded(a.da), cols_of(a.dc));
    e = hipGetLastError();
  }
  return e;
}

DaArgs base_args(const DecayAttnArgs &a, int64_t da, int64_t dc, Split sp, int combine) {
  DaArgs r{};
  r.combined = sp.nseg >= combine;
  r.L = a.L, r.da = da, r.dc = dc, r.g = a.g, r.g_b = a.g_b, r.g_t = a.g_t;
  r.nroles = 1;
  r.H = (int)a.H, r.BH = (int)(a.B * a.H), r.nseg = sp.nseg, r.seg_len = sp.seg_len;
  r.nslice = (int)slices_of(dc);
  return r;
}

int64_t edge_size(int64_t da, int64_t dc) { return padded(da) * cols_of(dc) * slices_of(dc); }

void take_segments(Carve &c, DaRole &r, const DaArgs &a) {
  if (a.nseg == 1) return;
  r.loc = c.take<float>((int64_t)a.BH * a.nseg * edge_size(a.da, a.dc));
  r.tot = c.take<float2>((int64_t)a.BH * a.nseg);
}

DaArgs fwd_args(const DecayAttnArgs &a, int io_dtype, Carve &c) {
  const int combine = combine_from(a.dk, a.dv, false);
  DaArgs r = base_args(a, a.dk, a.dv, split_of(a.L, a.B * a.H, a.dk, a.dv, io_dtype == 0 ? 4 : 2, combine), combine);
  DaRole &o = r.role[0];
  o.a = a.q, o.b = a.k, o.c = a.v;
  o.out = a.o;
  o.pscale = o.iscale = a.scale, o.sscale = 1.0f;
  o.state_in = a.state0, o.state_out = a.state_final;
  take_segments(c, o, r);
  return r;
}

// Steps between two edges: the shortest power of two for which writing and
// reading the states there (8 bytes per element) stays within an eighth of the
// bytes that the three passes read and write per step (8 rows of each kind), or a
// quarter for decays by head: in their gradient's sum over the steps a rounding
// counts as often as there are steps to its edge.
int edge_len_of(const DecayAttnArgs &a, int es, bool heads) {
  const int64_t state = 8 * padded(a.dv) * cols_of(a.dk) * slices_of(a.dk), step = es * (a.dk + a.dv);
  int e = 64;
  while (e < 1024 && state > (int64_t)e * step * (heads ? 2 : 1)) e *= 2;
  return e;
}

struct BwdSet {
  DaArgs q, k, v;        // dq and dk: state dv x dk; dv: state dk x dv
  float *dq_part, *dk_part, *sums;
  bool want_g;
};

BwdSet bwd_args(const DecayAttnArgs &a, int io_dtype, bool want_g, Carve &c) {
  BwdSet r{};
  const int edge_len = edge_len_of(a, io_dtype == 0 ? 4 : 2, a.g_t == 0);
  r.want_g = want_g;
  const int combine = combine_from(a.dk, a.dv, true);
  const Split sp = split_of(a.L, a.B * a.H, a.dv, a.dk, io_dtype == 0 ? 4 : 2, combine);
  r.q = r.k = base_args(a, a.dv, a.dk, sp, combine), r.v = base_args(a, a.dk, a.dv, sp, combine);
  DaRole &q = r.q.role[0], &k = r.k.role[0], &v = r.v.role[0];
  q.a = a.dout, q.b = a.v, q.c = a.k, q.e = a.q;
  k.a = a.v, k.b = a.dout, k.c = a.q, k.e = a.k;
  v.a = a.k, v.b = a.q, v.c = a.dout;
  q.pscale = q.iscale = a.scale, q.sscale = 1.0f;
  for (DaRole *x : {&k, &v}) x->pscale = a.scale, x->iscale = 1.0f, x->sscale = a.scale, x->reverse = 1, x->state_in = a.dstate_final;
  q.state_in = a.state0, q.state_in_t = 1, k.state_in_t = 1;
  v.state_out = a.dstate0;
  q.out = a.dq, k.out = a.dk_out, v.out = a.dv_out;
  take_segments(c, q, r.q), take_segments(c, k, r.k);
  if (r.k.nseg > 1) v.loc = k.loc, v.tot = k.tot, v.loc_t = 1, v.cols_t = cols_of(a.dk), v.nslice_t = (int)slices_of(a.dk), r.v.dc_t = padded(a.dv);
  if (a.G < a.H) {
    const int64_t n = a.B * a.L * a.H * a.dk;
    q.out = r.dq_part = c.take<float>(n), k.out = r.dk_part = c.take<float>(n);
    q.out_f32 = k.out_f32 = 1;
  }
  if (want_g) {
    const int64_t n = a.B * a.H * a.L * r.q.nslice;
    q.dots = c.take<float>(n), k.dots = c.take<float>(n);
    const int inner = (int)((a.L - 1) / edge_len);
    // the size goes by the shape: an edge after the last step whether dstate_final is given or not, as many as decays by head have
    const int64_t room = (a.L - 1) / edge_len_of(a, io_dtype == 0 ? 4 : 2, true) + 1;
    r.q.edge_shift = r.k.edge_shift = __builtin_ctz(edge_len);
    r.q.nedge = r.k.nedge = inner + 1, r.q.last_edge = r.k.last_edge = a.dstate_final != nullptr;
    q.edge = k.edge = c.take<float>(a.B * a.H * room * edge_size(a.dv, a.dk));
    q.edge_dot = c.take<float>(a.B * a.H * room * r.q.nslice * da_waves(a.dk));
    r.sums = c.take<float>(a.B * a.H * room);
  }
  return r;
}

}  // namespace

int64_t decay_attn_fwd_workspace_bytes(const DecayAttnArgs &a, int io_dtype) {
  Carve c{nullptr};
  fwd_args(a, io_dtype, c);
  return c.used;
}

int64_t decay_attn_bwd_workspace_bytes(const DecayAttnArgs &a, int io_dtype) {
  Carve c{nullptr};
  bwd_args(a, io_dtype, true, c);
  return c.used;
}

hipError_t launch_decay_attn_fwd(const DecayAttnArgs &a, int io_dtype, hipStream_t s) {
  Carve c{(char *)a.workspace};
  const DaArgs r = fwd_args(a, io_dtype, c);
  const hipError_t e = launch_first_pass(r, io_dtype, s);
  return e == hipSuccess ? launch_kernel(r, io_dtype, false, false, s) : e;
}

hipError_t launch_decay_attn_bwd(const DecayAttnArgs &a, int io_dtype, hipStream_t s) {
  Carve c{(char *)a.workspace};
  const BwdSet r = bwd_args(a, io_dtype, a.dlog_decay != nullptr, c);
  hipError_t e;
  // dk and dq have states of one shape: one first pass for both; dv's is dk's, transposed
  DaArgs first = r.k;
  first.nroles = 2, first.role[1] = r.q.role[0];
  if ((e = launch_first_pass(first, io_dtype, s)) != hipSuccess) return e;
  // backward in time before forward: it writes the states that the latter dots at edges
  for (const DaArgs *p : {&r.k, &r.v, &r.q})
    if ((e = launch_kernel(*p, io_dtype, r.want_g && p != &r.v, false, s)) != hipSuccess) return e;
  if (r.want_g) {
    DaDecayGrad d{};
    d.dots_q = r.q.role[0].dots, d.dots_k = r.k.role[0].dots, d.edge_dot = r.q.role[0].edge_dot;
    d.g = a.g, d.g_b = a.g_b, d.g_t = a.g_t, d.L = a.L;
    d.H = (int)a.H, d.BH = (int)(a.B * a.H), d.edge_len = 1 << r.q.edge_shift;
    d.nblock = r.q.nedge, d.last_edge = r.q.last_edge, d.state0 = a.state0 != nullptr;
    d.slices = r.q.nslice, d.parts = r.q.nslice * da_waves(a.dk);
    const bool heads = a.g_t == 0;
    d.out = heads ? nullptr : a.dlog_decay, d.sums = heads ? r.sums : nullptr;
    hipLaunchKernelGGL(decay_grad_kernel, dim3((unsigned)(d.BH * d.nblock)), dim3(256), 0, s, d);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (heads) {
      hipLaunchKernelGGL(decay_grad_heads_kernel, dim3((unsigned)((a.H + 63) / 64)), dim3(64), 0, s, r.sums, (int)a.B, (int)a.H, d.nblock, a.dlog_decay);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  if (r.dq_part) {
    const int64_t n4 = a.B * a.L * a.G * a.dk / 4;
    const dim3 grid((unsigned)((n4 + 255) / 256), 2);
    if (io_dtype == 0)
      hipLaunchKernelGGL(shared_heads_kernel<float>, grid, dim3(256), 0, s, r.dq_part, r.dk_part, n4, (int)(a.dk / 4), (int)(a.H / a.G), (float *)a.dq, (float *)a.dk_out);
    else
      hipLaunchKernelGGL(shared_heads_kernel<bf16>, grid, dim3(256), 0, s, r.dq_part, r.dk_part, n4, (int)(a.dk / 4), (int)(a.H / a.G), (bf16 *)a.dq, (bf16 *)a.dk_out);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace ssm
