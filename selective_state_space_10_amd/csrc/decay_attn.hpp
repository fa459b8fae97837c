// decay_attn.hpp -- the kernel of linear attention with a decay for each head,
//   S_t = exp(g_t) S_{t-1} + b_t c_t^T,   out_t = S_t^T a_t,
// with a query-like a, a key-like b (dimension da) and a value-like c
// (dimension dc).  The forward takes (a, b, c) = (q, k, v).  Its gradients are
// the same recurrence on other operands: dq is (do, v, k) forward in time, dk
// is (v, do, q) and dv is (k, q, do) backward in time, where the decay between
// two steps is the one of the later step.
//
// Chunked form.  A workgroup owns one (batch row, head, slice of dc) and walks
// over chunks of C steps with S in registers.  With G_t the sum of g over the
// chunk's steps up to t,
//   out_t = exp(G_t) S^T a_t + sum_{s<=t} exp(G_t - G_s) (a_t . b_s) c_s,
//   S    <- exp(G_last) S + sum_s b_s (exp(G_last - G_s) c_s)^T,
// which are four matrix products.  Every exponent is a sum of decays over a
// range of steps, so nothing overflows where the recurrence does not; G is
// summed in 64 bits and kept as a pair of floats, so that differences of
// nearby steps stay exact to fp32 after steps of very strong decay.
#pragma once

#include "block_kernels.hpp"
#include "device_common.hpp"

namespace ssm {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) short s16x4;

// Decays below this many powers of two are zero in fp32 whatever they meet
// (smallest fp32 2^-149): -inf is held at it, so that sums of decays stay finite.
constexpr float kMinLog2Decay = -256.0f;
__device__ __forceinline__ float decay_log2(float g) {
  return g < kMinLog2Decay * kLn2 ? kMinLog2Decay : g * kLog2e;  // NaN passes
}

// One direction and set of operands of the recurrence.
struct DaRole {
  View4 a, b, c, e;      // e: what the outputs are dotted with (the decays' gradient)
  void *out;             // (B, L, H, dc)
  int out_f32;           // fp32 output (partial sums of shared heads)
  float pscale, iscale, sscale;  // on products inside a chunk, with the state, into the state
  int reverse;
  const float *state_in; // (B, H, da, dc), or (B, H, dc, da) if state_in_t; NULL = 0
  int state_in_t;
  float *state_out;      // (B, H, da, dc), NULL = not wanted
  float *dots;           // (slices * waves, B * H, L) partial sums of out . e, or NULL
  float *loc, *tot;      // segments: end states from zero, total decays
  float *edge;           // states at segment boundaries, (B * H, nseg + 1, slices, tile), or NULL;
                         // forward in time the last one without the last step's own term
};

struct DaArgs {
  int64_t L, da, dc;
  const float *g;
  int64_t g_b, g_t;
  int H, BH, nseg, nslice, nroles;
  int64_t seg_len;       // a multiple of the chunk
  DaRole role[3];
};

// Matrix fragments of 32 along the contracted dimension and 16 along the
// other: lane l holds, for row (or column) l % 16, the contracted indices
// 4 (l / 16) + r and 16 + 4 (l / 16) + r, r = 0..3.  This order makes the
// accumulators of a 16 x 16 product (row 4 (l / 16) + r, column l % 16) usable
// as the next product's operand without moving data between lanes.
template <typename T>
struct Mx;

template <>
struct Mx<bf16> {
  typedef uint4 Frag;
  static constexpr int kChunk = 64;
  static constexpr int kPad = 8;  // row padding in elements: rows start 4 banks apart
  // Rows along the contracted dimension are stored so that the 8 values of a
  // fragment are adjacent: 32-blocks as [l / 16][half][r].
  static __device__ __forceinline__ int pos(int k) { return (k & ~31) | ((k & 12) << 1) | ((k & 16) >> 2) | (k & 3); }
  static __device__ __forceinline__ Frag rowfrag(const bf16 *m, int stride, int row0, int k0) {
    const int l = threadIdx.x & 63;
    return *(const uint4 *)(m + (row0 + (l & 15)) * stride + k0 + (l >> 4) * 8);
  }
  // transposed: contracted along rows; cols are col0 .. col0 + 15, given as the
  // storage offset of each group of four (off(j), j = l % 4)
  static __device__ __forceinline__ uint2 tr4(const bf16 *p) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p)));
  }
  static __device__ __forceinline__ Frag colfrag(const bf16 *m, int stride, int row0, int off) {
    const int l = threadIdx.x & 63;
    const bf16 *p = m + (row0 + (l >> 4) * 4 + ((l >> 2) & 3)) * stride + off;
    const uint2 x = tr4(p), y = tr4(p + 16 * stride);
    return make_uint4(x.x, x.y, y.x, y.y);
  }
  static __device__ __forceinline__ int coloff_perm(int ct) {  // columns 16 ct .. of a permuted row
    const int j = threadIdx.x & 3;
    return (ct >> 1) * 32 + j * 8 + (ct & 1) * 4;
  }
  static __device__ __forceinline__ int coloff(int col0) { return col0 + (threadIdx.x & 3) * 4; }
  static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ void floats(Frag f, float (&x)[8]) {
    const uint32_t w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  static __device__ __forceinline__ uint32_t pack_rne(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
  }
  // fp32 values as a sum of N bf16 pieces: one piece is rounded to nearest;
  // of more, each takes the next 8 significant bits (three pieces hold all 24
  // bits of an fp32 value, two leave a relative error below 2^-15).
  template <int N>
  static __device__ __forceinline__ void split2(float a, float b, uint32_t (&o)[N]) {
    if constexpr (N == 1) {
      o[0] = pack_rne(a, b);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        o[i] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
        a -= __uint_as_float(__float_as_uint(a) & 0xffff0000u);
        b -= __uint_as_float(__float_as_uint(b) & 0xffff0000u);
      }
    }
  }
  template <int N>
  static __device__ __forceinline__ void split(const float (&x)[8], Frag (&o)[N]) {
    uint32_t w[4][N];
#pragma unroll
    for (int i = 0; i < 4; ++i) split2<N>(x[2 * i], x[2 * i + 1], w[i]);
#pragma unroll
    for (int n = 0; n < N; ++n) o[n] = make_uint4(w[0][n], w[1][n], w[2][n], w[3][n]);
  }
  // four values along the contracted dimension, in N pieces `plane` elements apart
  template <int N>
  static __device__ __forceinline__ void put4(bf16 *p, int plane, const float (&x)[4]) {
    uint32_t a[N], b[N];
    split2<N>(x[0], x[1], a);
    split2<N>(x[2], x[3], b);
#pragma unroll
    for (int n = 0; n < N; ++n) *(uint2 *)(p + n * plane) = make_uint2(a[n], b[n]);
  }
  // 16 bytes of a row (elements k .. k + 7) into permuted order
  static __device__ __forceinline__ void put_perm(bf16 *row, int k, uint4 v) {
    const int o = pos(k);
    *(uint2 *)(row + o) = make_uint2(v.x, v.y);
    *(uint2 *)(row + o + 8) = make_uint2(v.z, v.w);
  }
  static __device__ __forceinline__ bool nonfinite(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
    return bad;
  }
};

template <>
struct Mx<float> {
  struct Frag {
    f32x4 a, b;
  };
  static constexpr int kChunk = 32;
  static constexpr int kPad = 4;
  static __device__ __forceinline__ int pos(int k) { return k; }
  static __device__ __forceinline__ Frag rowfrag(const float *m, int stride, int row0, int k0) {
    const int l = threadIdx.x & 63;
    const float *p = m + (row0 + (l & 15)) * stride + k0 + (l >> 4) * 4;
    return Frag{*(const f32x4 *)p, *(const f32x4 *)(p + 16)};
  }
  static __device__ __forceinline__ Frag colfrag(const float *m, int stride, int row0, int off) {
    const int l = threadIdx.x & 63;
    const float *p = m + (row0 + (l >> 4) * 4) * stride + off;
    Frag f;
#pragma unroll
    for (int r = 0; r < 4; ++r) f.a[r] = p[r * stride], f.b[r] = p[(16 + r) * stride];
    return f;
  }
  static __device__ __forceinline__ int coloff_perm(int ct) { return ct * 16 + (threadIdx.x & 15); }
  static __device__ __forceinline__ int coloff(int col0) { return col0 + (threadIdx.x & 15); }
  static __device__ __forceinline__ f32x4 mma(const Frag &a, const Frag &b, f32x4 c) {
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a[r], b.a[r], c, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b[r], b.b[r], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ void floats(const Frag &f, float (&x)[8]) {
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = f.a[r], x[4 + r] = f.b[r];
  }
  template <int N>
  static __device__ __forceinline__ void split(const float (&x)[8], Frag (&o)[N]) {
    static_assert(N == 1, "fp32 operands are whole");
#pragma unroll
    for (int r = 0; r < 4; ++r) o[0].a[r] = x[r], o[0].b[r] = x[4 + r];
  }
  template <int N>
  static __device__ __forceinline__ void put4(float *p, int, const float (&x)[4]) {
    static_assert(N == 1, "fp32 operands are whole");
    *(float4 *)p = make_float4(x[0], x[1], x[2], x[3]);
  }
  static __device__ __forceinline__ void put_perm(float *row, int k, uint4 v) { *(uint4 *)(row + k) = v; }
  static __device__ __forceinline__ bool nonfinite(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= (w[i] & 0x7f800000u) == 0x7f800000u;
    return bad;
  }
};

// A (ROWS, COLS) tile on its way from global memory to LDS, 16 bytes at a time.
template <typename T, int ROWS, int COLS, int NT>
struct TileRegs {
  static constexpr int EPP = 16 / (int)sizeof(T), PPR = COLS / EPP, N = (ROWS * PPR + NT - 1) / NT, RSTEP = NT / PPR;
  static_assert(PPR <= NT && NT % PPR == 0, "whole rows per step");
  uint4 r[N];
  // row0: first row's first element; rows, cols: how many there are (rows >= 1, cols >= 1)
  __device__ __forceinline__ void load(const T *row0, int64_t st, int rows, int cols) {
    const int row = threadIdx.x / PPR, col = (threadIdx.x % PPR) * EPP;
    const T *p = row0 + row * st + col;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool ok = row + i * RSTEP < rows && col < cols;
      r[i] = *(const uint4 *)(ok ? p + (int64_t)(i * RSTEP) * st : row0);
    }
  }
  // f(row, col, piece) for every piece of the tile, zeros outside rows x cols
  template <typename F>
  __device__ __forceinline__ void each(int rows, int cols, F f) const {
    const int row = threadIdx.x / PPR, col = (threadIdx.x % PPR) * EPP;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int rr = row + i * RSTEP;
      if (N * NT == ROWS * PPR || rr < ROWS) {
        const bool ok = rr < rows && col < cols;
        f(rr, col, ok ? r[i] : make_uint4(0, 0, 0, 0));
      }
    }
  }
};

template <typename T, int DA, int NW, int NC, int NP, bool STATE_ONLY>
struct DaLds {
  static constexpr int C = Mx<T>::kChunk, TV = NW * NC * 16;
  static constexpr int SA = DA + Mx<T>::kPad, SC = TV + Mx<T>::kPad, SP = C + Mx<T>::kPad;
  T a[STATE_ONLY ? 8 : C * SA];
  T b[C * SA];
  T c[C * SC];
  T p[STATE_ONLY ? 8 : NP * C * SP];
  float gh[C], gl[C], in[C], out[C], diag[C];
  float e;
  int bad[2];
};

// T: storage type; DA: da rounded up; NW waves of NC tiles of 16 columns of dc
// each; NP, NS: pieces of the products inside a chunk and of the state where
// they are operands.  STATE_ONLY: the end state of a segment from zero (a
// split sequence's first pass).
template <typename T, int DA, int NW, int NC, int NP, int NS, bool STATE_ONLY>
__global__ void __launch_bounds__(NW * 64) decay_attn_kernel(DaArgs args) {
  typedef Mx<T> M;
  typedef typename M::Frag Frag;
  typedef DaLds<T, DA, NW, NC, NP, STATE_ONLY> Lds;
  constexpr int C = M::kChunk, CT = C / 16, DT = DA / 16, NT = NW * 64, TV = Lds::TV;
  constexpr int SA = Lds::SA, SC = Lds::SC, SP = Lds::SP;
  constexpr int NB = sizeof(T) == 2 ? 3 : 1;  // pieces of c into the state: all of fp32
  __shared__ __attribute__((aligned(16))) Lds lds;

  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, l15 = lane & 15, lg = lane >> 4;
  // Workgroups go to the 8 XCDs in turn: give each XCD a contiguous run of
  // items, so that slices and roles that read the same rows share its L2.
  const int nitems = gridDim.x, xcd = blockIdx.x & 7, per = nitems >> 3, rem = nitems & 7;
  int item = xcd * per + min(xcd, rem) + (blockIdx.x >> 3);
  const int slice = item % args.nslice;
  item /= args.nslice;
  const DaRole &R = args.role[item % args.nroles];
  item /= args.nroles;
  const int segs = STATE_ONLY ? args.nseg - 1 : args.nseg;
  const bool rev = R.reverse != 0;
  const int seg = item % segs + (STATE_ONLY && rev ? 1 : 0);
  const int bh = item / segs;
  const int h = bh % args.H;
  const int64_t b = bh / args.H;
  const int col0 = slice * TV, wcol0 = col0 + w * NC * 16;
  const int64_t t0 = seg * args.seg_len;
  const int64_t n = min(args.seg_len, args.L - t0);
  const int64_t tfirst = rev ? t0 + n - 1 : t0;
  const int64_t dir = rev ? -1 : 1;
  const int da = (int)args.da, dc = (int)args.dc;

  const T *pa = (const T *)R.a.p + b * R.a.sb + (h / R.a.share) * R.a.sh + tfirst * R.a.st;
  const T *pb = (const T *)R.b.p + b * R.b.sb + (h / R.b.share) * R.b.sh + tfirst * R.b.st;
  const T *pc = (const T *)R.c.p + b * R.c.sb + (h / R.c.share) * R.c.sh + tfirst * R.c.st + col0;
  const float *pg = args.g + b * args.g_b + h;
  const int ccols = min(TV, dc - col0);

  // The state: S[dt][ct][r] is row dt * 16 + lg * 4 + r, column wcol0 + ct * 16 + l15.
  f32x4 S[DT][NC];
  constexpr int64_t kTile = (int64_t)DA * TV;
  const int64_t wtile = (int64_t)w * DT * NC * 256 + lane * 4;
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int ct = 0; ct < NC; ++ct) S[dt][ct] = f32x4{0, 0, 0, 0};
  if constexpr (!STATE_ONLY) {
    if (R.state_in) {
      const float *s = R.state_in + (int64_t)bh * da * dc;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int ct = 0; ct < NC; ++ct)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = dt * 16 + lg * 4 + r, col = wcol0 + ct * 16 + l15;
            if (row < da && col < dc) S[dt][ct][r] = s[R.state_in_t ? (int64_t)col * da + row : (int64_t)row * dc + col];
          }
    }
    // the segments before this one, in the order of the recurrence
    const int before = rev ? args.nseg - 1 - seg : seg;
    for (int i = 0; i < before; ++i) {
      const int64_t j = (int64_t)bh * args.nseg + (rev ? args.nseg - 1 - i : i);
      const float e = R.tot[j];
      const float *loc = R.loc + (j * args.nslice + slice) * kTile + wtile;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) S[dt][ct] = S[dt][ct] * e + *(const f32x4 *)(loc + (dt * NC + ct) * 256);
    }
    // boundary j lies between segments j - 1 and j
    if (R.edge && (rev || seg > 0)) {
      float *o = R.edge + (((int64_t)bh * (args.nseg + 1) + (rev ? seg + 1 : seg)) * args.nslice + slice) * kTile + wtile;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) *(f32x4 *)(o + (dt * NC + ct) * 256) = S[dt][ct];
    }
    // products of steps later in a chunk are never written: they stay zero
    for (int i = threadIdx.x; i < NP * C * SP * (int)sizeof(T) / 16; i += NT) ((uint4 *)lds.p)[i] = make_uint4(0, 0, 0, 0);
  }
  if (threadIdx.x < 2) lds.bad[threadIdx.x] = 0;

  TileRegs<T, C, DA, NT> ra, rb;
  TileRegs<T, C, TV, NT> rc;
  float rg = 0.0f;
  auto fetch = [&](int64_t u0) {
    const int rows = (int)min((int64_t)C, n - u0);
    if constexpr (!STATE_ONLY) ra.load(pa + dir * u0 * R.a.st, dir * R.a.st, rows, da);
    rb.load(pb + dir * u0 * R.b.st, dir * R.b.st, rows, da);
    rc.load(pc + dir * u0 * R.c.st, dir * R.c.st, rows, ccols);
    // backward in time the decay into a step is the later step's
    const int64_t t = tfirst + dir * (u0 + lane) + (rev ? 1 : 0);
    rg = lane < rows && t < args.L ? decay_log2(pg[t * args.g_t]) : 0.0f;
  };
  fetch(0);
  float total = 1.0f;

  for (int64_t u0 = 0; u0 < n; u0 += C) {
    const int rows = (int)min((int64_t)C, n - u0);
    const int par = (int)(u0 / C) & 1;
    __syncthreads();  // the last chunk's readers are done
    if constexpr (!STATE_ONLY)
      ra.each(rows, da, [&](int r, int k, uint4 v) { M::put_perm(lds.a + r * SA, k, v); });
    rb.each(rows, da, [&](int r, int k, uint4 v) { M::put_perm(lds.b + r * SA, k, v); });
    rc.each(rows, ccols, [&](int r, int k, uint4 v) {
      *(uint4 *)(lds.c + r * SC + k) = v;
      if (!STATE_ONLY && M::nonfinite(v)) lds.bad[par] = 1;
    });
    if (w == 0) {
      double G = rg;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_up(G, d, 64);
        if (lane >= d) G += o;
      }
      const double last = __shfl(G, 63, 64);
      const float hi = (float)G;
      // the last boundary's state leaves out the last step (see no_dot)
      const bool left_out = !STATE_ONLY && R.edge && !rev && t0 + u0 + lane == args.L - 1;
      if (lane < C) {
        lds.gh[lane] = hi;
        lds.gl[lane] = (float)(G - (double)hi);
        lds.in[lane] = fast_exp2(hi) * R.iscale;
        lds.out[lane] = left_out ? 0.0f : fast_exp2((float)(last - G)) * R.sscale;
      }
      if (lane == 0) lds.e = fast_exp2((float)last);
    }
    if (u0 + C < n) fetch(u0 + C);
    __syncthreads();
    const float e = lds.e;
    total *= e;

    f32x4 acc[CT][NC];
    if constexpr (!STATE_ONLY) {
      // products a_t . b_s of steps s <= t with their decays, 16 x 16 tiles over the waves
      for (int idx = w; idx < CT * (CT + 1) / 2; idx += NW) {
        const int tt = idx >= 6 ? 3 : idx >= 3 ? 2 : idx >= 1 ? 1 : 0, st = idx - tt * (tt + 1) / 2;
        f32x4 x = {0, 0, 0, 0};
#pragma unroll
        for (int kk = 0; kk < DA / 32; ++kk)
          x = M::mma(M::rowfrag(lds.b, SA, st * 16, kk * 32), M::rowfrag(lds.a, SA, tt * 16, kk * 32), x);
        const int t = tt * 16 + l15, s = st * 16 + lg * 4;
        const float th = lds.gh[t], tl = lds.gl[t];
        float p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float d = fast_exp2((th - lds.gh[s + r]) + (tl - lds.gl[s + r]));
          // for the dot products a step's own term is kept apart (below)
          p[r] = s + r < t + (R.dots ? 0 : 1) ? x[r] * (d * R.pscale) : 0.0f;
          if (s + r == t) lds.diag[t] = x[r] * R.pscale;
        }
        M::template put4<NP>(lds.p + t * SP + M::pos(s), C * SP, p);
      }
      // what the state gives
#pragma unroll
      for (int tt = 0; tt < CT; ++tt)
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) acc[tt][ct] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int kk = 0; kk < DA / 32; ++kk) {
        Frag sf[NC][NS];
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) {
          float x[8];
#pragma unroll
          for (int r = 0; r < 4; ++r) x[r] = S[2 * kk][ct][r], x[4 + r] = S[2 * kk + 1][ct][r];
          M::template split<NS>(x, sf[ct]);
        }
#pragma unroll
        for (int tt = 0; tt < CT; ++tt) {
          const Frag af = M::rowfrag(lds.a, SA, tt * 16, kk * 32);
#pragma unroll
          for (int ct = 0; ct < NC; ++ct)
#pragma unroll
            for (int i = NS - 1; i >= 0; --i) acc[tt][ct] = M::mma(sf[ct][i], af, acc[tt][ct]);
        }
      }
#pragma unroll
      for (int tt = 0; tt < CT; ++tt) {
        const float f = lds.in[tt * 16 + l15];
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) acc[tt][ct] *= f;
      }
    }
    Frag cf[C / 32][NC];
#pragma unroll
    for (int kk = 0; kk < C / 32; ++kk)
#pragma unroll
      for (int ct = 0; ct < NC; ++ct) cf[kk][ct] = M::colfrag(lds.c, SC, kk * 32, M::coloff((w * NC + ct) * 16));
    if constexpr (!STATE_ONLY) {
      __syncthreads();  // all products are there
      if (threadIdx.x == 0) lds.bad[par ^ 1] = 0;
      if (!lds.bad[par]) {
#pragma unroll
        for (int tt = 0; tt < CT; ++tt)
#pragma unroll
          for (int kk = 0; kk <= tt / 2; ++kk)
#pragma unroll
            for (int i = NP - 1; i >= 0; --i) {
              const Frag pf = M::rowfrag(lds.p + i * C * SP, SP, tt * 16, kk * 32);
#pragma unroll
              for (int ct = 0; ct < NC; ++ct) acc[tt][ct] = M::mma(cf[kk][ct], pf, acc[tt][ct]);
            }
      } else {
        // A NaN or infinity in c must not meet the zeros of later steps: sum over s <= t alone.
#pragma unroll
        for (int tt = 0; tt < CT; ++tt)
#pragma unroll
          for (int ct = 0; ct < NC; ++ct) {
            const int t = tt * 16 + l15;
            for (int s = 0; s <= t; ++s) {
              float p = 0.0f;
#pragma unroll
              for (int i = NP - 1; i >= 0; --i) p += load_io(lds.p + i * C * SP + t * SP, M::pos(s));
#pragma unroll
              for (int r = 0; r < 4; ++r)
                acc[tt][ct][r] = fmaf(p, load_io(lds.c + s * SC, (w * NC + ct) * 16 + lg * 4 + r), acc[tt][ct][r]);
            }
          }
      }
      // out^T: column wcol0 + ct * 16 + lg * 4 + r of step tt * 16 + l15
#pragma unroll
      for (int tt = 0; tt < CT; ++tt) {
        const int i = tt * 16 + l15;
        const int64_t t = tfirst + dir * (u0 + i);
        float dot = 0.0f;
        if (i < rows) {
          const int64_t o = ((b * args.L + t) * args.H + h) * dc;
          const T *pe = (const T *)R.e.p + b * R.e.sb + (h / R.e.share) * R.e.sh + t * R.e.st;
          // The dot products leave out a step's term with itself, and the last
          // step's with dstate_final: no decay lies between, so they cancel in
          // the decays' gradient, and where decays are strong they would leave
          // their rounding in place of much smaller sums.
          const float own = lds.diag[i];
          const bool no_dot = rev && t == args.L - 1;
#pragma unroll
          for (int ct = 0; ct < NC; ++ct) {
            const int col = wcol0 + ct * 16 + lg * 4;
            if (col < dc) {
              float4 v = make_float4(acc[tt][ct][0], acc[tt][ct][1], acc[tt][ct][2], acc[tt][ct][3]);
              if (R.dots) {
                const float4 x = Vec4<T>::cvt(Vec4<T>::load(pe, col));
                if (!no_dot) dot += v.x * x.x + v.y * x.y + v.z * x.z + v.w * x.w;
                const T *c = lds.c + i * SC + (w * NC + ct) * 16 + lg * 4;
                v.x = fmaf(own, load_io(c, 0), v.x), v.y = fmaf(own, load_io(c, 1), v.y);
                v.z = fmaf(own, load_io(c, 2), v.z), v.w = fmaf(own, load_io(c, 3), v.w);
              }
              if (R.out_f32)
                *(float4 *)((float *)R.out + o + col) = v;
              else
                Vec4<T>::store((T *)R.out, o + col, v);
            }
          }
        }
        if (R.dots) {
          dot += __shfl_xor(dot, 16, 64);
          dot += __shfl_xor(dot, 32, 64);
          if (lg == 0 && i < rows) R.dots[((int64_t)(slice * NW + w) * args.BH + bh) * args.L + t] = dot;
        }
      }
    }
    // the chunk's steps enter the state
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int ct = 0; ct < NC; ++ct) S[dt][ct] *= e;
#pragma unroll
    for (int kk = 0; kk < C / 32; ++kk) {
      Frag xf[NC][NB];
#pragma unroll
      for (int ct = 0; ct < NC; ++ct) {
        float x[8];
        M::floats(cf[kk][ct], x);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[r] *= lds.out[kk * 32 + lg * 4 + r];
          x[4 + r] *= lds.out[kk * 32 + 16 + lg * 4 + r];
        }
        M::template split<NB>(x, xf[ct]);
      }
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        const Frag bf = M::colfrag(lds.b, SA, kk * 32, M::coloff_perm(dt));
#pragma unroll
        for (int ct = 0; ct < NC; ++ct)
#pragma unroll
          for (int i = NB - 1; i >= 0; --i) S[dt][ct] = M::mma(bf, xf[ct][i], S[dt][ct]);
      }
    }
  }

  if constexpr (STATE_ONLY) {
    const int64_t j = (int64_t)bh * args.nseg + seg;
    float *loc = R.loc + (j * args.nslice + slice) * kTile + wtile;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int ct = 0; ct < NC; ++ct) *(f32x4 *)(loc + (dt * NC + ct) * 256) = S[dt][ct];
    if (threadIdx.x == 0 && slice == 0) R.tot[j] = total;
  } else if (seg == (rev ? 0 : args.nseg - 1)) {
    if (R.edge && !rev) {
      float *o = R.edge + (((int64_t)bh * (args.nseg + 1) + args.nseg) * args.nslice + slice) * kTile + wtile;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) *(f32x4 *)(o + (dt * NC + ct) * 256) = S[dt][ct];
    }
    if (R.state_out) {
      const float e = rev ? fast_exp2(decay_log2(pg[0])) : 1.0f;  // the first step's own decay
      float *s = R.state_out + (int64_t)bh * da * dc;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int ct = 0; ct < NC; ++ct)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = dt * 16 + lg * 4 + r, col = wcol0 + ct * 16 + l15;
            if (row < da && col < dc) s[(int64_t)row * dc + col] = S[dt][ct][r] * e;
          }
    }
  }
}

// Launches the kernel for one set of roles (decay_attn_f32.hip, decay_attn_bf16.hip).
// precise: outputs to fp32 (their dot products make the decays' gradient) and
// not only to the storage type.
hipError_t launch_decay_attn_f32(const DaArgs &a, int da_padded, bool precise, bool state_only, hipStream_t s);
hipError_t launch_decay_attn_bf16(const DaArgs &a, int da_padded, bool precise, bool state_only, hipStream_t s);

constexpr int kDaWaves = 4, kDaTiles = 1;
constexpr int kDaCols = kDaWaves * kDaTiles * 16;  // columns of dc per workgroup

template <typename T, int DA, int NP, int NS, bool STATE_ONLY>
hipError_t launch_da(const DaArgs &a, hipStream_t s) {
  const int64_t items = (int64_t)a.nslice * a.nroles * (STATE_ONLY ? a.nseg - 1 : a.nseg) * a.BH;
  if (items > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((decay_attn_kernel<T, DA, kDaWaves, kDaTiles, NP, NS, STATE_ONLY>), dim3((unsigned)items),
                     dim3(kDaWaves * 64), 0, s, a);
  return hipGetLastError();
}

template <typename T, int DA>
hipError_t launch_da_mode(const DaArgs &a, bool precise, bool state_only, hipStream_t s) {
  if (state_only) return launch_da<T, DA, 1, 1, true>(a, s);
  if constexpr (sizeof(T) == 2) {
    // One piece of the in-chunk products would leave the output an error of
    // 1.4 roundings instead of one; two pieces of both operands leave one.
    return precise ? launch_da<T, DA, 3, 3, false>(a, s) : launch_da<T, DA, 2, 2, false>(a, s);
  } else {
    return launch_da<T, DA, 1, 1, false>(a, s);
  }
}

template <typename T>
hipError_t launch_da_type(const DaArgs &a, int da_padded, bool precise, bool state_only, hipStream_t s) {
  switch (da_padded) {
    case 32: return launch_da_mode<T, 32>(a, precise, state_only, s);
    case 64: return launch_da_mode<T, 64>(a, precise, state_only, s);
    case 128: return launch_da_mode<T, 128>(a, precise, state_only, s);
    case 256: return launch_da_mode<T, 256>(a, precise, state_only, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace ssm
