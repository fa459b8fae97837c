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
// range of steps, so that nothing overflows where decays are at most one.  Where
// they grow, a factor of many steps may leave fp32's range although the states
// do not, being zero or small: there outputs and state are formed 2^-shift times
// as large, with factors of about half the exponent, and scaled at the end.  G
// is summed in 64 bits and kept as a pair of floats, so that differences of
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
// (smallest fp32 2^-149) and clear the state, as -inf does: they are held at a
// finite one, so that sums of decays stay finite, far below what growth after
// them can make up for.
constexpr float kMinLog2Decay = -256.0f, kClearLog2 = -4096.0f;
__device__ __forceinline__ float decay_log2(float g) {
  return g < kMinLog2Decay * kLn2 ? kClearLog2 : g * kLog2e;  // NaN passes
}

// 2^x in two factors, each in fp32's range for |x| up to 240.  Beyond, what they
// multiply is out of range itself, or a state that was cleared: zero.
__device__ __forceinline__ float2 exp2_in_two(double x) {
  const double n = rint(x);
  const int k = n < -240.0 ? -400 : (int)fmin(n, 240.0), k1 = k >> 1;
  return make_float2(ldexpf(fast_exp2((float)(x - n)), k1), ldexpf(1.0f, k - k1));
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
  float *dots;           // (slices, B * H, L) partial sums of out . e, or NULL
  float *loc;            // segments: end states from zero (or, combined, the states before them),
  float2 *tot;           // total decays, in two factors
  int loc_t, cols_t, nslice_t;  // loc is of a role with the transposed state, with slices of cols_t
  float *edge;           // states at edges (below), (B * H, edges, slices, tile), or NULL
  float *edge_dot;       // forward in time: <exp(g) S, R> at edges, (slices * waves, B * H, edges)
};

struct DaArgs {
  int64_t L, da, dc;
  const float *g;
  int64_t g_b, g_t;
  int H, BH, nseg, nslice, nroles;
  int dc_t;              // rows of the transposed role's tiles
  int combined;          // loc holds the states before the segments
  int64_t seg_len;       // a multiple of the chunk
  // An edge lies before every step E, 2 E, ..., E = 2^edge_shift; edge i - 1 before
  // step i * E, the last one (if last_edge) after the last step.  The
  // backward direction writes its states R there, the forward one dots its own
  // with them: the decays' gradient starts from them (decay_attn.hip).
  int edge_shift, nedge, last_edge;
  DaRole role[2];
};

// Matrix fragments of 32 along the contracted dimension and 16 along the
// other: lane l holds, for row (or column) l % 16, the contracted indices
// 4 (l / 16) + r and 16 + 4 (l / 16) + r, r = 0..3.  This order makes the
// accumulators of a 16 x 16 product (row 4 (l / 16) + r, column l % 16) usable
// as the next product's operand without moving data between lanes.
//
// In LDS, matrices read only as rows hold the 8 bf16 values of a fragment side
// by side (32-blocks as [l / 16][half][r], pos()); one that is also read by
// columns keeps its order.  Rows are padded so that reads meet no bank
// conflicts; measured clocks per fragment (8 waves of one workgroup) by row
// stride modulo 256 bytes:
//                                             +16 bytes   +32
//   bf16 row, side by side, ds_read_b128          8.0     4.1
//   bf16 row in order, 2 x ds_read_b64            4.8     8.1   (ds_read2_b64: 16, 32)
//   bf16 column in order, 2 x ds_read_b64_tr      8.1     4.8
//   bf16 column, side by side, the same          16.1     8.1
//
// Matrices in LDS are bf16.  Values of fp32 (inputs of that type, the state,
// products of steps, decayed rows) are sums of three bf16 pieces that hold all 24
// bits: each is what is left, rounded to nearest, so that the second is at most
// 2^-8 of the value's power of two and the third 2^-17.  Of the products of two
// such operands the six largest are formed, at 6 / 16 of the time of the fp32
// matrix instructions.  The other three add up to at most 2^-24 of the operands'
// powers of two, of either sign: a rounding of fp32.  (Pieces that are cut off
// leave up to 2^-21, always towards zero, which adds up over like-signed sums.)
template <int N>
struct Pieces {
  uint4 p[N];
};

// acc[x] += a(x) b(x) for x = 0 .. X - 1, smallest products first, neighbours independent
template <int NA, int NB, int X, typename A, typename B, typename Acc>
__device__ __forceinline__ void mma_pieces(A a, B b, Acc acc) {
  constexpr int M = (NA > NB ? NA : NB) - 1;
#pragma unroll
  for (int s = M; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB)
#pragma unroll
        for (int x = 0; x < X; ++x)
          acc(x) = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a(x).p[i]), __builtin_bit_cast(bf16x8, b(x).p[s - i]), acc(x), 0, 0, 0);
}

constexpr int kPad = 16;  // elements between rows

__device__ __forceinline__ constexpr int pos(int k) { return (k & ~31) | ((k & 12) << 1) | ((k & 16) >> 2) | (k & 3); }

// Fragments of a matrix of N planes, `plane` elements apart; l: the lane.
template <int N>
__device__ __forceinline__ Pieces<N> rowfrag(const bf16 *m, int plane, int stride, int row0, int k0, int l) {
  Pieces<N> f;
#pragma unroll
  for (int i = 0; i < N; ++i) f.p[i] = *(const uint4 *)(m + i * plane + (row0 + (l & 15)) * stride + k0 + (l >> 4) * 8);
  return f;
}
// from a row whose 16-byte units are permuted by x
__device__ __forceinline__ int swizzled(int k, int x) { return pos(k) ^ (x * 8); }
template <int N>
__device__ __forceinline__ Pieces<N> rowfrag_swizzled(const bf16 *row, int plane, int k0, int x, int l) {
  Pieces<N> f;
#pragma unroll
  for (int i = 0; i < N; ++i) f.p[i] = *(const uint4 *)(row + i * plane + ((k0 + (l >> 4) * 8) ^ (x * 8)));
  return f;
}
// from a matrix in order: two reads, volatile so that they do not become one ds_read2_b64
template <int N>
__device__ __forceinline__ Pieces<N> rowfrag_inorder(const bf16 *m, int plane, int stride, int row0, int k0, int l) {
  typedef __attribute__((address_space(3))) const volatile uint64_t lds_u64;
  Pieces<N> f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    lds_u64 *p = (lds_u64 *)(m + i * plane + (row0 + (l & 15)) * stride + k0 + (l >> 4) * 4);
    const uint2 x = __builtin_bit_cast(uint2, (uint64_t)p[0]), y = __builtin_bit_cast(uint2, (uint64_t)p[4]);
    f.p[i] = make_uint4(x.x, x.y, y.x, y.y);
  }
  return f;
}
// transposed: contracted along rows, column col0 + l % 16.  The transposing
// read gives lane i of 16 column i of a block of 4 rows x 16 columns, of
// which it addresses row i / 4, columns 4 (i % 4) ...
__device__ __forceinline__ uint2 tr4(const bf16 *p) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p)));
}
template <int N>
__device__ __forceinline__ Pieces<N> colfrag(const bf16 *m, int plane, int stride, int row0, int col0, int l) {
  Pieces<N> f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bf16 *p = m + i * plane + (row0 + (l >> 4) * 4 + ((l >> 2) & 3)) * stride + col0 + (l & 3) * 4;
    const uint2 x = tr4(p), y = tr4(p + 16 * stride);
    f.p[i] = make_uint4(x.x, x.y, y.x, y.y);
  }
  return f;
}
template <int N>
__device__ __forceinline__ void floats(const Pieces<N> &f, float (&x)[8]) {
#pragma unroll
  for (int n = N - 1; n >= 0; --n) {
    const uint32_t w[4] = {f.p[n].x, f.p[n].y, f.p[n].z, f.p[n].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xffff0000u);
      x[2 * i] = n == N - 1 ? a : x[2 * i] + a, x[2 * i + 1] = n == N - 1 ? b : x[2 * i + 1] + b;
    }
  }
}
__device__ __forceinline__ uint32_t pack_rne(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}
// Two fp32 values as N pieces, each rounded to nearest.
template <int N>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&o)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    o[i] = pack_rne(a, b);
    a -= __uint_as_float(o[i] << 16);
    b -= __uint_as_float(o[i] & 0xffff0000u);
  }
}
// From here on a value's first piece is infinite.
constexpr float kRoundsToInf = 0x1.ffp127f;
template <int N>
__device__ __forceinline__ Pieces<N> split(const float (&x)[8]) {
  uint32_t w[4][N];
#pragma unroll
  for (int i = 0; i < 4; ++i) split2<N>(x[2 * i], x[2 * i + 1], w[i]);
  Pieces<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) f.p[n] = make_uint4(w[0][n], w[1][n], w[2][n], w[3][n]);
  return f;
}
// four adjacent values
template <int N>
__device__ __forceinline__ void put4(bf16 *p, int plane, const float (&x)[4]) {
  uint32_t a[N], b[N];
  split2<N>(x[0], x[1], a);
  split2<N>(x[2], x[3], b);
#pragma unroll
  for (int n = 0; n < N; ++n) *(uint2 *)(p + n * plane) = make_uint2(a[n], b[n]);
}
template <int N>
__device__ __forceinline__ f32x4 get4(const bf16 *p, int plane) {
  f32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int n = N - 1; n >= 0; --n) {
    const uint2 w = *(const uint2 *)(p + n * plane);
    v += f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u)};
  }
  return v;
}
// zeros in place of NaN and infinities
template <int N>
__device__ __forceinline__ void make_finite(Pieces<N> &f) {
#pragma unroll
  for (int n = N - 1; n >= 0; --n) {
    uint32_t w[4] = {f.p[n].x, f.p[n].y, f.p[n].z, f.p[n].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
      if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu;
    }
    f.p[n] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Storage types: pieces of an element, steps per chunk (what LDS holds), and 16
// bytes of a row of elements k .. on.
template <typename T>
struct Store;
template <>
struct Store<bf16> {
  static constexpr int NX = 1, kChunk = 64;
  static __device__ __forceinline__ void put_inorder(bf16 *row, int, int k, uint4 v) { *(uint4 *)(row + k) = v; }
  static __device__ __forceinline__ void put_row(bf16 *row, int, int k, uint4 v) {
    *(uint2 *)(row + pos(k)) = make_uint2(v.x, v.y);
    *(uint2 *)(row + pos(k) + 8) = make_uint2(v.z, v.w);
  }
  static __device__ __forceinline__ void store4(void *p, f32x4 v) { *(uint2 *)p = make_uint2(pack_rne(v[0], v[1]), pack_rne(v[2], v[3])); }
  // sign bits of the result are set where an exponent is all ones
  static __device__ __forceinline__ uint32_t nonfinite(uint4 v) {
    constexpr uint32_t m = 0x7f807f80u, one = 0x00800080u;
    return (((v.x & m) + one) | ((v.y & m) + one) | ((v.z & m) + one) | ((v.w & m) + one)) & 0x80008000u;
  }
  static __device__ __forceinline__ float element(uint4 v, int j) {
    const uint32_t w = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
    return __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
  }
};
template <>
struct Store<float> {
  static constexpr int NX = 3, kChunk = 32;
  static __device__ __forceinline__ void put_inorder(bf16 *row, int plane, int k, uint4 v) {
    const float x[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
    put4<3>(row + k, plane, x);
  }
  static __device__ __forceinline__ void put_row(bf16 *row, int plane, int k, uint4 v) { put_inorder(row + pos(k) - k, plane, k, v); }
  static __device__ __forceinline__ void store4(void *p, f32x4 v) { *(f32x4 *)p = v; }
  static __device__ __forceinline__ uint32_t nonfinite(uint4 v) {
    // (values that round to it count as infinite)
    constexpr uint32_t m = 0x7fffffffu, one = 0x80000000u - 0x7f7f8000u;
    return (((v.x & m) + one) | ((v.y & m) + one) | ((v.z & m) + one) | ((v.w & m) + one)) & 0x80000000u;
  }
  static __device__ __forceinline__ float element(uint4 v, int j) { return __uint_as_float(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w); }
};

// The value, opaque to the compiler: what is computed from it stays where it is
// written and holds no registers over a loop (a spill there would cost a wait
// for all loads under way).
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// A (ROWS, COLS) tile on its way from global memory to LDS, 16 bytes at a time.
// Offsets within a tile are 32-bit, from a base that is the same for all lanes.
template <typename T, int ROWS, int COLS, int NT>
struct TileRegs {
  static constexpr int EPP = 16 / (int)sizeof(T), PPR = COLS / EPP, N = (ROWS * PPR + NT - 1) / NT, RSTEP = NT / PPR;
  static_assert(PPR <= NT && NT % PPR == 0, "whole rows per step");
  uint4 r[N];
  // row0: the first row; st: bytes from row to row; rows, cols: how many there are (both >= 1)
  __device__ __forceinline__ void load(const char *row0, uint32_t st, int rows, int cols) {
    const int tid = here(threadIdx.x), row = tid / PPR, col = (tid % PPR) * EPP;
    const uint32_t c = col < cols ? col * (uint32_t)sizeof(T) : 0;
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = *(const uint4 *)(row0 + ((uint32_t)min(row + i * RSTEP, rows - 1) * st + c));
  }
  // Puts the tile into LDS rows `stride` elements apart, zeros outside
  // rows x cols, in reverse order of rows if rev.  CHECK: first[col] becomes the
  // first row of a column with a NaN or an infinity, and *any nonzero.
  // ROWS_ONLY: side by side for row fragments.
  template <bool ROWS_ONLY, bool CHECK>
  __device__ __forceinline__ void put(bf16 *lds, int plane, int stride, int rows, int cols, bool rev, int *first = nullptr, int *any = nullptr) const {
    const int tid = here(threadIdx.x), row = tid / PPR, col = (tid % PPR) * EPP;
    auto one = [&](int lr, uint4 v) {
      if (ROWS_ONLY)
        Store<T>::put_row(lds + lr * stride, plane, col, v);
      else
        Store<T>::put_inorder(lds + lr * stride, plane, col, v);
      if (CHECK && Store<T>::nonfinite(v)) {
        *any = 1;
        for (int j = 0; j < EPP; ++j)
          if (!(fabsf(Store<T>::element(v, j)) < kRoundsToInf)) atomicMin(first + col + j, lr);
      }
    };
    if (rows == ROWS && cols == COLS && N * NT == ROWS * PPR) {  // the same for all lanes
#pragma unroll
      for (int i = 0; i < N; ++i) one(rev ? ROWS - 1 - row - i * RSTEP : row + i * RSTEP, r[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int rr = row + i * RSTEP;
        const bool in = rr < rows;
        if (N * NT == ROWS * PPR || rr < ROWS) one(rev && in ? rows - 1 - rr : rr, in && col < cols ? r[i] : make_uint4(0, 0, 0, 0));
      }
    }
  }
};

// What a chunk's decays enter as.
template <int C>
struct __attribute__((aligned(16))) DaDecays {
  float gh[C], gl[C];  // G_t as a pair of floats
  float in[C];         // exp(G_t), of the state in a step's output
  float out[C];        // exp(G_last - G_s), of a step in the next chunk's state
  float shift[C];      // in a chunk that grows: powers of two that a step's output is formed too small by
  float e[4];          // [0]: exp(G_last); [1]: not zero if the chunk grows, then [2]: 2^shift of the state
};
// A chunk can grow by 2^100 only if a step of it grows by more than this.
template <int C>
constexpr float kGrows = 100.0f / C;
// A shift is half of the growth, at most kMostShift (what does not grow must stay
// far from fp32's smallest numbers); factors are kept finite, so that zeros stay zero.
constexpr float kMostShift = 100.0f, kMostPowers = 120.0f;
// (NaN and infinities pass)
__device__ __forceinline__ float in_range(float x) { return x > kMostPowers && x < 1e30f ? kMostPowers : x; }
__device__ __forceinline__ float shift_of(float growth) { return growth < 1e30f ? fminf(rintf(0.5f * growth), kMostShift) : 0.0f; }

// Sums over lanes 0 .. lane, by DPP moves within rows of 16 lanes and then
// from row to row (as wave_affine_scan).
template <int CTRL, int ROWMASK>
__device__ __forceinline__ double dpp_add(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWMASK, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWMASK, 0xF, false);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum_scan(double v) {
  v = dpp_add<0x111, 0xF>(v);
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);
  return dpp_add<0x143, 0xC>(v);
}

template <typename T, int DA, int NW, bool STATE_ONLY>
struct __attribute__((aligned(16))) DaLds {
  // Pieces of the products inside a chunk: all of fp32, for bf16 inputs too.  (Two
  // of them and of the state round one bf16 result in 500 the other way, and sums
  // that cancel lose 16 bits' worth; 8 x 2048 steps of 16 heads of 128: 117 us
  // against 124.)
  static constexpr int NP = 3;
  static constexpr int C = Store<T>::kChunk, NX = Store<T>::NX, TV = NW * 16;
  static constexpr int SA = DA + kPad, SC = TV + kPad;  // rows of a and b, of c
  // Products of steps, only blocks of 32 x 32 up to the diagonal: two row tiles of
  // 32 columns, then two of 64, without padding; instead the 16-byte units of a
  // row are permuted by its number (swizzle), so that 16 rows meet all banks.
  static constexpr int PLANE = 32 * 32 + (C > 32 ? 32 * 64 : 0);
  static __device__ __forceinline__ int pwidth(int tt) { return tt < 2 ? 32 : 64; }
  static __device__ __forceinline__ int prow(int tt, int r) { return (tt < 2 ? tt * 16 * 32 : 32 * 32 + (tt - 2) * 16 * 64) + r * pwidth(tt); }
  static __device__ __forceinline__ int swizzle(int tt, int r) { return tt < 2 ? (r >> 2) & 3 : (r >> 1) & 7; }
  bf16 a[STATE_ONLY ? 8 : NX * C * SA];
  bf16 b[NX * C * SA];
  bf16 c[NX * C * SC];
  bf16 p[STATE_ONLY ? 8 : NP * PLANE];
  DaDecays<C> dec[2];  // of this chunk and the next
  float diag[C];
  float dots[NW][C];
  int bad[2];      // whether c has a NaN or an infinity, in this chunk and the next,
  int first[TV];   // and from which step on, by column (C: nowhere)
};

// T: storage type; DA: da rounded up; NW waves of 16 columns of dc each.
// STATE_ONLY: the end state of a segment from zero (a split sequence's
// first pass).  DOTS: out . e wanted.
//
// What bounds it: no unit by itself.  At 8 x 2048 steps of 16 heads of 128, bf16,
// the main pass of 512 workgroups takes 92 to 96 us.  Of that its 304 MB past L2
// would take 61 at a large copy's rate; the 3.9 M matrix instructions keep the
// SIMDs' matrix units busy for 41% of the clocks, and the 28 M vector
// instructions (decays onto products, the state and c, and their pieces) fill 37%
// of the issue slots if two waves always pair up, 74% if they never do.  Waves
// wait 36% of their time for a slot and 37% for data and barriers: the phases of
// a chunk (rows to LDS, products of steps, what the state gives, the update)
// follow one another between three barriers.  The first pass of 384 workgroups
// takes 36 us for 127 MB, 7.9 M vector and 1.2 M matrix instructions; with DOTS 112
// to 135 us for 425 MB and 35 M.  In fp32 (2 x 1537 steps, 32 heads of 64) a main pass
// takes 40 us, 45 to 51 with DOTS.
// Chosen when the 8 x 2048 forward took 117 us: 16 columns to a wave (32 leave one
// workgroup to a CU, 124 us); 8 waves for 128 columns (126 against 167 us with 4
// waves, in twice the workgroups that read a and b).  Chunks are as long as LDS
// holds for two workgroups per CU (fp32, 128 wide: one): longer ones have more
// products inside, shorter ones more updates of the state.
template <typename T, int DA, int NW, bool DOTS, bool STATE_ONLY>
__global__ void __launch_bounds__(NW * 64, DA <= 128 ? 4 : 2) decay_attn_kernel(DaArgs args) {
  typedef Store<T> M;
  typedef DaLds<T, DA, NW, STATE_ONLY> Lds;
  constexpr int C = M::kChunk, NX = M::NX, CT = C / 16, DT = DA / 16, NT = NW * 64, TV = Lds::TV;
  constexpr int SA = Lds::SA, SC = Lds::SC, PLANE = Lds::PLANE, PA = C * SA, PC = C * SC;  // rows, planes
  constexpr int ES = sizeof(T);
  constexpr int NP = Lds::NP, NS = 3, NB = 3;  // pieces of products inside a chunk, of the state, of decayed rows into it: all of fp32
  __shared__ Lds lds;

  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l15 = lane & 15, lg = lane >> 4;
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
  const int col0 = slice * TV, wcol0 = col0 + w * 16;
  const int64_t t0 = seg * args.seg_len;
  const int n = (int)min(args.seg_len, args.L - t0);
  const int da = (int)args.da, dc = (int)args.dc;
  const int ccols = min(TV, dc - col0);

  // Rows t0 + u of the operands; strides in bytes.
  const char *pa = (const char *)R.a.p + (b * R.a.sb + (h / R.a.share) * R.a.sh + t0 * R.a.st) * ES;
  const char *pb = (const char *)R.b.p + (b * R.b.sb + (h / R.b.share) * R.b.sh + t0 * R.b.st) * ES;
  const char *pc = (const char *)R.c.p + (b * R.c.sb + (h / R.c.share) * R.c.sh + t0 * R.c.st + col0) * ES;
  const char *pe = DOTS ? (const char *)R.e.p + (b * R.e.sb + (h / R.e.share) * R.e.sh + t0 * R.e.st) * ES : nullptr;
  const uint32_t sta = (uint32_t)R.a.st * ES, stb = (uint32_t)R.b.st * ES, stc = (uint32_t)R.c.st * ES, ste = (uint32_t)R.e.st * ES;
  const bool out_f32 = R.out_f32 != 0;
  const int oes = out_f32 ? 4 : ES;
  const uint32_t sto = (uint32_t)args.H * (uint32_t)dc * oes;
  char *po = (char *)R.out + (((b * args.L + t0) * args.H + h) * dc) * oes;
  float *dots = DOTS ? R.dots + ((int64_t)slice * args.BH + bh) * args.L + t0 : nullptr;
  const float *pg = args.g + b * args.g_b + h;
  const float iscale = R.iscale, pscale = R.pscale, sscale = R.sscale;

  // The state: S[dt][r] is row dt * 16 + lg * 4 + r, column wcol0 + l15.
  f32x4 S[DT];
  constexpr int64_t kTile = (int64_t)DA * TV;
  const int64_t wtile = (int64_t)w * DT * 256 + lane * 4;
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) S[dt] = f32x4{0, 0, 0, 0};
  auto edge_tile = [&](int i) { return R.edge + (((int64_t)bh * args.nedge + i) * args.nslice + slice) * kTile + wtile; };
  auto store_edge = [&](int i) {
    float *o = edge_tile(i);
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) *(f32x4 *)(o + dt * 256) = S[dt];
  };
  // exp(g) of the step after the edge comes to S first: <S, R> may be out of range where this is not
  auto dot_edge = [&](int i, int64_t t) {
    const float *o = edge_tile(i);
    const float2 e = exp2_in_two(t < args.L ? decay_log2(pg[t * args.g_t]) : 0.0f);
    f32x4 d = {0, 0, 0, 0};
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      const f32x4 x = *(const f32x4 *)(o + dt * 256);
#pragma unroll
      for (int r = 0; r < 4; ++r) d[r] = fmaf(S[dt][r] * e.x * e.y, x[r], d[r]);
    }
    float v = (d[0] + d[1]) + (d[2] + d[3]);
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1) v += __shfl_xor(v, k, 64);
    if (lane == 0) R.edge_dot[((int64_t)(slice * NW + w) * args.BH + bh) * args.nedge + i] = v;
  };
  auto load_state_in = [&] {
    if (R.state_in) {
      const float *s = R.state_in + (int64_t)bh * da * dc;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = dt * 16 + lg * 4 + r, col = wcol0 + l15;
          if (row < da && col < dc) S[dt][r] = s[R.state_in_t ? col * da + row : row * dc + col];
        }
    }
  };
  if constexpr (!STATE_ONLY) {
    if (R.loc_t) {
      // From the states of a role whose state is this one's transpose: its tile
      // of row x (a step of this role's columns) and column y holds, for lane
      // (x % 16) / 4 * 16 + y % 16, element x % 4.
      const int cols_t = R.cols_t, tiles_t = (args.dc_t >> 4);
      auto add = [&](int64_t j, float2 e) {
        const int x = wcol0 + l15;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
          const int y = dt * 16 + lg * 4, w_t = y % cols_t / 16;
          const float *p = R.loc + ((j * R.nslice_t + y / cols_t) * cols_t * args.dc_t) + (int64_t)(w_t * tiles_t + x / 16) * 256 + ((x % 16) / 4 * 16 + y % 16) * 4 + x % 4;
#pragma unroll
          for (int r = 0; r < 4; ++r) S[dt][r] = S[dt][r] * e.x * e.y + (x < dc && y + r < da ? p[r * 4] : 0.0f);
        }
      };
      const int before = rev ? args.nseg - 1 - seg : seg;
      if (args.combined) {
        add((int64_t)bh * args.nseg + seg, make_float2(0.0f, 0.0f));
      } else {
        load_state_in();
        for (int i = 0; i < before; ++i) {
          const int64_t j = (int64_t)bh * args.nseg + (rev ? args.nseg - 1 - i : i);
          add(j, R.tot[j]);
        }
      }
    } else if (args.combined) {
      const float *loc = R.loc + (((int64_t)bh * args.nseg + seg) * args.nslice + slice) * kTile + wtile;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) S[dt] = *(const f32x4 *)(loc + dt * 256);
    } else {
      load_state_in();
      // the segments before this one, in the order of the recurrence
      const int before = rev ? args.nseg - 1 - seg : seg;
      for (int i = 0; i < before; ++i) {
        const int64_t j = (int64_t)bh * args.nseg + (rev ? args.nseg - 1 - i : i);
        const float2 e = R.tot[j];
        const float *loc = R.loc + (j * args.nslice + slice) * kTile + wtile;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) S[dt] = S[dt] * e.x * e.y + *(const f32x4 *)(loc + dt * 256);
      }
    }
    if (DOTS && rev && args.last_edge && seg == args.nseg - 1) store_edge(args.nedge - 1);
    // products of steps later in a chunk are never written: they stay zero
    for (int i = threadIdx.x; i < NP * PLANE / 8; i += NT) ((uint4 *)lds.p)[i] = make_uint4(0, 0, 0, 0);
  }
  if (threadIdx.x < 2) lds.bad[threadIdx.x] = 0;
  for (int i = threadIdx.x; i < TV; i += NT) lds.first[i] = C;
  // (the first chunk's barrier comes after its own tile is put, so:)
  __syncthreads();

  // Chunk i of the recurrence holds rows low .. low + rows - 1 of the segment,
  // in reverse order backward in time.
  TileRegs<T, C, DA, NT> ra, rb;
  TileRegs<T, C, TV, NT> rc;
  const int nchunk = (n + C - 1) / C;
  auto low_of = [&](int i) { return (rev ? nchunk - 1 - i : i) * C; };
  auto fetch = [&](int i) {
    const int low = low_of(i), rows = min(C, n - low);
    if constexpr (!STATE_ONLY) ra.load(pa + (int64_t)low * sta, sta, rows, da);
    rb.load(pb + (int64_t)low * stb, stb, rows, da);
    rc.load(pc + (int64_t)low * stc, stc, rows, ccols);
  };
  // The last wave, which has the fewest products inside a chunk, prepares the
  // next chunk's decays beside them and loads those of the one after.
  float rg = 0.0f;
  bool have_g = false;
  auto fetch_decays = [&](int i) {
    // backward in time the decay into a step is the later step's
    const int low = low_of(i), rows = min(C, n - low);
    const int64_t t = t0 + low + (rev ? rows - lane : lane);
    have_g = i < nchunk && lane < rows && t < args.L;
    rg = pg[have_g ? t * args.g_t : 0];
  };
  double total = 0.0;  // of all chunks, in the last wave
  auto put_decays = [&](int i, DaDecays<C> &d) {
    const float g2 = have_g ? decay_log2(rg) : 0.0f;
    const bool grow = __ballot(g2 > kGrows<C>) != 0;
    const double G = wave_sum_scan(g2);
    const uint64_t gb = __builtin_bit_cast(uint64_t, G);
    const double last = __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(gb >> 32), 63) << 32 |
                                                       (uint32_t)__builtin_amdgcn_readlane((int)gb, 63));
    const float hi = (float)G;
    // the last edge's state leaves out the last step (see no_dot)
    const bool left_out = DOTS && args.last_edge && !rev && t0 + low_of(i) + lane == args.L - 1;
    float in = hi, out = (float)(last - G), e = (float)last;
    if (grow) {
      float least = fminf(hi, 0.0f);  // of G up to this step
#pragma unroll
      for (int k = 1; k < 64; k *= 2) {
        const float o = __shfl_up(least, k, 64);
        if (lane >= k) least = fminf(least, o);
      }
      const float shift = shift_of(hi - least), state_shift = shift_of(e - __shfl(least, 63, 64));
      in = in_range(in - shift), out = in_range(out - state_shift), e = in_range(e - state_shift);
      if (lane < C) d.shift[lane] = shift;
      if (lane == 0) d.e[2] = ldexpf(1.0f, (int)state_shift);
    }
    if (lane < C) {
      d.gh[lane] = hi;
      d.gl[lane] = (float)(G - (double)hi);
      d.in[lane] = fast_exp2(in) * iscale;
      d.out[lane] = left_out ? 0.0f : fast_exp2(out) * sscale;
    }
    if (lane == 0) d.e[0] = fast_exp2(e), d.e[1] = grow ? 1.0f : 0.0f;
    if (STATE_ONLY) total += last;
  };
  // a chunk's dot products, of all waves
  auto flush_dots = [&](int ci) {
    const int i = threadIdx.x, low = low_of(ci), rows = min(C, n - low);
    if (i < rows) {
      float d = lds.dots[0][i];
#pragma unroll
      for (int k = 1; k < NW; ++k) d += lds.dots[k][i];
      dots[low + (rev ? rows - 1 - i : i)] = d;
    }
  };
  fetch(0);
  if (w == NW - 1) {
    fetch_decays(0);
    put_decays(0, lds.dec[0]);
    fetch_decays(1);
  }
  int par = 0;

  for (int ci = 0; ci < nchunk; ++ci, par ^= 1) {
    const int low = low_of(ci), rows = min(C, n - low);
    // the edge before this chunk's rows, -1 if there is none
    const int edge = DOTS && ((t0 + low) & ((1 << args.edge_shift) - 1)) == 0 ? (int)((t0 + low) >> args.edge_shift) - 1 : -1;
    if (DOTS && !rev && edge >= 0) dot_edge(edge, t0 + low);
    __syncthreads();  // the last chunk's readers are done
    if constexpr (!STATE_ONLY) ra.template put<true, false>(lds.a, PA, SA, rows, da, rev);
    rb.template put<false, false>(lds.b, PA, SA, rows, da, rev);
    rc.template put<false, !STATE_ONLY>(lds.c, PC, SC, rows, ccols, rev, lds.first, lds.bad + par);
    if (DOTS && ci > 0) flush_dots(ci - 1);
    __syncthreads();
    const DaDecays<C> &dec = lds.dec[par];
    const float e = dec.e[0];
    const bool grow = __builtin_amdgcn_readfirstlane(__float_as_int(dec.e[1])) != 0;
    if (w == NW - 1 && ci + 1 < nchunk) {
      put_decays(ci + 1, lds.dec[par ^ 1]);
      fetch_decays(ci + 2);
    }

    f32x4 acc[CT];
    typename Vec4<T>::raw ev[DOTS ? CT : 1];
    if constexpr (!STATE_ONLY) {
      // products a_t . b_s of steps s <= t with their decays, 16 x 16 tiles over the waves
      constexpr int NTILE = CT * (CT + 1) / 2;
#pragma unroll
      for (int j = 0; j < (NTILE + NW - 1) / NW; ++j) {
        // (opaque, so that addresses are formed here and hold no registers over the loop)
        int idx = w + j * NW;
        asm volatile("" : "+s"(idx));
        if (idx >= NTILE) break;
        const int l = here(lane), l15 = l & 15, lg = l >> 4;
        const int tt = idx >= 6 ? 3 : idx >= 3 ? 2 : idx >= 1 ? 1 : 0, st = idx - tt * (tt + 1) / 2;
        // two chains of products, their reads first
        constexpr int KB = DA / 32 < 2 ? 1 : 2;
        f32x4 y[KB];
#pragma unroll
        for (int k = 0; k < KB; ++k) y[k] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int k0 = 0; k0 < DA / 32; k0 += KB) {
          Pieces<NX> fa[KB], fb[KB];
#pragma unroll
          for (int k = 0; k < KB; ++k) {
            fb[k] = rowfrag_inorder<NX>(lds.b, PA, SA, st * 16, (k0 + k) * 32, l);
            fa[k] = rowfrag<NX>(lds.a, PA, SA, tt * 16, (k0 + k) * 32, l);
          }
          mma_pieces<NX, NX, KB>([&](int k) { return fb[k]; }, [&](int k) { return fa[k]; }, [&](int k) -> f32x4 & { return y[k]; });
        }
        f32x4 x = y[0];
        if (KB == 2) x += y[KB - 1];
        const int t = tt * 16 + l15, s = st * 16 + lg * 4;
        const float th = dec.gh[t], tl = dec.gl[t];
        const f32x4 sh = *(const f32x4 *)(dec.gh + s), sl = *(const f32x4 *)(dec.gl + s);
        f32x4 d;
#pragma unroll
        for (int r = 0; r < 4; ++r) d[r] = (th - sh[r]) + (tl - sl[r]);
        if (grow) {
          const float shift = dec.shift[t];
#pragma unroll
          for (int r = 0; r < 4; ++r) d[r] = in_range(((th - shift) - sh[r]) + (tl - sl[r]));
        }
        float p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          // for the dot products a step's own term is kept apart (below)
          p[r] = s + r < t + (DOTS ? 0 : 1) ? x[r] * (fast_exp2(d[r]) * pscale) : 0.0f;
          if (DOTS && s + r == t) lds.diag[t] = x[r] * pscale;
        }
        put4<NP>(lds.p + Lds::prow(tt, l15) + swizzled(s, Lds::swizzle(tt, l15)), PLANE, p);
      }
      if constexpr (DOTS) {
#pragma unroll
        for (int tt = 0; tt < CT; ++tt) {
          const int l = here(lane), col = min(wcol0 + (l >> 4) * 4, dc - 4), row = min(tt * 16 + (l & 15), rows - 1);
          ev[tt] = Vec4<T>::load_b(pe + (int64_t)low * ste, (uint32_t)(rev ? rows - 1 - row : row) * ste + col * ES);
        }
      }
      // what the state gives
#pragma unroll
      for (int tt = 0; tt < CT; ++tt) acc[tt] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int kk = 0; kk < DA / 32; ++kk) {
        float x[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = S[2 * kk][r], x[4 + r] = S[2 * kk + 1][r];
        const Pieces<NS> sf = split<NS>(x);
        constexpr int G = DOTS ? CT / 2 : CT;  // row tiles at a time
#pragma unroll
        for (int t0 = 0; t0 < CT; t0 += G) {
          Pieces<NX> af[G];
#pragma unroll
          for (int i = 0; i < G; ++i) af[i] = rowfrag<NX>(lds.a, PA, SA, (t0 + i) * 16, kk * 32, lane);
          mma_pieces<NS, NX, G>([&](int) { return sf; }, [&](int i) { return af[i]; }, [&](int i) -> f32x4 & { return acc[t0 + i]; });
        }
      }
#pragma unroll
      for (int tt = 0; tt < CT; ++tt) {
        const float f = dec.in[tt * 16 + l15];
        acc[tt] *= f;
      }
    }
    // The next chunk's rows travel during the rest of this one (and hold no
    // registers before; with dot products, which need more, from the state on).
    if ((STATE_ONLY || !DOTS) && ci + 1 < nchunk) fetch(ci + 1);
    if constexpr (!STATE_ONLY) __syncthreads();  // all products are there
    Pieces<NX> cf[C / 32];
#pragma unroll
    for (int kk = 0; kk < C / 32; ++kk) cf[kk] = colfrag<NX>(lds.c, PC, SC, kk * 32, w * 16, here(lane));
    if constexpr (!STATE_ONLY) {
      if (threadIdx.x == 0) lds.bad[par ^ 1] = 0;
      // A NaN or an infinity in c must not meet the zeros of earlier steps in
      // the products: it is left out of them and poisons what comes after.
      const int bad = __builtin_amdgcn_readfirstlane(lds.bad[par]);
      if (bad) {
#pragma unroll
        for (int kk = 0; kk < C / 32; ++kk) make_finite(cf[kk]);
      }
      const int lp = here(lane);
      // (steps kk * 32 on meet row tiles 2 kk on; one piece of the products at a time)
#pragma unroll
      for (int kk = 0; kk < C / 32; ++kk)
#pragma unroll
        for (int i = NP - 1; i >= 0; --i) {
          Pieces<1> pf[CT];
#pragma unroll
          for (int tt = 2 * kk; tt < CT; ++tt) pf[tt] = rowfrag_swizzled<1>(lds.p + i * PLANE + Lds::prow(tt, lp & 15), 0, kk * 32, Lds::swizzle(tt, lp & 15), lp);
#pragma unroll
          for (int j = NX == 1 ? 0 : NP - 1 - i; j >= 0; --j)
#pragma unroll
            for (int tt = 2 * kk; tt < CT; ++tt)
              acc[tt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, cf[kk].p[j]), __builtin_bit_cast(bf16x8, pf[tt].p[0]), acc[tt], 0, 0, 0);
        }
      if (grow) {
#pragma unroll
        for (int tt = 0; tt < CT; ++tt) {
          const int shift = (int)dec.shift[tt * 16 + (lp & 15)];
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[tt][r] = ldexpf(acc[tt][r], shift);
        }
      }
      if (bad) {
        int *first = lds.first + w * 16;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int f = first[(lp >> 4) * 4 + r];
#pragma unroll
          for (int tt = 0; tt < CT; ++tt)
            if (tt * 16 + (lp & 15) >= f) acc[tt][r] = NAN;
        }
        if (first[lp & 15] < C) {
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) S[dt] = f32x4{NAN, NAN, NAN, NAN};
        }
        first[lp & 15] = C;  // for the next chunk; these columns are this wave's alone
      }
      // out^T: column wcol0 + lg * 4 + r of step tt * 16 + l15; loff: byte
      // offset of this lane's row and columns from those of row `low`
      const int lo = here(lane), l15 = lo & 15, lg = lo >> 4;
      const uint32_t loff = (uint32_t)(rev ? rows - 1 - l15 : l15) * sto + (wcol0 + lg * 4) * oes;
#pragma unroll
      for (int tt = 0; tt < CT; ++tt) {
        const int i = tt * 16 + l15;
        if constexpr (DOTS) {
          // The dot products leave out a step's term with itself, and the last
          // step's with dstate_final: no decay lies between, so they cancel in
          // the decays' gradient, and where decays are strong they would leave
          // their rounding in place of much smaller sums.
          const bool no_dot = rev && t0 + n == args.L && ci == 0 && i == 0;
          const float own = lds.diag[i];
          float dot = 0.0f;
          const int col = wcol0 + lg * 4;
          const f32x4 cv = get4<NX>(lds.c + i * SC + w * 16 + lg * 4, PC);
          const float4 x = Vec4<T>::cvt(ev[tt]);
          const f32x4 xv = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (col < dc) dot = fmaf(acc[tt][r], xv[r], dot);
            acc[tt][r] = fmaf(own, cv[r], acc[tt][r]);
          }
          dot += __shfl_xor(dot, 16, 64);
          dot += __shfl_xor(dot, 32, 64);
          if (lg == 0) lds.dots[w][i] = no_dot ? 0.0f : dot;
        }
        if (i < rows && wcol0 + lg * 4 < dc) {
          char *p = po + (int64_t)(low + (rev ? -tt * 16 : tt * 16)) * sto + loff;
          if (out_f32)
            *(f32x4 *)p = acc[tt];
          else
            M::store4(p, acc[tt]);
        }
      }
    }
    if (!STATE_ONLY && DOTS && ci + 1 < nchunk) fetch(ci + 1);
    // the chunk's steps enter the state
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) S[dt] *= e;
#pragma unroll
    for (int kk = 0; kk < C / 32; ++kk) {
      const f32x4 y0 = *(const f32x4 *)(dec.out + kk * 32 + lg * 4), y1 = *(const f32x4 *)(dec.out + kk * 32 + 16 + lg * 4);
      float x[8];
      floats(cf[kk], x);
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] *= y0[r], x[4 + r] *= y1[r];
      const Pieces<NB> xf = split<NB>(x);
      const int ls = here(lane);
      constexpr int G = (DT < 4 ? DT : 4) / (NX == 1 ? 1 : 2);  // independent products side by side
#pragma unroll
      for (int d0 = 0; d0 < DT; d0 += G) {
        Pieces<NX> bf[G];
#pragma unroll
        for (int d = 0; d < G; ++d) bf[d] = colfrag<NX>(lds.b, PA, SA, kk * 32, (d0 + d) * 16, ls);
        mma_pieces<NX, NB, G>([&](int d) { return bf[d]; }, [&](int) { return xf; }, [&](int d) -> f32x4 & { return S[d0 + d]; });
      }
    }
    if (grow) {
      const float f = dec.e[2];
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) S[dt] *= f;
    }
    if (DOTS && rev && edge >= 0) store_edge(edge);
  }
  if constexpr (DOTS) {
    __syncthreads();
    flush_dots(nchunk - 1);
  }

  if constexpr (STATE_ONLY) {
    const int64_t j = (int64_t)bh * args.nseg + seg;
    float *loc = R.loc + (j * args.nslice + slice) * kTile + wtile;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) *(f32x4 *)(loc + dt * 256) = S[dt];
    if (w == NW - 1 && lane == 0 && slice == 0) R.tot[j] = exp2_in_two(total);
  } else if (seg == (rev ? 0 : args.nseg - 1)) {
    if (DOTS && !rev && args.last_edge) dot_edge(args.nedge - 1, args.L);
    if (R.state_out) {
      const float e = rev ? fast_exp2(decay_log2(pg[0])) : 1.0f;  // the first step's own decay
      float *s = R.state_out + (int64_t)bh * da * dc;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = dt * 16 + lg * 4 + r, col = wcol0 + l15;
          if (row < da && col < dc) s[row * dc + col] = S[dt][r] * e;
        }
    }
  }
}

// Launches the kernel for one set of roles (decay_attn_f32.hip, decay_attn_bf16.hip).
// dots: the outputs' dot products with e, and outputs to fp32 for them.
hipError_t launch_decay_attn_f32(const DaArgs &a, int da_padded, bool dots, bool state_only, hipStream_t s);
hipError_t launch_decay_attn_bf16(const DaArgs &a, int da_padded, bool dots, bool state_only, hipStream_t s);

// Waves per workgroup, of 16 columns of dc each.
inline int da_waves(int64_t dc) { return dc > 64 ? 8 : 4; }

template <typename T, int DA, int NW, bool DOTS, bool STATE_ONLY>
hipError_t launch_da(const DaArgs &a, hipStream_t s) {
  const int64_t items = (int64_t)a.nslice * a.nroles * (STATE_ONLY ? a.nseg - 1 : a.nseg) * a.BH;
  if (items > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((decay_attn_kernel<T, DA, NW, DOTS, STATE_ONLY>), dim3((unsigned)items), dim3(NW * 64), 0, s, a);
  return hipGetLastError();
}

template <typename T, int DA, int NW>
hipError_t launch_da_mode(const DaArgs &a, bool dots, bool state_only, hipStream_t s) {
  if (state_only) return launch_da<T, DA, NW, false, true>(a, s);
  return dots ? launch_da<T, DA, NW, true, false>(a, s) : launch_da<T, DA, NW, false, false>(a, s);
}

template <typename T, int DA>
hipError_t launch_da_waves(const DaArgs &a, bool dots, bool state_only, hipStream_t s) {
  return da_waves(a.dc) == 8 ? launch_da_mode<T, DA, 8>(a, dots, state_only, s) : launch_da_mode<T, DA, 4>(a, dots, state_only, s);
}

template <typename T>
hipError_t launch_da_type(const DaArgs &a, int da_padded, bool dots, bool state_only, hipStream_t s) {
  switch (da_padded) {
    case 32: return launch_da_waves<T, 32>(a, dots, state_only, s);
    case 64: return launch_da_waves<T, 64>(a, dots, state_only, s);
    case 128: return launch_da_waves<T, 128>(a, dots, state_only, s);
    case 256: return launch_da_waves<T, 256>(a, dots, state_only, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace ssm
