// mixer_device.hpp -- device helpers of the gated recurrence, the causal
// convolution and the norm and rotation of heads: vectors of the io types and
// the gates.
#pragma once

#include "device_common.hpp"

namespace ssm {

// Two fp32 values as bf16, round to nearest even, in one instruction of gfx950.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const f2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));
}

// Inputs that a call reads once are loaded past the caches' usual order (non-temporal), so
// that outputs, which the next operator reads, stay in them instead: kStream marks a buffer load,
// load_once is a load of 8 or 16 bytes.  Recurrence 8 x 2048 x 2048 bf16 68 -> 65 us forward, 127 -> 118
// backward (201 -> 183 with an elementwise pass over its outputs behind it, 223 -> 212 with one over its
// inputs before it), fp32 logistic forward 90 -> 77, 32K context 346 -> 334; convolution 4 x 4096 x 5120
// 76 -> 72 forward (124 -> 114 after such a pass), 120 -> 108 backward.  It loses only where inputs would
// stay in the last-level cache from one use to the next (3 x 1537 x 1000 fp32 backward after such a pass 80 -> 89).
constexpr int kStream = 2;
__device__ __forceinline__ uint2 load_once(const uint2 *p) {
  typedef uint32_t u2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint2, __builtin_nontemporal_load((const u2 *)p));
}
__device__ __forceinline__ float4 load_once(const float4 *p) {
  typedef float f4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(float4, __builtin_nontemporal_load((const f4 *)p));
}

// Adjacent elements at an address aligned to 16 bytes, 8 in bf16: 4 of them, of fp32 any multiple of 4.
template <int N>
__device__ __forceinline__ void load_vec(const float *p, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 a = *(const float4 *)(p + i);
    v[i] = a.x, v[i + 1] = a.y, v[i + 2] = a.z, v[i + 3] = a.w;
  }
}
__device__ __forceinline__ void load_vec(const bf16 *p, float (&v)[4]) {
  const uint2 a = *(const uint2 *)p;
  const uint32_t w[2] = {a.x, a.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}
__device__ __forceinline__ void store_vec(float *p, const float (&v)[4]) { *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void store_vec(bf16 *p, const float (&v)[4]) { *(uint2 *)p = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])); }

// sigmoid(v) and 1 - sigmoid(v), neither from the other by a subtraction: e^-v
// over 1 + e^-v keeps the digits of a nearly open gate's complement.
__device__ __forceinline__ void sigmoid_both(float v, float &one, float &other) {
  const float e = fast_exp2(-v * kLog2e);
  one = fast_rcp(1.0f + e);
  other = v < -64.0f ? 1.0f : e * one;  // (e is infinite from about -88 on)
}

// sigmoid(v), and in one register what its derivative needs too: a sigmoid up to 1/2
// itself, a larger one as minus its complement (so that the other side is the fraction
// that is left to the next whole number; -2^-126 instead of nothing at all keeps the sign).  The
// complement formed as 1 minus the sigmoid has lost 3% of itself at v = 12 and all at 17.
__device__ __forceinline__ float sigmoid_folded(float v, float &folded) {
  const float e = fast_exp2(-v * kLog2e), one = fast_rcp(1.0f + e);
  folded = v >= 0.0f ? fmaf(-e, one, -0x1p-126f) : one;
  return one;
}
// the sigmoid and its derivative, sigmoid times complement
__device__ __forceinline__ void unfold(float folded, float &one, float &slope) {
  one = __builtin_amdgcn_fractf(folded);
  slope = fmaf(-fabsf(folded), fabsf(folded), fabsf(folded));
}

// z sigmoid(z) and its derivative
__device__ __forceinline__ void silu_both(float z, float &f, float &df) {
  float g, o;
  sigmoid_both(z, g, o);
  f = z * g;
  df = g * fmaf(z, o, 1.0f);
}

__device__ __forceinline__ int row_length(const int32_t *lengths, int64_t b, int64_t L) {
  const int64_t n = lengths ? (int64_t)lengths[b] : L;
  return (int)(n < 0 ? 0 : n < L ? n : L);
}

}  // namespace ssm
