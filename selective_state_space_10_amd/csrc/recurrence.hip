// recurrence.hip -- the gated recurrence h_t = a_t h_{t-1} + s_t i_t x_t over whole
// sequences, its gradients, and one token.
//
// Every input is read once and every output written once, and the bytes are the
// floor; what keeps the kernels above it is that a workgroup loads, computes, waits for
// the state before its chunk and stores in turn, and registers let only two workgroups
// share a CU.  Vector units are active for half of the time (34 vector instructions
// per element forward, 6 of them transcendental, and 68 with 7 backward), waves wait two fifths of it.
// Measured, per call (a large copy moves 5.1 TB/s), bf16 in power form with an input gate:
//   forward   8 x 2048 x 2048 (268 MB)            62 us, 4.3 TB/s (one lane per channel: 1782 us)
//             4 x 4096 x 5120 (671 MB)           134 us, 5.0 TB/s
//             1 x 32768 x 5120, z (1.68 GB)      334 us, 5.0 TB/s
//             1 x 1048576 x 1024 (8.6 GB)        2.00 ms, 4.3 TB/s
//   backward  8 x 2048 x 2048 (471 MB)           116 to 125 us, 3.8 to 4.0 TB/s (one lane per channel: 3298 us)
//             1 x 32768 x 5120, z (3.0 GB)       698 us, 4.3 TB/s
//   one token 256 x 5120, z (24 MB)              6 us
//   narrow and long, where the states' way through the chunks is what takes the time:
//             1 x 32768 x 256                    54 us forward, 47 backward (67 and 118 MB)
//             1 x 32768 x 1024                   72 and 122 us (268 and 471 MB)
#include "mixer_device.hpp"
#include "mixer_kernels.hpp"

namespace ssm {

using namespace recurrence;

namespace {

// The decay's gate.  Power form: r = sigmoid(g), log2 a = rate2 r, s^2 = 1 - a^2,
// by the series of -expm1(2 log a) where a is near 1: four terms up to 1/8 leave
// (1/8)^5 / 720 < 2^-24 relative, beyond it 1 - a^2 loses 2^-24 / (1 - e^-1/8) of
// itself, half of that in s.  Logistic form: a = r, s = 1 - r.
// keep: of the gate, what its gradient needs: the folded sigmoid, or 1 - r.
struct Gate {
  float a, s, keep;
};
__device__ __forceinline__ float scale_of(float la2, float a) {
  const float v = 2.0f * kLn2 * la2;
  const float p = fmaf(v, fmaf(v, fmaf(v, fmaf(v, 1.0f / 120, 1.0f / 24), 1.0f / 6), 0.5f), 1.0f);
  return __builtin_amdgcn_sqrtf(fabsf(v) < 0.125f ? -v * p : fmaf(-a, a, 1.0f));
}
template <bool POWER>
__device__ __forceinline__ Gate gate_of(float g, float rate2) {
  Gate q;
  if constexpr (POWER) {
    const float la2 = rate2 * sigmoid_folded(g, q.keep);
    q.a = fast_exp2(la2);
    q.s = scale_of(la2, q.a);
  } else {
    sigmoid_both(g, q.a, q.s);
    q.keep = q.s;
  }
  return q;
}

// softplus to fp32's rounding: e^-|v| by the exponent's rounded product and what that
// leaves out, log1p by the logarithm of the rounded 1 + w and what that leaves out.
// (Below -200, -infinity too, e^-|v| is zero; a comparison, which lets NaN through.)
__device__ __forceinline__ float softplus_full(float v) {
  const float m = fabsf(v) > 200.0f ? -200.0f : -fabsf(v), t = m * kLog2e;
  const float rest = fmaf(m, kLog2e, -t) + m * 1.9259629911266175e-8f;  // log2 e = kLog2e + 1.93e-8
  float w = fast_exp2(t);
  w = fmaf(w, rest * kLn2, w);
  const float u = 1.0f + w;
  return fmaxf(v, 0.0f) + (fast_log2(u) * kLn2 - ((u - 1.0f) - w));
}
// log2 of the smallest decay, of the parameter v
__device__ __forceinline__ float rate_of(float sharpness, float v) { return -sharpness * kLog2e * softplus_full(v); }

// ---- whole sequences
//
// A workgroup takes a chunk of 128 steps of a tile of channels, a wave 16 of the
// steps, a lane CPL channels.  What a stretch of steps does to the state is an affine
// map h -> P h + H: a wave forms that of its steps in registers, the workgroup
// composes its waves' over LDS and hands the chunk's map on in the workspace; with the state
// before its chunk a wave walks its steps again and writes.  So every input is read
// once and every output written once.
//
// The state before a chunk comes from the workgroups of the chunks before it, all of
// which have started: a workgroup draws its chunk of the tile from a counter.  (Loads
// for the chunk that it most likely is, before the draw is back, lose more when it is another
// than the draw's two microseconds: 3 x 1537 x 1000 fp32 backward 56 against 45 us.)  It
// waits for words that hold a value and say that they do, each published by one
// 64-bit store.  Every `group` chunks a state is published; in between a workgroup
// composes the maps of the chunks before its own since then, always in the same
// order, so that results do not depend on who was first.  A wait that is not served
// within about a second (a workspace written to meanwhile) ends with NaN.

// A value that is the same in all lanes, in a scalar register.
__device__ __forceinline__ int uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane((int)v); }

// A map whose P is minus zero has met a document's start: h -> H, whatever h is.
constexpr uint32_t kCleared = 0x80000000u;
struct Map {
  float p, h;
};
__device__ __forceinline__ bool cleared(float p) { return __float_as_uint(p) == kCleared; }
__device__ __forceinline__ float apply(const Map &m, float h) { return cleared(m.p) ? m.h : fmaf(m.p, h, m.h); }
// first, then m
__device__ __forceinline__ Map compose(const Map &first, const Map &m) { return cleared(m.p) ? m : Map{m.p * first.p, fmaf(m.p, first.h, m.h)}; }

struct Chain {
  uint32_t tiles, tiles_c;  // tiles of channels, of them a batch row's
  int chunks, groups, group;  // chunks per published state
  uint32_t *counter;        // one per tile, 64 bytes apart
  uint64_t *maps, *states;  // (tiles, chunks, tile's channels), (tiles, groups, tile's channels)
};

// Words: the upper half is not zero once the word holds something.
__device__ __forceinline__ void publish(uint64_t *p, uint32_t hi, float lo) {
  __hip_atomic_store(p, ((uint64_t)hi << 32) | __float_as_uint(lo), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish_map(uint64_t *p, const Map &m) { publish(p, (m.p != m.p ? 0x7fc00000u : __float_as_uint(m.p)) + 1, m.h); }
__device__ __forceinline__ uint64_t wait_word(const uint64_t *p) {
#pragma unroll 1
  for (int n = 0; n < (1 << 20); ++n) {
    const uint64_t v = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (v >> 32) return v;
    __builtin_amdgcn_s_sleep(1);
  }
  return 0x7fc000017fc00000ull;
}
__device__ __forceinline__ Map map_of(uint64_t v) { return {__uint_as_float((uint32_t)(v >> 32) - 1), __uint_as_float((uint32_t)v)}; }

// What lies between the last published state and chunk k (in the order of the
// walk), composed by the waves two words each; then, after a barrier, applied in order.
template <int CPL>
__device__ __forceinline__ void collect(const Chain &n, int64_t tile, int k, int w, int lane, const float (&first)[CPL], Map (*pre)[CPL][64]) {
  const int g = k / n.group, words = 1 + k - g * n.group;
  if (2 * w >= words) return;
#pragma unroll
  for (int q = 0; q < CPL; ++q) {
    Map m;
    const uint64_t *maps = n.maps + (tile * n.chunks + g * n.group) * (64 * CPL) + q * 64 + lane;
    if (w == 0) {
      const float h = g == 0 ? first[q] : __uint_as_float((uint32_t)wait_word(n.states + (tile * n.groups + g - 1) * (64 * CPL) + q * 64 + lane));
      m = {__uint_as_float(kCleared), h};
    } else {
      m = map_of(wait_word(maps + (int64_t)(2 * w - 1) * (64 * CPL)));
    }
    if (2 * w + 1 < words) m = compose(m, map_of(wait_word(maps + (int64_t)(2 * w) * (64 * CPL))));
    pre[w][q][lane] = m;
  }
}
template <int CPL>
__device__ __forceinline__ void collected(const Chain &n, int k, int lane, const Map (*pre)[CPL][64], float (&h)[CPL]) {
  const int words = 1 + k % n.group;
#pragma unroll
  for (int q = 0; q < CPL; ++q) {
    h[q] = pre[0][q][lane].h;
#pragma unroll 1
    for (int i = 1; 2 * i < words; ++i) h[q] = apply(pre[i][q][lane], h[q]);
  }
}

// A lane's channels of one step as they lie in memory, at a byte offset of a buffer.
// A buffer is the wave's steps of a tensor: an address is a base and a step's offset in
// scalar registers and the lane's offset in one vector register.  Loads stay inside by
// their offsets.  A store of a lane that has nothing to store takes kNoLane as the
// lane's offset, behind any buffer's end, and is dropped; the end is that of all
// kSteps steps, so that no step's offset lies behind it.
typedef __amdgpu_buffer_rsrc_t Buffer;
constexpr uint32_t kNoLane = 0x80000000u;
__device__ __forceinline__ Buffer buffer_of(const void *p, int64_t offset, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((char *)p + offset, 0, bytes, 0x00027000);
}
template <typename T, int CPL>
struct Raw;
template <>
struct Raw<float, 1> {
  uint32_t v;
  __device__ __forceinline__ void load(Buffer p, uint32_t lane, uint32_t step) { v = __builtin_amdgcn_raw_buffer_load_b32(p, lane, step, kStream); }
  __device__ __forceinline__ void get(float (&o)[1]) const { o[0] = __uint_as_float(v); }
  static __device__ __forceinline__ void put(Buffer p, uint32_t lane, uint32_t step, const float (&o)[1]) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(o[0]), p, lane, step, 0);
  }
};
template <>
struct Raw<bf16, 1> {
  uint16_t v;
  __device__ __forceinline__ void load(Buffer p, uint32_t lane, uint32_t step) { v = __builtin_amdgcn_raw_buffer_load_b16(p, lane, step, kStream); }
  __device__ __forceinline__ void get(float (&o)[1]) const { o[0] = __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ void put(Buffer p, uint32_t lane, uint32_t step, const float (&o)[1]) {
    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pack_bf16(o[0], o[0]), p, lane, step, 0);
  }
};
template <>
struct Raw<bf16, 2> {
  uint32_t v;
  __device__ __forceinline__ void load(Buffer p, uint32_t lane, uint32_t step) { v = __builtin_amdgcn_raw_buffer_load_b32(p, lane, step, kStream); }
  __device__ __forceinline__ void get(float (&o)[2]) const { o[0] = __uint_as_float(v << 16), o[1] = __uint_as_float(v & 0xffff0000u); }
  static __device__ __forceinline__ void put(Buffer p, uint32_t lane, uint32_t step, const float (&o)[2]) {
    __builtin_amdgcn_raw_buffer_store_b32(pack_bf16(o[0], o[1]), p, lane, step, 0);
  }
};

// Of the wave's steps, those before the end of the sequence.
__device__ __forceinline__ int rows_of(int t0, int L) { return L - t0 < 0 ? 0 : L - t0 < kSteps ? L - t0 : kSteps; }

// The wave's steps of a tensor, the sequence's last step again for those behind it; a
// step's stride and 16 of them stay below 2^29 bytes.
template <typename T, int CPL>
__device__ __forceinline__ void load_steps(const View3 &v, int D, int64_t b, int t0, int L, uint32_t lane_bytes, Raw<T, CPL> (&r)[kSteps]) {
  const int step = (int)v.st * (int)sizeof(T), from = t0 < L ? t0 : L - 1, last = (rows_of(from, L) - 1) * step;
  const Buffer p = buffer_of(v.p, (b * v.sb + from * v.st) * (int64_t)sizeof(T), last + D * (int)sizeof(T));
#pragma unroll
  for (int j = 0; j < kSteps; ++j) r[j].load(p, lane_bytes, j * step < last ? j * step : last);
}

// Bit j: a document starts at the wave's step j, before the row's length.
__device__ __forceinline__ uint32_t start_bits(const uint8_t *starts, int64_t b, int t0, int L, int len, int lane) {
  if (!starts) return 0;
  const bool on = lane < kSteps && t0 + lane < len && starts[b * L + t0 + lane] != 0;
  return (uint32_t)__ballot(on);
}

// MARKS: document starts or lengths of rows are given.
template <typename T, int CPL, bool POWER, bool IG, bool Z, bool MARKS>
__global__ void __launch_bounds__(64 * kWaves) recurrence_fwd_kernel(RecurrenceArgs a, Chain n) {
  __shared__ Map agg[kWaves][CPL][64], pre[kWaves][CPL][64];
  __shared__ int drawn;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const uint32_t tile32 = uniform(blockIdx.x % n.tiles), b32 = uniform(tile32 / n.tiles_c);
  const int64_t tile = tile32, b = b32;
  const int64_t c_lane = (int64_t)(tile32 - b32 * n.tiles_c) * (64 * CPL) + lane * CPL;
  const bool on = c_lane < a.D;
  const int64_t c = on ? c_lane : a.D - CPL;
  const uint32_t lane_bytes = (uint32_t)(c * sizeof(T));
  const bool chain = n.chunks > 1;
  const int D = (int)a.D, L = (int)a.L;  // (both below 2^30: a launch's workgroups)
  if (chain && threadIdx.x == 0) drawn = (int)atomicAdd(n.counter + tile * 16, 1u);
  float rate2[CPL];
#pragma unroll
  for (int q = 0; q < CPL; ++q) rate2[q] = POWER ? rate_of(a.sharpness, a.decay[c + q]) : 0.0f;
  int k = 0;
  if (chain) {
    __syncthreads();
    k = uniform(drawn);
    if ((uint32_t)k >= (uint32_t)n.chunks) return;  // (the workspace was written to meanwhile)
  }
  const int t0 = k * kRecurrenceChunk + w * kSteps;
  Raw<T, CPL> rx[kSteps], rg[kSteps], ri[kSteps], rz[kSteps];
  load_steps<T, CPL>(a.g, D, b, t0, L, lane_bytes, rg);
  if (IG) load_steps<T, CPL>(a.ig, D, b, t0, L, lane_bytes, ri);
  load_steps<T, CPL>(a.x, D, b, t0, L, lane_bytes, rx);
  if (Z) load_steps<T, CPL>(a.z, D, b, t0, L, lane_bytes, rz);
  const int len = MARKS ? uniform(row_length(a.lengths, b, L)) : L, nv = rows_of(t0, len);
  const uint32_t first = MARKS ? start_bits(a.starts, b, t0, L, len, lane) : 0;

  float da[kSteps][CPL], in[kSteps][CPL];
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    float g[CPL], x[CPL], i[CPL];
    rg[j].get(g);
    rx[j].get(x);
    if (IG) ri[j].get(i);
#pragma unroll
    for (int q = 0; q < CPL; ++q) {
      Gate t = gate_of<POWER>(g[q], rate2[q]);
      if (MARKS && (first >> j & 1)) t.a = 0.0f, t.s = 1.0f;
      da[j][q] = t.a;
      in[j][q] = t.s * (IG ? x[q] * sigmoid_f(i[q]) : x[q]);
    }
  }
  if (nv < kSteps)
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
      if (j >= nv)
#pragma unroll
        for (int q = 0; q < CPL; ++q) da[j][q] = 1.0f, in[j][q] = 0.0f;
#pragma unroll
  for (int q = 0; q < CPL; ++q) {
    Map m = {1.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      m.h = MARKS && (first >> j & 1) ? in[j][q] : fmaf(da[j][q], m.h, in[j][q]);
      m.p *= da[j][q];
    }
    if (MARKS && first) m.p = __uint_as_float(kCleared);
    agg[w][q][lane] = m;
  }
  float h0[CPL];  // the state before the first chunk
#pragma unroll
  for (int q = 0; q < CPL; ++q) h0[q] = a.state0 && k < n.group ? a.state0[b * a.D + c + q] : 0.0f;
  __syncthreads();
  Map before[CPL];  // what the waves before this one do
#pragma unroll
  for (int q = 0; q < CPL; ++q) {
    before[q] = {1.0f, 0.0f};
#pragma unroll 1
    for (int i = 0; i < w; ++i) before[q] = compose(before[q], agg[i][q][lane]);
  }
  const bool last = (k + 1) % n.group == 0, more = k + 1 < n.chunks;
  if (more && !last && w == kWaves - 1)
#pragma unroll
    for (int q = 0; q < CPL; ++q) publish_map(n.maps + (tile * n.chunks + k) * (64 * CPL) + q * 64 + lane, compose(before[q], agg[w][q][lane]));
  float h[CPL];
  if (chain) {
    collect<CPL>(n, tile, k, w, lane, h0, pre);
    __syncthreads();
    collected<CPL>(n, k, lane, pre, h);
  } else {
#pragma unroll
    for (int q = 0; q < CPL; ++q) h[q] = h0[q];
  }
  if (a.states && w == 0 && on)
#pragma unroll
    for (int q = 0; q < CPL; ++q) a.states[(b * n.chunks + k) * a.D + c + q] = h[q];
#pragma unroll
  for (int q = 0; q < CPL; ++q) {
    h[q] = apply(before[q], h[q]);
    if (w == kWaves - 1) {
      const float end = apply(agg[w][q][lane], h[q]);
      if (more && last) publish(n.states + (tile * n.groups + k / n.group) * (64 * CPL) + q * 64 + lane, 1, end);
      if (!more && a.state_final && on) a.state_final[b * a.D + c + q] = end;
    }
  }
  const int row = D * (int)sizeof(T);
  const Buffer y = buffer_of(a.y, (b * L + t0) * row, kSteps * row);
  const uint32_t out = on ? lane_bytes : kNoLane;
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    float o[CPL];
    if (Z) rz[j].get(o);
#pragma unroll
    for (int q = 0; q < CPL; ++q) {
      h[q] = MARKS && (first >> j & 1) ? in[j][q] : fmaf(da[j][q], h[q], in[j][q]);
      o[q] = Z ? h[q] * silu_f(o[q]) : h[q];
      if (MARKS && j >= nv) o[q] = 0.0f;
    }
    Raw<T, CPL>::put(y, t0 + j < L ? out : kNoLane, j * row, o);
  }
}

// Backward: the chunks in reverse, w_t = e_t + a_{t+1} w_{t+1}.  What flows from step t
// to t - 1 is q = a_t w_t, and a stretch of steps is q -> P q + Q with the P of the
// forward map.  The states inside a chunk are formed again from the one before it, its
// maps and those of the adjoint in one exchange.  For a step's gradients a lane keeps each
// gate's sigmoid and complement in one register (of the logistic form's decay 1 - a), and s in LDS:
//   log a da/d(log a) w (h_{t-1} - u a / s) = dLoss / d(log a) log a,  u = sigmoid(i) x.
template <typename T, bool POWER, bool IG, bool Z, bool MARKS>
__global__ void __launch_bounds__(64 * kWaves, 4) recurrence_bwd_kernel(RecurrenceArgs a, Chain n, float *part) {
  __shared__ Map agg[kWaves][1][64], pre[kWaves][1][64];
  __shared__ float back[kWaves][64];
  // of each lane's steps, what registers do not hold: s, and dy silu'(z)
  __shared__ float scale[POWER ? kWaves : 1][POWER ? kSteps : 1][64], gate_grad[Z ? kWaves : 1][Z ? kSteps : 1][64];
  __shared__ int drawn;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const uint32_t tile32 = uniform(blockIdx.x % n.tiles), b32 = uniform(tile32 / n.tiles_c);
  const int64_t tile = tile32, b = b32;
  const int64_t c_lane = (int64_t)(tile32 - b32 * n.tiles_c) * 64 + lane;
  const bool on = c_lane < a.D;
  const int64_t c = on ? c_lane : a.D - 1;
  const uint32_t lane_bytes = (uint32_t)(c * sizeof(T));
  const bool chain = n.chunks > 1;
  const int D = (int)a.D, L = (int)a.L;  // (both below 2^30: a launch's workgroups)
  if (chain && threadIdx.x == 0) drawn = (int)atomicAdd(n.counter + tile * 16, 1u);
  const float param = POWER ? a.decay[c] : 0.0f;
  const float rate2 = POWER ? rate_of(a.sharpness, param) : 0.0f, rate = kLn2 * rate2;
  int kr = 0;
  if (chain) {
    __syncthreads();
    kr = uniform(drawn);
    if ((uint32_t)kr >= (uint32_t)n.chunks) return;  // (the workspace was written to meanwhile)
  }
  const int k = n.chunks - 1 - kr, t0 = k * kRecurrenceChunk + w * kSteps;
  Raw<T, 1> rx[kSteps], rg[kSteps], ri[kSteps], rz[kSteps], rd[kSteps];
  load_steps<T, 1>(a.g, D, b, t0, L, lane_bytes, rg);
  if (IG) load_steps<T, 1>(a.ig, D, b, t0, L, lane_bytes, ri);
  load_steps<T, 1>(a.x, D, b, t0, L, lane_bytes, rx);
  load_steps<T, 1>(a.dy, D, b, t0, L, lane_bytes, rd);
  if (Z) load_steps<T, 1>(a.z, D, b, t0, L, lane_bytes, rz);
  const int len = MARKS ? uniform(row_length(a.lengths, b, L)) : L, nv = rows_of(t0, len);
  const uint32_t first = MARKS ? start_bits(a.starts, b, t0, L, len, lane) : 0;
  float h = a.states[(b * n.chunks + k) * a.D + c];

  // keep: the folded gate or 1 - a; ii: the folded input gate; steps behind the end: a = 1, nothing comes in
  float da[kSteps], keep[kSteps], in[kSteps], ii[kSteps], xs[kSteps], es[kSteps];
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    float g[1], v[1];
    rg[j].get(g);
    const Gate t = gate_of<POWER>(g[0], rate2);
    da[j] = t.a, keep[j] = t.keep;
    rx[j].get(v), xs[j] = v[0];
    rd[j].get(v), es[j] = v[0];
    if (Z) {
      float f, df;
      rz[j].get(v);
      silu_both(v[0], f, df);
      gate_grad[w][j][lane] = es[j] * df;
      es[j] *= f;
    }
    float i = 1.0f;
    ii[j] = 0.0f;
    if (IG) ri[j].get(v), i = sigmoid_folded(v[0], ii[j]);
    float s = t.s;
    // (at a start the gate is not used, whatever it holds)
    if (MARKS && (first >> j & 1)) da[j] = 0.0f, s = 1.0f, keep[j] = 0.0f;
    if (POWER) scale[w][j][lane] = s;
    in[j] = s * (i * xs[j]);
    if (j % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // (more steps at once do not fit registers)
  }
  if (nv < kSteps)
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
      if (j >= nv) da[j] = 1.0f, keep[j] = in[j] = ii[j] = xs[j] = es[j] = 0.0f;
  Map m = {1.0f, 0.0f};
  float q = 0.0f;
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    m.h = MARKS && (first >> j & 1) ? in[j] : fmaf(da[j], m.h, in[j]);
    m.p *= da[j];
  }
#pragma unroll
  for (int j = kSteps - 1; j >= 0; --j) q = MARKS && (first >> j & 1) ? 0.0f : da[j] * (es[j] + q);
  if (MARKS && first) m.p = __uint_as_float(kCleared);
  agg[w][0][lane] = m;
  back[w][lane] = q;
  const float q0[1] = {a.dstate_final && kr < n.group ? a.dstate_final[b * a.D + c] : 0.0f};
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < w; ++i) h = apply(agg[i][0][lane], h);
  Map after = {1.0f, 0.0f};  // what the waves behind this one do
#pragma unroll 1
  for (int i = kWaves - 1; i > w; --i) after = compose(after, Map{agg[i][0][lane].p, back[i][lane]});
  const bool last = (kr + 1) % n.group == 0, more = kr + 1 < n.chunks;
  if (more && !last && w == 0) publish_map(n.maps + (tile * n.chunks + kr) * 64 + lane, compose(after, Map{m.p, q}));
  float from[1] = {q0[0]};
  if (chain) {
    collect<1>(n, tile, kr, w, lane, q0, pre);
    __syncthreads();
    collected<1>(n, kr, lane, pre, from);
  }
  q = apply(after, from[0]);
  if (w == 0) {
    const float end = apply(Map{m.p, back[0][lane]}, q);
    if (more && last) publish(n.states + (tile * n.groups + kr / n.group) * 64 + lane, 1, end);
    if (!more && a.dstate0 && on) a.dstate0[b * a.D + c] = end;
  }
  // in[j] becomes the state before step j
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const float next = MARKS && (first >> j & 1) ? in[j] : fmaf(da[j], h, in[j]);
    in[j] = h;
    h = next;
  }
  const int row = D * (int)sizeof(T), rows_bytes = kSteps * row;
  const int64_t row0 = (b * L + t0) * row;
  const Buffer bx = buffer_of(a.dx, row0, rows_bytes), bg = buffer_of(a.dg, row0, rows_bytes), bi = buffer_of(a.dig, row0, rows_bytes);
  const Buffer bz = buffer_of(a.dz, row0, rows_bytes);
  const uint32_t out = on ? lane_bytes : kNoLane;
  float sum = 0.0f;
#pragma unroll
  for (int j = kSteps - 1; j >= 0; --j) {
    const bool start = MARKS && (first >> j & 1);
    float dz[1] = {Z ? gate_grad[w][j][lane] * h : 0.0f};
    h = in[j];
    float i = 1.0f, di_v = 0.0f;
    if (IG) unfold(ii[j], i, di_v);
    const float wt = es[j] + q, flow = wt * da[j], u = i * xs[j];
    const float s = POWER ? scale[w][j][lane] : start ? 1.0f : keep[j], ws = wt * s;
    float dx[1] = {ws * i}, di[1] = {ws * (xs[j] * di_v)}, dg[1];
    if constexpr (POWER) {
      // (a step behind the row's length has no part in ddecay, not even 0 times a state that is not finite)
      float r, dr;
      unfold(keep[j], r, dr);
      const float f = start || (MARKS && j >= nv) ? 0.0f : flow * rate * fmaf(-u * da[j], s > 0.0f ? fast_rcp(s) : 0.0f, h);
      sum = fmaf(f, r, sum);
      dg[0] = f * dr;
    } else {
      dg[0] = start ? 0.0f : flow * s * (h - u);
    }
    q = start ? 0.0f : flow;
    if (MARKS && j >= nv) dx[0] = dg[0] = di[0] = dz[0] = 0.0f;
    const uint32_t to = t0 + j < L ? out : kNoLane;
    Raw<T, 1>::put(bx, to, j * row, dx);
    Raw<T, 1>::put(bg, to, j * row, dg);
    if (IG) Raw<T, 1>::put(bi, to, j * row, di);
    if (Z) Raw<T, 1>::put(bz, to, j * row, dz);
  }
  if constexpr (POWER) {  // the chunk's part of ddecay, waves in order
    __syncthreads();
    back[w][lane] = sum;
    __syncthreads();
    if (w == 0 && on) {
      sum = 0.0f;
      for (int i = 0; i < kWaves; ++i) sum += back[i][lane];
      // sigmoid / softplus goes to 1 where both vanish
      part[(b * n.chunks + k) * a.D + c] = sum * (param < -40.0f ? 1.0f : sigmoid_f(param) / softplus_full(param));
    }
  }
}

__global__ void __launch_bounds__(256) recurrence_clear_kernel(uint4 *p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = make_uint4(0, 0, 0, 0);
}

// One token: 4 channels per lane.
template <typename T, bool POWER>
__global__ void __launch_bounds__(256) recurrence_update_kernel(RecurrenceUpdateArgs a) {
  const uint32_t n4 = (uint32_t)(a.D / 4), i4 = blockIdx.x * 256 + threadIdx.x;  // (fewer than 2^32 threads)
  if (i4 >= a.B * n4) return;
  const int64_t b = i4 / n4, c = i4 % n4 * 4;
  float x[4], g[4], i[4], z[4], h[4], l[4];
  load_vec((const T *)a.x.p + b * a.x.sb + c, x);
  load_vec((const T *)a.g.p + b * a.g.sb + c, g);
  if (a.ig.p) load_vec((const T *)a.ig.p + b * a.ig.sb + c, i);
  if (a.z.p) load_vec((const T *)a.z.p + b * a.z.sb + c, z);
  if (POWER) load_vec(a.decay + c, l);
  load_vec(a.state + b * a.D + c, h);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const Gate q = gate_of<POWER>(g[j], POWER ? rate_of(a.sharpness, l[j]) : 0.0f);
    h[j] = fmaf(q.a, h[j], q.s * (a.ig.p ? x[j] * sigmoid_f(i[j]) : x[j]));
    x[j] = a.z.p ? h[j] * silu_f(z[j]) : h[j];
  }
  store_vec(a.state + b * a.D + c, h);
  store_vec((T *)a.y + b * a.D + c, x);
}

template <int X>
struct Int {
  static constexpr int v = X;
};
// Calls f with the four switches as integral constants.
template <typename F>
hipError_t by_switches(bool power, bool ig, bool z, bool marks, F f) {
  auto m = [&](auto p, auto i, auto zz) { return marks ? f(p, i, zz, Int<1>{}) : f(p, i, zz, Int<0>{}); };
  auto l = [&](auto p, auto i) { return z ? m(p, i, Int<1>{}) : m(p, i, Int<0>{}); };
  auto o = [&](auto p) { return ig ? l(p, Int<1>{}) : l(p, Int<0>{}); };
  return power ? o(Int<1>{}) : o(Int<0>{});
}

// cpl: channels per lane, es: bytes of an element
Chain chain_of(int64_t B, int64_t L, int64_t D, int cpl, int es, void *workspace) {
  Chain n;
  n.tiles_c = (uint32_t)((D + 64 * cpl - 1) / (64 * cpl));
  n.tiles = (uint32_t)B * n.tiles_c;
  n.chunks = (int)((L + kRecurrenceChunk - 1) / kRecurrenceChunk);
  n.group = group_of(B, L, D, es);
  n.groups = (n.chunks + n.group - 1) / n.group;
  n.counter = (uint32_t *)workspace;
  n.states = (uint64_t *)((char *)workspace + (int64_t)n.tiles * 64);
  n.maps = n.states + (int64_t)n.tiles * n.groups * 64 * cpl;
  return n;
}
int64_t chain_bytes(const Chain &n, int cpl) {
  return n.chunks == 1 ? 0 : (int64_t)n.tiles * (64 + (int64_t)(n.groups + (n.group > 1 ? n.chunks : 0)) * 64 * cpl * 8);
}
hipError_t clear(void *p, int64_t bytes, hipStream_t s) {
  const int64_t n = bytes / 16, grid = (n + 255) / 256;
  hipLaunchKernelGGL(recurrence_clear_kernel, dim3((unsigned)(grid < 2048 ? grid : 2048)), dim3(256), 0, s, (uint4 *)p, n);
  return hipGetLastError();
}

template <typename T, int CPL>
hipError_t fwd(const RecurrenceArgs &a, hipStream_t s) {
  const Chain n = chain_of(a.B, a.L, a.D, CPL, sizeof(T), a.workspace);
  if (n.chunks > 1) {
    const hipError_t e = clear(a.workspace, chain_bytes(n, CPL), s);
    if (e != hipSuccess) return e;
  }
  return by_switches(a.decay, a.ig.p, a.z.p, a.starts || a.lengths, [&](auto p, auto i, auto z, auto m) {
    hipLaunchKernelGGL((recurrence_fwd_kernel<T, CPL, decltype(p)::v, decltype(i)::v, decltype(z)::v, decltype(m)::v>), dim3(n.tiles * n.chunks),
                       dim3(64 * kWaves), 0, s, a, n);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t bwd(const RecurrenceArgs &a, hipStream_t s) {
  const Chain n = chain_of(a.B, a.L, a.D, 1, sizeof(T), a.workspace);
  const int64_t bytes = chain_bytes(n, 1);
  float *part = (float *)((char *)a.workspace + bytes);
  if (n.chunks > 1) {
    const hipError_t e = clear(a.workspace, bytes, s);
    if (e != hipSuccess) return e;
  }
  const hipError_t e = by_switches(a.decay, a.ig.p, a.z.p, a.starts || a.lengths, [&](auto p, auto i, auto z, auto m) {
    hipLaunchKernelGGL((recurrence_bwd_kernel<T, decltype(p)::v, decltype(i)::v, decltype(z)::v, decltype(m)::v>), dim3(n.tiles * n.chunks),
                       dim3(64 * kWaves), 0, s, a, n, part);
    return hipGetLastError();
  });
  return e == hipSuccess && a.decay ? launch_sum_rows(part, a.B * n.chunks, a.D, a.D, a.ddecay, nullptr, s) : e;
}

template <typename T>
hipError_t update(const RecurrenceUpdateArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.B * (a.D / 4) + 255) / 256));
  if (a.decay)
    hipLaunchKernelGGL((recurrence_update_kernel<T, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((recurrence_update_kernel<T, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

int64_t recurrence_fwd_workspace_bytes(int64_t B, int64_t L, int64_t D, int io_dtype) {
  const int cpl = io_dtype == 0 ? 1 : 2;
  return chain_bytes(chain_of(B, L, D, cpl, io_dtype == 0 ? 4 : 2, nullptr), cpl);
}
int64_t recurrence_bwd_workspace_bytes(int64_t B, int64_t L, int64_t D, int io_dtype) {
  const Chain n = chain_of(B, L, D, 1, io_dtype == 0 ? 4 : 2, nullptr);
  return chain_bytes(n, 1) + B * n.chunks * D * 4;
}

hipError_t launch_recurrence_fwd(const RecurrenceArgs &a, int io_dtype, hipStream_t s) {
  return io_dtype == 0 ? fwd<float, 1>(a, s) : fwd<bf16, 2>(a, s);
}
hipError_t launch_recurrence_bwd(const RecurrenceArgs &a, int io_dtype, hipStream_t s) {
  return io_dtype == 0 ? bwd<float>(a, s) : bwd<bf16>(a, s);
}
hipError_t launch_recurrence_update(const RecurrenceUpdateArgs &a, int io_dtype, hipStream_t s) {
  return io_dtype == 0 ? update<float>(a, s) : update<bf16>(a, s);
}

}  // namespace ssm
