// mixer_plans.hpp -- how the gated recurrence, the causal convolution and the norm and
// rotation of heads are split over workgroups: host arithmetic on sizes alone, without
// HIP, so that it can be read and checked by itself.
#pragma once

#include <stdint.h>

namespace ssm {

constexpr int kRecurrenceChunk = 128;  // SSM_RECURRENCE_CHUNK

namespace recurrence {

constexpr int kWaves = 8, kSteps = 16;
static_assert(kWaves * kSteps == kRecurrenceChunk, "a wave takes kSteps steps of a chunk");
constexpr int kMaxGroup = 2 * kWaves;  // two words per wave: a state and the maps of 15 chunks

// Chunks per published state.  A state's way from one workgroup to the next takes
// about 1.25 us, and the maps between states are words to read in every workgroup
// behind: as few maps as keep the states' way through the sequence below 2/5 of the
// time that the tensors need (x, both gates and y at 4 TB/s).
inline int group_of(int64_t B, int64_t L, int64_t D, int es) {
  const double us = (double)(B * L) * (double)(4 * D * es) / 4e6, way = (double)((L + kRecurrenceChunk - 1) / kRecurrenceChunk) * 1.25;
  int g = 1;
  while (g < kMaxGroup && way > 0.4 * us * g) g *= 2;
  return g;
}

}  // namespace recurrence

namespace conv {

constexpr int kRows = 8;  // rows whose loads are under way together
constexpr int kBwdRows = 120;  // at most: two words of starts of documents, offsets below 2^32 bytes

// Steps per wave and chunk, from 16 to kBwdRows: the workgroups that are resident at
// once (four of four waves per CU in bf16, three in fp32) take equal numbers of chunks, and
// the fewest steps in all are walked over, with the K-1 that a chunk shares with the next
// and about 6 for its start (8 x 2048 x 2048 bf16 packed: 58 us with 64 steps, of which
// 1088 workgroups are not all resident).
struct BwdPlan {
  int64_t ctiles, nchunk, nruns;
  int nrow;
};
inline BwdPlan bwd_plan(int64_t B, int64_t L, int64_t D, int width, int es) {
  const int64_t ctiles = (D + 127) / 128, resident = es == 2 ? 1024 : 768, most = ctiles < resident ? resident / ctiles : 1;
  BwdPlan best{};
  int64_t least = -1;
  for (int nrow = 16; nrow <= kBwdRows; nrow += kRows) {
    const int64_t nchunk = (L + nrow - width) / (nrow - width + 1), need = (B * nchunk + 3) / 4, each = (need + most - 1) / most;
    if (least < 0 || each * (nrow + 6) < least) least = each * (nrow + 6), best = {ctiles, nchunk, (need + each - 1) / each, nrow};
  }
  return best;
}

}  // namespace conv

namespace heads {

constexpr int kThreads = 256;
constexpr int kMaxTable = 2048;  // angles in LDS
// Rows of a group between two fillings of the table: few start sooner and leave more workgroups to
// even out (8 x 2048, 32 and 4 heads of 64 bf16: forward 41 -> 39 us with 4 for 8, backward 62 -> 56; 16 and 16
// of 128 fp32 backward 135 -> 130, interleaved forward 104 -> 96; 32K context backward 244 -> 236), but one
// token at a time in the bf16 forward waits for each filling (40 and 8 heads of 128 176 against 172, 16 and
// 16 interleaved 56 against 52; two rows lose 2 to 20% nearly everywhere).
constexpr int max_rows(bool bwd, int es, int tpr) { return !bwd && es == 2 && tpr >= 16 ? 8 : 4; }

struct Plan {
  int tpr, nblk, hb, tsub, rows;  // lanes per head, blocks of heads, heads per block, tokens at once, rows per group of a chunk of tokens
  int64_t nchunk, nruns;
};

constexpr int64_t kFwdWorkgroups = 65536, kBwdWorkgroups = 1024;

inline int64_t most_runs(int nblk, int64_t workgroups) { return nblk < workgroups ? workgroups / nblk : 1; }

inline int lanes_of(int d) { return d <= 32 ? 4 : d <= 64 ? 8 : d <= 128 ? 16 : 32; }
inline int least_blocks(int HT, int tpr) { return (HT + kThreads / tpr - 1) / (kThreads / tpr); }
constexpr int kMoreBlocks = 8;

inline Plan plan_of(int64_t B, int64_t L, int HT, int d, int rot, bool bwd, int es) {
  const int64_t workgroups = bwd ? kBwdWorkgroups : kFwdWorkgroups;
  Plan p;
  p.tpr = lanes_of(d);
  // Blocks of heads: few, since each forms the angles of its tokens, and so that few groups
  // of lanes are left over.  Per token: a row is about 120 instructions of a lane, an
  // angle 50 of one of the workgroup's lanes (36 heads of 64 on 32 groups in 5 blocks of 8
  // heads and 4 tokens, not in 2 of 18 and one).
  const int groups = kThreads / p.tpr;
  double least = 0.0;
  for (int nblk = least_blocks(HT, p.tpr); nblk <= HT && nblk <= least_blocks(HT, p.tpr) + kMoreBlocks; ++nblk) {
    const int hb = (HT + nblk - 1) / nblk, tsub = groups / hb;
    const double cost = 120.0 * nblk / tsub + 50.0 * nblk * (rot / 2) / kThreads;
    if (least == 0.0 || cost < least) least = cost, p.nblk = (HT + hb - 1) / hb, p.hb = hb, p.tsub = tsub;
  }
  p.rows = max_rows(bwd, es, p.tpr);
  while (p.rows > 1 && (p.tsub * p.rows * (rot / 2) > kMaxTable)) p.rows /= 2;
  const int64_t tt = p.tsub * p.rows;
  p.nchunk = B * ((L + tt - 1) / tt);
  const int64_t most = most_runs(p.nblk, workgroups);
  p.nruns = p.nchunk < most ? p.nchunk : most;
  return p;
}

// The largest that any rotation, any strides and either kind of weights of these sizes need.
inline int64_t bwd_workspace_bytes(int64_t B, int64_t L, int64_t Hq, int64_t Hk, int64_t d) {
  const int64_t HT = Hq + Hk, N = B * L, few = least_blocks((int)HT, lanes_of((int)d)), many = few + kMoreBlocks;
  const int64_t runs = most_runs((int)few, kBwdWorkgroups), per_head = (N < runs ? N : runs) * HT;
  const int64_t all = many < kBwdWorkgroups ? kBwdWorkgroups : many, shared = 2 * (N < all / many ? N * many : all);
  return (per_head > shared ? per_head : shared) * d * 4;
}

}  // namespace heads

}  // namespace ssm
