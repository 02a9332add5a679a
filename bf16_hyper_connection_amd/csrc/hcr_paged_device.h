// Device helpers of the paged cache's kernels: which sequence a row of the batch belongs to.
#pragma once

#include "hcr_device.h"
#include "hcr_paged_layout.h"

namespace hcr {

// A sequence, the same for the whole wave.  Its three numbers are loaded together: the compiler would put each load
// behind the checks of the one before, three waits instead of one (about 1 us of a call).
__device__ __forceinline__ Seq wave_seq(const BatchArgs& b, int i) {
  int s0 = __builtin_amdgcn_readfirstlane(b.q_start[i]), s1 = __builtin_amdgcn_readfirstlane(b.q_start[i + 1]);
  int ctx = __builtin_amdgcn_readfirstlane(b.ctx_len[i]);
  asm volatile("" : "+s"(s0), "+s"(s1), "+s"(ctx));
  return seq_of(b, s0, s1, ctx);
}
// The sequences 64 at a time, one per lane.
__device__ __forceinline__ Seq lane_seq(const BatchArgs& b, int first, int lane) {
  const int i = min(first + lane, b.n_seqs - 1);
  int s0 = b.q_start[i], s1 = b.q_start[i + 1], ctx = b.ctx_len[i];
  asm volatile("" : "+v"(s0), "+v"(s1), "+v"(ctx));
  return seq_of(b, first + lane < b.n_seqs ? s0 : -1, s1, ctx);
}
__device__ __forceinline__ Seq of_lane(const Seq& s, int l) {
  return Seq{__builtin_amdgcn_readlane(s.row, l), __builtin_amdgcn_readlane(s.tokens, l),
             __builtin_amdgcn_readlane(s.first, l)};
}

// The sequence that row `row` of the batch belongs to and its token among the sequence's new ones (b < 0: none).
struct RowOf {
  Seq seq;
  int b, token;
};
__device__ __forceinline__ RowOf seq_of_row(const BatchArgs& b, int row, int lane) {
  // 64 first rows at a time, of every 4,096th sequence, then of every 64th: they ascend
  int i = 0, step = 1;
  while ((long long)step * 64 < b.n_seqs) step *= 64;
  for (; step > 1; step /= 64) {
    const long long at = i + (long long)lane * step;
    const unsigned long long upto = __ballot(at < b.n_seqs && b.q_start[min(at, (long long)b.n_seqs - 1)] <= row);
    if (upto) i += (63 - __clzll(upto)) * step;
  }
  const Seq s = lane_seq(b, i, lane);
  const unsigned long long at = __ballot(row >= s.row && row < s.row + s.tokens);
  if (!at) return RowOf{Seq{0, 0, 0}, -1, 0};
  const int l = __ffsll(at) - 1;
  const Seq q = of_lane(s, l);
  return RowOf{q, i + l, row - q.row};
}

}  // namespace hcr
