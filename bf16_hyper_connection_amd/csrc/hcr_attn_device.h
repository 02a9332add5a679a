// Attention of a decode window over the paged cache, gfx950 (MI355X):
//   out[n] = sum_p softmax_p(scale q[n] . k[p]) v[p],   p <= the token's position
// for every page of a sequence, for the pages listed per token and kv head, or through a window (SEEN), over pages of
// BF16 or of 8-bit codes (CODE).
//
// A unit is one kv head of one sequence: its rows are the T x G (tokens x heads of the group) query rows, which
// all read the same keys and values.  A wave takes tiles of 32 positions and holds 16 or 32 of the rows:
//   S^T = K Q^T : A = 16 keys (two row tiles per 32 positions), B = 16 query rows; S^T arrives with one query row
//                 per lane column, so a row's maximum and sum run over a lane's 8 values and the 4 lane rows.
//   O^T += V^T P^T : the K index of this product is a position.  Row r of key tile t is position
//                 8 (r / 4) + 4 t + r % 4, so the 8 probabilities that a lane holds after S^T are 8 consecutive
//                 positions, its B operand as they are; the value pages keep 8 positions of a dimension in 16
//                 bytes, its A operand as loaded.  Nothing goes through LDS inside the loop.
// Probabilities are powers of two against a running maximum that moves only when a tile passes it by 2^8 (sums
// and products are FP32, so the offset costs no precision), split into BF16 parts: two (2^-17) for BF16 outputs,
// three (the whole FP32 value) for float ones, where two would be the largest error of all (2^-18 of a probability, up
// to 3.8e-6; the third costs matrix products that the loop has time for).
//
// Codes are widened to BF16, which holds each exactly, on their way into the matrix cores; a key's scale multiplies its
// product, a value's scale its probability ahead of the split:
//   out = sum_p softmax_p(scale sk[p] (q . ck[p])) sv[p] cv[p]
// so that scales cost a multiplication a product and no code is ever rounded again.  16 bytes of a page are 16 codes, two
// operands: a lane's key loads hold 16 dimensions of a key, its value loads the 16 positions whose products it has (tiles
// of 64 positions, rows 16 (r / 4) + 4 t + r % 4; of D = 256, whose accumulators leave no room, 8 positions in 8 bytes).
//
// Through a window a row sees [0, first) and [len - size, len).  Tiles that no row sees are not visited; in a tile that
// some rows see in part, what a row does not see is hidden by bit masks ahead of its maximum (a product there may be
// anything) and, of values, ahead of the product.
//
// Work: the tiles of all sequences, one behind the other, are cut into equal runs, one for each work-group that the
// chip holds at once (AttnPlan), so that unlike lengths and loose bounds cost nothing; a run goes from one sequence
// on to the next.  The waves of a work-group take its tiles in turn and join in LDS; sequences that lie in several
// runs are joined by a second launch; each join is (m, l, O) -> (max, sum of l 2^(m - max), sum of O 2^(m - max)),
// in a fixed order.  Where the chip is full of sequences or they are short, a work-group takes a whole one instead and
// nothing is left to join (there a long one among short ones, or a bound far above them, does cost: the plan's rule
// keeps that to sequences of 4,096).  Where prompts and single tokens share a batch, the pairs of a sequence and a row
// block are cut, as many as the device finds, in place of each row block's sequences (pair_cut).
//
// Bound by the bytes of keys and values.  Measured on MI355X (graphs of calls, inputs rotated): one sequence of
// 420,000 positions, 48 heads of 256 over 8, 2 tokens: 505 us, 6.8 TB/s (a 4 GiB device copy moves 4.8); 64 sequences
// of 1,000 to 8,192, 32 heads of 128 over 8: 194 us, 6.2 TB/s.  36 rows of 4 sequences of up to 9,001: 51 us, 3.3 TB/s:
// a work-group has 10 tiles behind 6 us of first loads, three row waves share each of them, so that a CU has 64 KB on
// their way where it has 256 KB with one row wave, and the second launch takes 7.  (Rows past 16 over codes and windows
// go to hcr_attn_rows.h.)
// Codes, the same calls: 420,000 positions (E4M3, float outputs) 273 us, 6.4 TB/s; 64 sequences (int8) 116 us, 5.4 TB/s;
// one of 700 positions 10.0 us, mostly waits for first loads, one behind the other (lengths, table, keys).  64 windows
// of 4,096 of BF16 165 us, 6.5 TB/s.
// Not taken: tiles of 32 for codes of D = 128 with 16 waves (batch 143 us where whole sets took 108, short call 11.8), tiles of 64 for D = 256 (25
// registers spilled), two to four row tiles a wave over codes (36 rows of D = 256 130 to 190 us where four waves that
// share them take 115: past 256 registers each use is a copy).

#pragma once

#include <float.h>
#include <math.h>
#include <type_traits>
#include <hip/hip_runtime.h>

#include "hcr_paged_device.h"

namespace hcr {

// Which positions a row sees: all up to its own, those of the listed pages, those of a sliding window and the first
// ones.
enum Seen { DENSE, LISTED, WINDOW };

// What pages hold, and the tile that one wave takes at a time.
template <int CODE, int D>
struct Format {
  static constexpr bool CODED = CODE != HCR_BF16;
  static constexpr int SHIFT = tile_shift(CODED, D);
  static constexpr int TILE = 1 << SHIFT;
  static constexpr int BYTES = CODED ? 1 : 2;   // of a value
  static constexpr int HALVES = CODED ? 2 : 1;  // operands in 16 bytes of keys
  static constexpr int KT = TILE / 16;          // tiles of 16 keys
  static constexpr int EACH = TILE / 4;         // positions of a lane: its products, its bytes of values / BYTES
};

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;

__device__ __forceinline__ bf16x8 as_bf16x8(const uint4& u) { return __builtin_bit_cast(bf16x8, u); }
__device__ __forceinline__ uint4 ld16(const void* p) { return *static_cast<const uint4*>(p); }
// Keys and values: past the caches where nobody else reads them (ONCE).  Measured on MI355X: 64 sequences of up to
// 8,192 positions 193 against 215 us, 420,000 positions 529 against 590; with three row waves on the same tiles 62
// against 51.
template <bool ONCE>
__device__ __forceinline__ uint4 ld_kv(const void* p) {
  if constexpr (ONCE) return ldw16(p);
  return ld16(p);
}
template <bool ONCE>
__device__ __forceinline__ uint2 ld_kv8(const void* p) {
  if constexpr (ONCE) return ldw8(p);
  return *static_cast<const uint2*>(p);
}
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// The larger of each value over the 4 lane rows (lanes l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float rows_max(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float rows_sum(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// What the high and low BF16 parts of 8 values leave of them, as BF16.
__device__ __forceinline__ uint4 split_rest(const float (&v)[8], const uint4& hi, const uint4& lo) {
  const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
  uint32_t r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f32x2 x = {v[2 * e], v[2 * e + 1]};
    x -= f32x2{__uint_as_float(h[e] << 16), __uint_as_float(h[e] & 0xFFFF0000u)};  // exact, twice
    x -= f32x2{__uint_as_float(l[e] << 16), __uint_as_float(l[e] & 0xFFFF0000u)};
    r[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ uint2 split_rest4(const f32x4& v, const uint2& hi, const uint2& lo) {
  const uint32_t h[2] = {hi.x, hi.y}, l[2] = {lo.x, lo.y};
  uint32_t r[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    f32x2 x = {v[2 * e], v[2 * e + 1]};
    x -= f32x2{__uint_as_float(h[e] << 16), __uint_as_float(h[e] & 0xFFFF0000u)};
    x -= f32x2{__uint_as_float(l[e] << 16), __uint_as_float(l[e] & 0xFFFF0000u)};
    r[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
  }
  return make_uint2(r[0], r[1]);
}

__device__ __forceinline__ void store4(void* out, int type, size_t at, const f32x4& v) {
  if (type == HCR_F32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + at) = v;
  } else {
    const f32x2 a = {v[0], v[1]}, b = {v[2], v[3]};
    uint2 u;
    u.x = __builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2));
    u.y = __builtin_bit_cast(uint32_t, __builtin_convertvector(b, bf16x2));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = u;
  }
}

// A barrier for LDS alone: loads on their way to registers stay on their way.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The rows of a set that a work-group takes, and which positions they see: [0, len), through a window [start, len)
// and [0, firsts).
template <int SEEN>
struct Rows {
  int first, count;      // of the set's rows; the work-group's first one, the set's number
  int len_min, len_max;  // of the work-group's rows
  int start_min, start_max;
  __device__ __forceinline__ Rows(const AttnArgs& a, const Seq& seq, int token, int rb) {
    constexpr bool one = SEEN == LISTED;
    first = rb * attn_rows(a.plan);
    count = one ? a.group : seq.tokens * a.group;
    const int last = min(first + attn_rows(a.plan), count) - 1;
    len_min = seq.first + (one ? token : first / a.group) + 1;
    len_max = seq.first + (one ? token : last / a.group) + 1;
    start_min = SEEN == WINDOW ? max(len_min - a.window.size, 0) : 0;
    start_max = SEEN == WINDOW ? max(len_max - a.window.size, 0) : 0;
  }
  // Whether each of the rows sees all of n positions from p on.
  __device__ __forceinline__ bool all_see(const AttnArgs& a, int p, int n) const {
    return p + n <= len_min && (SEEN != WINDOW || p >= start_max || p + n <= a.window.first);
  }
};

// Tiles of a sequence, for row block rb through a window.
template <int SEEN, int SHIFT>
struct Count {
  const AttnArgs& a;
  const int low, high;  // the row block's first token, and its last
  __device__ __forceinline__ Count(const AttnArgs& a_, int rb)
      : a(a_), low(SEEN == WINDOW ? rb * attn_rows(a_.plan) / a_.group : 0),
        high(SEEN == WINDOW ? ((rb + 1) * attn_rows(a_.plan) - 1) / a_.group : 0) {}
  __device__ __forceinline__ int operator()(const Seq& s) const {
    if (SEEN == WINDOW) {
      const int tiles =
          window_tiles(a.window, s.first + low + 1, s.first + min(high, s.tokens - 1) + 1, SHIFT).tiles;
      return low < s.tokens ? tiles : 0;
    }
    return s.tokens ? max(ceil_div(s.first + s.tokens, 1 << SHIFT), 1) : 0;
  }
};
// Inclusive prefix sum over the first n lanes.
__device__ __forceinline__ int lane_prefix(int v, int lane, int n) {
  for (int o = 1; o < min(n, 64); o *= 2) {
    const int y = __shfl_up(v, o);
    if (lane >= o) v += y;
  }
  return v;
}
// A set of rows among the tiles of all: its sequence and token (listed pages), its tiles [first, first + tiles).
struct Set {
  Seq seq;
  int b, token, first, tiles;  // b < 0: none
};
// How the call's tiles are cut: runs of `run` tiles, each set in runs of its own (`apart`) or not.
struct Cut {
  int run;
  bool apart;
};
// The sequence that run x begins in (x < 0: the one that row `row` belongs to).
template <class C>
__device__ __forceinline__ Set find_seq(const BatchArgs& b, int x, int row, int lane, const AttnPlan& p,
                                        const C& tiles_of, Cut* cut) {
  const int B = b.n_seqs;
  const Seq s0 = lane_seq(b, 0, lane);
  const int n0 = tiles_of(s0);
  int upto0 = lane_prefix(n0, lane, B);
  int all = __builtin_amdgcn_readlane(upto0, min(B, 64) - 1);
  for (int i = 64; i < B; i += 64) {
    const int t = lane_prefix(tiles_of(lane_seq(b, i, lane)), lane, B - i);
    all += __builtin_amdgcn_readlane(t, min(B - i, 64) - 1);
  }
  *cut = Cut{run_tiles(p, all), false};
  if (B <= 64) {  // the sequences' runs counted, once or twice
    int run = cut->run;
    int runs = ceil_div(n0, run), upto = lane_prefix(runs, lane, B);
    bool fits = __builtin_amdgcn_readlane(upto, B - 1) <= p.items;
    if (!fits) {
      run = run_tiles_apart(p, all, B);
      fits = run > 0;
      if (fits) {
        runs = ceil_div(n0, run);
        upto = lane_prefix(runs, lane, B);
      }
    }
    if (fits) {
      *cut = Cut{run, true};
      const bool mine = x >= 0 ? upto - runs <= x && x < upto : row >= s0.row && row < s0.row + s0.tokens;
      const unsigned long long at = __ballot(mine);
      if (!at) return Set{Seq{0, 0, 0}, -1, 0, 0, 0};
      const int l = __ffsll(at) - 1;
      return Set{of_lane(s0, l), l, 0, __builtin_amdgcn_readlane(upto - runs, l) * run,
                 __builtin_amdgcn_readlane(n0, l)};
    }
  }
  const int tile = x * cut->run;
  int before = 0;
  for (int i = 0; i < B; i += 64) {
    const Seq s = i == 0 ? s0 : lane_seq(b, i, lane);
    const int n = i == 0 ? n0 : tiles_of(s);
    const int upto = i == 0 ? upto0 : before + lane_prefix(n, lane, B - i);
    const bool mine = x >= 0 ? upto - n <= tile && tile < upto : row >= s.row && row < s.row + s.tokens;
    const unsigned long long at = __ballot(mine);
    if (at) {
      const int l = __ffsll(at) - 1;
      return Set{of_lane(s, l), i + l, 0, __builtin_amdgcn_readlane(upto - n, l), __builtin_amdgcn_readlane(n, l)};
    }
    before = __builtin_amdgcn_readlane(upto, min(B - i, 64) - 1);
  }
  return Set{Seq{0, 0, 0}, -1, 0, 0, 0};
}
// A sequence's set where no other is counted.
template <class C>
__device__ __forceinline__ Set seq_set(const BatchArgs& b, int i, const C& tiles_of) {
  const Seq q = wave_seq(b, i);
  return Set{q, q.tokens ? i : -1, 0, 0, tiles_of(q)};
}
// Listed pages: every token's list in `runs` runs of `run` tiles, whole ones as one.
template <int SHIFT>
struct Lists {
  int tiles, run, runs;
  __device__ __forceinline__ explicit Lists(const AttnArgs& a)
      : tiles(a.n_sel << (a.c.shift - SHIFT)),
        run(a.plan.whole ? tiles : run_tiles_listed(a.plan, tiles, a.b.n_tokens)), runs(ceil_div(tiles, run)) {}
  __device__ __forceinline__ Set set(const AttnArgs& a, int row, int lane) const {
    const RowOf r = seq_of_row(a.b, row, lane);
    return Set{r.seq, r.b, r.token, row * runs * run, tiles};
  }
};
// The sequence with new tokens (of this row block) behind this one, its tiles next (tiles 0: none); 64 looked at
// together, since a padded batch may hold many without.
template <int SEEN, class C>
__device__ __forceinline__ Set next_seq(const AttnArgs& a, const Set& s, int lane, const C& tiles_of) {
  const int first = s.first + s.tiles;
  for (int b = s.b + 1; b < a.b.n_seqs; b += 64) {
    const Seq q = lane_seq(a.b, b, lane);
    const unsigned long long at = __ballot(SEEN == WINDOW ? tiles_of(q) > 0 : q.tokens > 0);
    if (at) {
      const int l = __ffsll(at) - 1;
      const Seq found = of_lane(q, l);
      return Set{found, b + l, 0, first, tiles_of(found)};
    }
  }
  return Set{Seq{0, 0, 0}, -1, 0, first, 0};
}

// How the pairs of the sequences and their row blocks are cut (AttnPlan::paired).
template <int SHIFT>
__device__ __forceinline__ PairCut cut_of_pairs(const AttnArgs& a, const Seq& s0, int lane) {
  if (a.plan.whole) return pair_cut(a.plan, 0, 0, 0, 0, 0);
  long long tiles = 0;
  int pairs = 0, fewest = 1 << 30, most = 0;
  for (int i = 0; i < a.b.n_seqs; i += 64) {
    const Seq s = i == 0 ? s0 : lane_seq(a.b, i, lane);
    const int blocks = set_blocks(a.plan, s.tokens * a.group);
    pairs += blocks;
    tiles += (long long)blocks * pair_tiles(a.plan, a.window, s, a.group, SHIFT);
    fewest = blocks ? min(fewest, blocks) : fewest;
    most = max(most, blocks);
  }
  for (int o = 32; o; o >>= 1) {
    pairs += __shfl_xor(pairs, o);
    tiles += __shfl_xor(tiles, o);
    fewest = min(fewest, __shfl_xor(fewest, o));
    most = max(most, __shfl_xor(most, o));
  }
  const PairCut c = pair_cut(a.plan, tiles, pairs, a.b.n_seqs, fewest, most);
  return PairCut{__builtin_amdgcn_readfirstlane(c.kind), __builtin_amdgcn_readfirstlane(c.run),
                 __builtin_amdgcn_readfirstlane(c.blocks), __builtin_amdgcn_readfirstlane(c.joins)};
}
// Left for the join by one work-group: how the pairs are cut, and whether one of them is in several runs at all.
template <int SHIFT>
__device__ __forceinline__ void leave_cut(const AttnArgs& a, PairCut c, const Seq& s0, int lane, size_t slots) {
  if (c.kind == APART) {
    int cut = 0;
    for (int i = 0; i < a.b.n_seqs; i += 64) {
      const Seq s = i == 0 ? s0 : lane_seq(a.b, i, lane);
      cut |= s.tokens > 0 && pair_tiles(a.plan, a.window, s, a.group, SHIFT) > c.run;
    }
    c.joins = __any(cut);
  }
  if (threadIdx.x == 0) *reinterpret_cast<PairCut*>(a.part + slots * attn_rows(a.plan) * (a.c.head_dim + 2)) = c;
}
// A pair that is cut EVEN or APART: the one that run x begins in, or (x < 0) that of row `row`, head g of its group.  A set's
// row blocks stand from the last on, which sees the most positions; of pairs APART the runs of the same tiles stand
// together.
struct Pair {
  Set set;  // EVEN: its first tile among all; APART: its tiles from 0 on
  int rb;
  int part, parts, each;  // APART: the run (of x), how many there are, and their tiles,
  int slot, step;         // the place of its first part, and how far the next ones are from each other
};
template <int SHIFT>
__device__ __forceinline__ Pair find_pair(const AttnArgs& a, const PairCut& cut, const Seq& s0, int x, int row, int g,
                                          int lane) {
  const BatchArgs& b = a.b;
  const bool even = cut.kind == EVEN;
  const int want = even ? x * cut.run : x;  // (x is under the shares, tiles under 2^30)
  int before = 0, slots = 0;
  for (int i = 0; i < b.n_seqs; i += 64) {
    const Seq s = i == 0 ? s0 : lane_seq(b, i, lane);
    const int blocks = set_blocks(a.plan, s.tokens * a.group), tiles = pair_tiles(a.plan, a.window, s, a.group, SHIFT);
    const PairRuns r = even ? PairRuns{tiles, 1} : pair_runs(tiles, cut.run);
    const int n = blocks * r.parts, split = r.parts > 1 ? n : 0;  // tiles, or runs
    const int upto = before + lane_prefix(n, lane, b.n_seqs - i), slots_upto = slots + lane_prefix(split, lane, b.n_seqs - i);
    const bool mine = x >= 0 ? upto - n <= want && want < upto : row >= s.row && row < s.row + s.tokens;
    const unsigned long long at = __ballot(mine);
    if (at) {
      const int l = __ffsll(at) - 1;
      const int first = __builtin_amdgcn_readlane(upto - n, l), sets_blocks = __builtin_amdgcn_readlane(blocks, l);
      Pair p;
      p.set = Set{of_lane(s, l), i + l, 0, 0, __builtin_amdgcn_readlane(tiles, l)};
      p.parts = __builtin_amdgcn_readlane(r.parts, l);
      p.each = __builtin_amdgcn_readlane(r.each, l);
      const int from_last = x < 0 ? sets_blocks - 1 - ((row - p.set.seq.row) * a.group + g) / attn_rows(a.plan)
                            : even ? (want - first) / p.set.tiles
                                   : (want - first) % sets_blocks;
      p.rb = sets_blocks - 1 - from_last;
      p.part = x < 0 || even ? 0 : (want - first) / sets_blocks;
      if (even) p.set.first = first + from_last * p.set.tiles;
      p.slot = __builtin_amdgcn_readlane(slots_upto - split, l) + from_last;
      p.step = sets_blocks;
      return p;
    }
    const int last = min(b.n_seqs - i, 64) - 1;
    before = __builtin_amdgcn_readlane(upto, last);
    slots = __builtin_amdgcn_readlane(slots_upto, last);
  }
  return Pair{Set{Seq{0, 0, 0}, -1, 0, 0, 0}, 0, 0, 1, 1, 0, 1};
}
// The pair behind this one where they are cut EVEN.
template <int SHIFT>
__device__ __forceinline__ Set next_pair(const AttnArgs& a, const Set& s, int& rb, int lane) {
  if (rb > 0) {
    --rb;
    return Set{s.seq, s.b, 0, s.first + s.tiles, s.tiles};
  }
  for (int b = s.b + 1; b < a.b.n_seqs; b += 64) {
    const Seq q = lane_seq(a.b, b, lane);
    const unsigned long long at = __ballot(q.tokens > 0);
    if (at) {
      const int l = __ffsll(at) - 1;
      const Seq found = of_lane(q, l);
      rb = set_blocks(a.plan, found.tokens * a.group) - 1;
      return Set{found, b + l, 0, s.first + s.tiles, pair_tiles(a.plan, a.window, found, a.group, SHIFT)};
    }
  }
  return Set{Seq{0, 0, 0}, -1, 0, 0, 0};
}

// Entry idx of a row's list of pages (behind its end the last one, which no tile takes).
__device__ __forceinline__ int listed(const AttnArgs& a, int row, int h, int idx) {
  return a.sel[((size_t)row * a.c.kv_heads + h) * a.n_sel + min(idx, a.n_sel - 1)];
}

// The tiles of a set from `tile` to `hi`, every `step`-th, those without a visible position left out.  Lane l holds
// entry `from` + l of the page list, as the page's number (any: the table's) and its index in the sequence.  Through a
// window a set's tiles are the first ones and those of the window; the first 64 entries of the table are held besides.
template <int D, int SEEN, class F>
struct Tiles {
  const AttnArgs& a;
  const Set& set;
  const int h, len_max, lane, psh, hi, step;
  int tile, from, number, index;
  int firsts, skip, first_number;  // of a window
  int p0;                          // of the tile found: its first position,
  const char *kp, *vp;             // its keys and values (the same for the whole wave),
  size_t scales;                   // and its scales
  __device__ __forceinline__ Tiles(const AttnArgs& a_, const Set& set_, int h_, const Rows<SEEN>& rows, int lane_,
                                   int lo, int hi_, int skip_, int step_, int entry)
      : a(a_), set(set_), h(h_), len_max(rows.len_max), lane(lane_), psh(a_.c.shift - F::SHIFT), hi(hi_), step(step_),
        tile(lo + skip_), from(lo >> psh), number(-1), index(-1), firsts(0), skip(0), first_number(-1), p0(0),
        kp(nullptr), vp(nullptr), scales(0) {
    if (SEEN == WINDOW) {
      const WindowTiles w = window_tiles(a.window, rows.len_min, len_max, F::SHIFT);
      firsts = w.firsts;
      skip = w.low - w.firsts;
      from = max(tile + skip, w.low) >> psh;  // the wave's first tile of the window itself
      if (len_max > 0 && tile < firsts)
        first_number = a.b.table[(size_t)set.b * a.b.table_stride + min(lane, a.b.table_stride - 1)];
    }
    list(entry);
  }
  // Raw entries, not looked at before find(): the query rows' loads go out behind these without a wait.  entry: of a
  // list of pages, loaded before.
  __device__ __forceinline__ void list(int entry) {
    if (len_max <= 0) return;  // nothing to see; the table may have no columns
    const int* table = a.b.table + (size_t)set.b * a.b.table_stride;
    if (SEEN == LISTED) {
      const bool in = entry >= 0 && entry <= (len_max - 1) >> a.c.shift;
      number = table[in ? entry : 0];
      index = in ? entry : 1 << 30 >> a.c.shift;  // at positions that no row sees
    } else {
      number = table[min(from + lane, a.b.table_stride - 1)];
    }
  }
  __device__ __forceinline__ bool find() {
    for (; tile < hi; tile += step) {
      int t = tile, at, raw;
      if (SEEN == WINDOW && tile < firsts && tile >> psh < 64) {
        at = tile >> psh;
        raw = __builtin_amdgcn_readlane(first_number, at);
      } else {
        if (SEEN == WINDOW && tile >= firsts) t = tile + skip;
        // (tiles of the window lie at `from` or behind it; first ones past the 64 entries may lie before it)
        if ((t >> psh) - from >= 64 || (SEEN == WINDOW && t >> psh < from)) {
          from = t >> psh;
          list(SEEN == LISTED ? listed(a, set.seq.row + set.token, h, from + lane) : 0);
          asm volatile("" : "+v"(number), "+v"(index));  // waited for here, not by every tile behind the branch
        }
        at = (t >> psh) - from;
        raw = __builtin_amdgcn_readlane(number, at);
      }
      const int pn = page_or_none(raw, a.c.n_pages);
      const int off = (t << F::SHIFT) & ((1 << a.c.shift) - 1);
      p0 = SEEN == LISTED ? (__builtin_amdgcn_readlane(index, at) << a.c.shift) + off : t << F::SHIFT;
      if (pn < 0 || p0 >= len_max) continue;
      const size_t base = head_base(a.c, pn, h) * F::BYTES;
      kp = reinterpret_cast<const char*>(a.c.k) + base + off * 16;
      vp = reinterpret_cast<const char*>(a.c.v) + base + off * (D * F::BYTES);
      if (F::CODED) scales = scale_base(a.c, pn, h) + off;
      tile += step;
      return true;
    }
    return false;
  }
};

// Values behind the last visible position may be anything: zeros in their place (their probabilities are zero, but
// zero times NaN is not).  p: the position of the first of 8.
__device__ __forceinline__ uint4 visible8(const uint4& v, int p, int len) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = p + 2 * e + 1 < len ? w[e] : p + 2 * e < len ? w[e] & 0xFFFFu : 0u;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Whether one of the wave's values is infinite or NaN.
template <int N>
__device__ __forceinline__ bool any_odd(const uint4 (&v)[N]) {
  typedef __attribute__((ext_vector_type(2))) uint16_t u16x2;
  u16x2 top = {0, 0};
#pragma unroll
  for (int d = 0; d < N; ++d) {
    const uint32_t w[4] = {v[d].x, v[d].y, v[d].z, v[d].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[e] & 0x7FFF7FFFu));
  }
  return __any(top[0] >= 0x7F80 || top[1] >= 0x7F80);
}

// The values from position `from` on that are no numbers become zeros; in their place, ones where they were and zeros
// elsewhere.  p: the position of the first of 8.
__device__ __forceinline__ uint4 drop_odd(uint4& v, int p, int from) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w}, at[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t half = e & 1 ? 0x7F800000u : 0x7F80u;
    if ((w[e >> 1] & half) == half && p + e >= from) {
      w[e >> 1] &= e & 1 ? 0xFFFFu : 0xFFFF0000u;
      at[e >> 1] |= e & 1 ? 0x3F800000u : 0x3F80u;
    }
  }
  v = make_uint4(w[0], w[1], w[2], w[3]);
  return make_uint4(at[0], at[1], at[2], at[3]);
}
// The same through a window, and for codes: the positions that a row, all rows or any row sees, as bits and words of
// masks (a comparison's result for each position would be 16 pairs of scalar registers).
struct Reach {
  int start, len, first;  // [start, len) and [0, first)
  // Bit i: position p + i, i < N.
  template <int N>
  __device__ __forceinline__ uint32_t bits(int p) const {
    const auto below = [&](int end) { return (1u << min(max(end - p, 0), N)) - 1; };
    return below(len) & (~below(start) | below(first));
  }
};
__device__ __forceinline__ uint32_t bit_mask(uint32_t bits, int i) { return (uint32_t)((int32_t)(bits << (31 - i)) >> 31); }
// Masks of the BF16 values of positions 2 e and 2 e + 1.
__device__ __forceinline__ uint32_t pair_mask(uint32_t bits, int e) {
  return (bit_mask(bits, 2 * e) & 0xFFFFu) | (bit_mask(bits, 2 * e + 1) & 0xFFFF0000u);
}
__device__ __forceinline__ uint4 masked8(const uint4& v, uint32_t bits) {
  return make_uint4(v.x & pair_mask(bits, 0), v.y & pair_mask(bits, 1), v.z & pair_mask(bits, 2),
                    v.w & pair_mask(bits, 3));
}
// Ones at the positions of the bits.
__device__ __forceinline__ uint4 ones8(uint32_t bits) {
  return masked8(make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u), bits);
}
// The values that are no numbers where the bits are not set become zeros; in their place, ones.
__device__ __forceinline__ uint4 drop_odd_but(uint4& v, uint32_t bits) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t odd = ((w[e] & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) |
                         ((w[e] & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
    const uint32_t drop = odd & ~pair_mask(bits, e);
    w[e] &= ~drop;
    (e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w) = w[e];
    w[e] = drop & 0x3F803F80u;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Of a word of four E4M3 codes, bit 8 k + 7 where code k is a NaN (0x7F, 0xFF).
__device__ __forceinline__ uint32_t odd_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
// The same as drop_odd_but for 8 codes.
__device__ __forceinline__ uint4 drop_odd_codes(uint32_t& lo, uint32_t& hi, uint32_t bits) {
  uint32_t drop = 0;  // bit i: code i
#pragma unroll
  for (int k = 0; k < 4; ++k)
    drop |= (odd_codes(lo) >> (8 * k + 7) & 1u) << k | (odd_codes(hi) >> (8 * k + 7) & 1u) << (4 + k);
  drop &= ~bits;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    lo &= ~(bit_mask(drop, k) & 0xFFu << 8 * k);
    hi &= ~(bit_mask(drop, 4 + k) & 0xFFu << 8 * k);
  }
  return ones8(drop);
}
// Ones at the positions, of 8 from p on, that a row of length len sees.
__device__ __forceinline__ uint4 seen8(int p, int len) {
  return visible8(make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u), p, len);
}

// Of 16 lanes that hold a value each, the I-th's (a scale of a position, to the lanes that hold its products).
template <int I>
__device__ __forceinline__ float of_sixteen(float v) {
  return dpp<0x150 + I>(v);
}
template <int N, int I = 0>
__device__ __forceinline__ void times_each(float (&x)[N], float v) {
  if constexpr (I < N) {
    x[I] *= of_sixteen<I>(v);
    times_each<N, I + 1>(x, v);
  }
}

// The lane's products s of one row (8 for a tile of 32 positions, 16 for one of 64) as probabilities against the row's
// running maximum; its sum and values follow where the maximum moves.  p0: the position of the first; whole: every row
// sees all of them, or those that it does not see are `hidden` already.
template <int N, int DT>
__device__ __forceinline__ void probabilities(const AttnArgs& a, const float (&s)[N], bool whole, int p0, int len,
                                              float& mx, float& sum, f32x4 (&acc)[DT], float (&p)[N]) {
  float y[N];  // as exponents of two
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = s[i] * a.scale_hi;
  if (!whole) {
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = p0 + i < len ? y[i] : -INFINITY;
  }
  float top = fmaxf(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), fmaxf(fmaxf(y[4], y[5]), fmaxf(y[6], y[7])));
  if constexpr (N == 16)
    top = fmaxf(top, fmaxf(fmaxf(fmaxf(y[8], y[9]), fmaxf(y[10], y[11])),
                           fmaxf(fmaxf(y[12], y[13]), fmaxf(y[14], y[15]))));
  top = rows_max(top);
  if (__any(top > mx + 8.f)) {
    const float high = top > mx + 8.f ? top : mx;  // a row's own: no row feels another's
    const float f = exp2_of(mx - high);
    mx = high;
    sum *= f;
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[d] *= f;
  }
  // exponents with the scale in two parts, the small one's product added to the difference from the maximum: both sums
  // round at the difference's size (the other way round the first would round at the maximum's)
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] = exp2_of(__builtin_fmaf(s[i], a.scale_lo, __builtin_fmaf(s[i], a.scale_hi, -mx)));
  if (!whole) {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = p0 + i < len ? p[i] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < N; i += 8)
    sum += ((p[i] + p[i + 1]) + (p[i + 2] + p[i + 3])) + ((p[i + 4] + p[i + 5]) + (p[i + 6] + p[i + 7]));
}

// Products of positions that the row does not see, as a value that weighs nothing: the scale's parts are not zero.
template <int N>
__device__ __forceinline__ void hide(float (&s)[N], uint32_t bits, float scale) {
  const uint32_t hidden = scale > 0.f ? 0xFF800000u : 0x7F800000u;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t m = bit_mask(bits, i);
    s[i] = __uint_as_float((__float_as_uint(s[i]) & m) | (hidden & ~m));
  }
}

// 8 codes as BF16, which holds them exactly.
template <int CODE>
__device__ __forceinline__ uint4 widened(uint32_t lo, uint32_t hi) {
  uint32_t w[4];
  const uint32_t u[2] = {lo, hi};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t x = u[e >> 1];
    if constexpr (CODE == HCR_INT8) {
      const f32x2 v = {code(x, 2 * (e & 1)), code(x, 2 * (e & 1) + 1)};
      w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    } else {
      const bf16x2 v = e & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.f, true)
                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.f, false);
      w[e] = __builtin_bit_cast(uint32_t, v);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The matrix cores' operand in half h of 16 loaded bytes.
template <int CODE>
__device__ __forceinline__ uint4 operand(const uint4& u, int h) {
  if constexpr (CODE == HCR_BF16)
    return u;
  else
    return h ? widened<CODE>(u.z, u.w) : widened<CODE>(u.x, u.y);
}

__device__ __forceinline__ f32x4 mfma(const uint4& x, const uint4& y, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(x), as_bf16x8(y), c, 0, 0, 0);
}

// One row's values out: its outputs where the work-group had all of its tiles, else its part for the join.
struct Out {
  const AttnArgs& a;
  const bool only;
  const size_t slot, slots;
  __device__ __forceinline__ void values(int D, int rid, int slot_row, int d, const f32x4& o, float sum) const {
    if (only)
      store4(a.out, a.out_type, (size_t)rid * D + d, o * (sum > 0.f ? 1.f / sum : 0.f));
    else
      *reinterpret_cast<f32x4*>(a.part + (slot * attn_rows(a.plan) + slot_row) * D + d) = o;
  }
  __device__ __forceinline__ void state(int D, int slot_row, float mx, float sum) const {
    const size_t rows = attn_rows(a.plan);
    if (!only) *reinterpret_cast<f32x2*>(a.part + slots * rows * D + (slot * rows + slot_row) * 2) = f32x2{mx, sum};
  }
};

// A set's tiles [lo, hi) (counted from its own first) in one work-group: its rows' part of the softmax.
template <int D, int MT, int SEEN, bool ONCE, int CODE>
__device__ __forceinline__ void attn_run(const AttnArgs& a, const Set& set, int h, int rb, int lo, int hi,
                                         int entry, const Out& out, uint4* lds) {
  using F = Format<CODE, D>;
  constexpr bool SEL = SEEN == LISTED;
  constexpr int KS = D / 32, DT = D / 16;             // operands of a key and of a tile's values
  constexpr int KT = F::KT, HALVES = F::HALVES, KL = KS / HALVES;  // loads of a key
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int RT = a.plan.row_waves, TG = a.plan.groups;  // waves: TG groups over the tiles x RT over the rows
  const int rt = wave % RT, tg = wave / RT;
  const int G = a.group;
  const Rows<SEEN> rows(a, set.seq, set.token, rb);
  if (rows.first >= rows.count) return;
  // a wave behind the last row takes the last row again, and stores nothing
  const int r0 = rows.first + rt * 16 * MT;
  const bool idle = r0 >= rows.count;
  Tiles<D, SEEN, F> tiles(a, set, h, rows, lane, lo, hi, tg, TG, entry);

  // Keys of the next tile are loaded behind their last use in this one, values likewise.  Loads return in order and a
  // wait counts the loads issued behind the one it is for: behind a branch there is no count, and the wait for the keys
  // covers the values too.  BLIND: no branch, past the last tile every lane asks for the tile's first 16 bytes again.
  // Taken where several row waves of D = 64, or of two tiles of D = 256, share the tiles: 60 rows of D = 64 over 50,000
  // 69 against 81 us, over 20,000 39 against 43, 64 of D = 256 over 16,400 49 against 51 (1,000 and 300 positions, 256
  // rows of D = 64: 1 % slower).  Not elsewhere, where the loads for nothing cost as much as they gain: 60 rows of
  // D = 128 110 against 107, 96 of D = 256 362 against 339, one row over 700 9.6 against 9.1, over 420,000 536 against
  // 529; for 36 rows of D = 256 49.7 against 50.7.
  constexpr bool BLIND = !ONCE && SEEN == DENSE && !F::CODED && (D == 64 || (D == 256 && MT == 2));
  // the values' loads: 16 bytes, or 8 where 32 codes of a dimension go to four lanes
  using V = std::conditional_t<F::EACH * F::BYTES == 16, uint4, uint2>;
  constexpr int NV = F::EACH;  // products of a lane
  const uint32_t k_lane = ((uint32_t)(lg << a.c.shift) + F::TILE / 4 * (li >> 2) + (li & 3)) * 16;  // key tile 0's row li
  const uint32_t v_lane = sizeof(V) == 16 ? (uint32_t)(lg * D + li) * 16
                                          : (uint32_t)((lg >> 1) * D + li) * 16 + (lg & 1) * 8;
  const int mine_of = F::EACH * lg + (li & (F::EACH - 1));  // codes: the position whose scales the lane holds
  const uint32_t k_step = 4u << a.c.shift << 4;  // 4 groups of dimensions on
  uint4 kf[KT][KL];
  V vf[DT];
  float ks = 0.f, vs = 0.f;  // codes: scales of a position
  auto load_keys = [&](uint32_t on) {
#pragma unroll
    for (int k = 0; k < KL; ++k) {
      const char* at = tiles.kp + (k * k_step & on);
#pragma unroll
      for (int t = 0; t < KT; ++t) kf[t][k] = ld_kv<ONCE>(at + (k_lane & on) + (t * 4 * 16 & on));
    }
    if constexpr (F::CODED) ks = a.code.k_scales[tiles.scales + mine_of];
  };
  auto load_values = [&](uint32_t on) {
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const char* at = tiles.vp + (v_lane & on) + (16 * 16 * d & on);
      if constexpr (sizeof(V) == 16)
        vf[d] = ld_kv<ONCE>(at);
      else
        vf[d] = ld_kv8<ONCE>(at);
    }
    if constexpr (F::CODED) vs = a.code.v_scales[tiles.scales + mine_of];
  };
  // the lane's query row of each 16-row tile and its length; the rows as operands in LDS, one copy for all groups
  // (in registers they would push the loop's operands out)
  uint4* lds_q = lds + (size_t)rt * MT * KS * 64 + lane;  // [RT][MT][KS][64]
  uint4 qf[MT][KS];
  int len[MT];
  int rid[MT];  // row of q and out: under 2^30
  bool live[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = min(r0 + 16 * m + li, rows.count - 1);
    live[m] = r0 + 16 * m + li < rows.count;
    const int t = SEL ? set.token : r / G, g = SEL ? r : r % G;
    len[m] = set.seq.first + t + 1;
    rid[m] = (set.seq.row + t) * a.heads + h * G + g;
    if (tg == 0) {
#pragma unroll
      for (int k = 0; k < KS; ++k)  // the dimensions that the lane's operand of a key holds
        qf[m][k] = ld16(a.q + (size_t)rid[m] * D +
                        (F::CODED ? 16 * lg + 64 * (k / 2) + 8 * (k % 2) : 8 * lg + 32 * k));
    }
  }
  const auto row_reach = [&](int m) {
    return Reach{SEEN == WINDOW ? len[m] - a.window.size : 0, len[m], SEEN == WINDOW ? a.window.first : 0};
  };
  // row waves alone keep step, so that the first one's misses are the others' hits in L1 (36 rows of D = 256: 314
  // against 342 us; all of them find the same tiles)
  const bool together = TG == 1 && RT > 1;
  f32x4 acc[MT][DT];
  float mx[MT], sum[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    mx[m] = -FLT_MAX;
    sum[m] = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[m][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  bool more = tiles.find();
  if (tg == 0) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int k = 0; k < KS; ++k) lds_q[(m * KS + k) * 64] = qf[m][k];
    }
  }
  if (BLIND && (idle || !more)) {
    lds_barrier();
    while (more) {
      more = tiles.find();
      if (together) __builtin_amdgcn_s_barrier();
    }
  } else {
    if (BLIND || (more && !idle)) {
      load_keys(~0u);
      load_values(~0u);
    }
    lds_barrier();
  }

  while (more) {
    if (!BLIND && idle) {
      more = tiles.find();
      if (together) __builtin_amdgcn_s_barrier();
      continue;
    }
    const int now = tiles.p0;
    const bool whole = rows.all_see(a, now, F::TILE);
    f32x4 s[MT][KT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int t = 0; t < KT; ++t) s[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if constexpr (F::CODED) {  // a key's operands once for all row tiles
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint4 qk[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) qk[m] = lds_q[(m * KS + k) * 64];
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          const uint4 key = operand<CODE>(kf[t][k / 2], k % 2);
#pragma unroll
          for (int m = 0; m < MT; ++m) s[m][t] = mfma(key, qk[m], s[m][t]);
        }
        __builtin_amdgcn_sched_barrier(0x100);  // one step's operands at a time (LDS reads may go ahead)
      }
    } else {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint4 qk = lds_q[(m * KS + k) * 64];
#pragma unroll
          for (int t = 0; t < KT; ++t) s[m][t] = mfma(kf[t][k], qk, s[m][t]);
        }
      }
    }
    const float ks_now = ks;
    __builtin_amdgcn_sched_barrier(0);
    more = tiles.find();
    if (together) __builtin_amdgcn_s_barrier();
    const uint32_t on = !BLIND || more ? ~0u : 0u;
    if (BLIND || more) load_keys(on);
    __builtin_amdgcn_sched_barrier(0);

    const int mine = now + F::TILE / 4 * lg;  // the position of the lane's first product and value
    // A value that is no number and that only some of the rows see: zero times it would reach the others.  It leaves the
    // product, and its dimension of the rows that see it becomes NaN: those where a product of such places with the
    // rows' visible ones is not zero.
    const auto spoil = [&](int m, int d, const f32x4& met) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][d][i] = met[i] > 0.f ? NAN : acc[m][d][i];
    };
    const f32x4 none = {0.f, 0.f, 0.f, 0.f};
    const Reach any{rows.start_min, rows.len_max, a.window.first}, all{rows.start_max, rows.len_min, a.window.first};
    if constexpr (!F::CODED && SEEN != WINDOW) {
      if (!whole) {
#pragma unroll
        for (int d = 0; d < DT; ++d) vf[d] = visible8(vf[d], mine, rows.len_max);
      }
      if (!SEL && !whole && rows.len_min < rows.len_max && any_odd(vf)) {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const uint4 at = drop_odd(vf[d], mine, rows.len_min);
#pragma unroll
          for (int m = 0; m < MT; ++m) spoil(m, d, mfma(at, seen8(mine, len[m]), none));
        }
      }
    } else if constexpr (!F::CODED) {
      if (!whole) {
        const uint32_t seen = any.bits<8>(mine), common = all.bits<8>(mine);
#pragma unroll
        for (int d = 0; d < DT; ++d) vf[d] = masked8(vf[d], seen);
        if (rows.len_min < rows.len_max && any_odd(vf)) {
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            const uint4 at = drop_odd_but(vf[d], common);
#pragma unroll
            for (int m = 0; m < MT; ++m) spoil(m, d, mfma(at, ones8(row_reach(m).template bits<8>(mine)), none));
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
    }
    if constexpr (F::CODED) {
      float p[MT][NV];  // a row tile's probabilities, times their values' scales
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = s[m][i >> 2][i & 3];
        times_each(v, ks_now);
        if (!whole) hide(v, row_reach(m).template bits<NV>(mine), a.scale_hi);
        probabilities(a, v, true, 0, 0, mx[m], sum[m], acc[m], p[m]);
        times_each(p[m], vs);
      }
      // what a row does not see may be anything: a scale there, and an E4M3 code that is no number (which goes as other
      // such values do)
      if (!whole) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint32_t seen = row_reach(m).template bits<NV>(mine);
#pragma unroll
          for (int i = 0; i < NV; ++i) p[m][i] = __uint_as_float(__float_as_uint(p[m][i]) & bit_mask(seen, i));
        }
        if constexpr (CODE == HCR_E4M3) {
          uint32_t hit = 0;
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            hit |= odd_codes(vf[d].x) | odd_codes(vf[d].y);
            if constexpr (sizeof(V) == 16) hit |= odd_codes(vf[d].z) | odd_codes(vf[d].w);
          }
          if (__any(hit != 0)) {
            const uint32_t common = all.bits<NV>(mine);
            const auto drop = [&](int d, uint32_t& lo, uint32_t& hi, int u) {  // codes 8 u and on
              const uint4 at = drop_odd_codes(lo, hi, common >> 8 * u & 0xFFu);
#pragma unroll
              for (int m = 0; !SEL && m < MT; ++m)  // (a list's rows see the same positions: what is dropped nobody sees)
                spoil(m, d, mfma(at, ones8(row_reach(m).template bits<8>(mine + 8 * u)), none));
              __builtin_amdgcn_sched_barrier(0);
            };
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              drop(d, vf[d].x, vf[d].y, 0);
              if constexpr (sizeof(V) == 16) drop(d, vf[d].z, vf[d].w, 1);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < NV / 8; ++u) {
        uint4 ph[MT], pl[MT], pr[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = p[m][8 * u + i];
          split_hi_lo(x, ph[m], pl[m]);
          if (a.out_type == HCR_F32) pr[m] = split_rest(x, ph[m], pl[m]);
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          uint4 value;
          if constexpr (sizeof(V) == 16)
            value = operand<CODE>(vf[d], u);
          else
            value = widened<CODE>(vf[d].x, vf[d].y);
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[m][d] = mfma(value, ph[m], acc[m][d]);
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[m][d] = mfma(value, pl[m], acc[m][d]);
          if (a.out_type == HCR_F32) {  // (one branch for several dimensions was slower: 62 against 53 us at D = 64)
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[m][d] = mfma(value, pr[m], acc[m][d]);
          }
          if (d % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        }
      }
    } else {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float v[8], p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = s[m][i >> 2][i & 3];
        if (SEEN == WINDOW && !whole) hide(v, row_reach(m).template bits<8>(mine), a.scale_hi);
        probabilities(a, v, SEEN == WINDOW || whole, mine, len[m], mx[m], sum[m], acc[m], p);
        uint4 ph, pl;
        split_hi_lo(p, ph, pl);
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[m][d] = mfma(vf[d], ph, acc[m][d]);
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[m][d] = mfma(vf[d], pl, acc[m][d]);
        if (a.out_type == HCR_F32) {
          const uint4 pr = split_rest(p, ph, pl);
#pragma unroll
          for (int d = 0; d < DT; ++d) acc[m][d] = mfma(vf[d], pr, acc[m][d]);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (BLIND || more) load_values(on);
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) sum[m] = rows_sum(sum[m]);

  // the groups joined, a 16-row tile at a time: every wave leaves its values in LDS and takes its share of the row
  // tile's (the values where the query rows were, which nobody reads behind the first barrier here)
  f32x4* lds_acc = reinterpret_cast<f32x4*>(lds);                       // [TG][RT][DT][64]
  float* lds_m = reinterpret_cast<float*>(lds_acc + TG * RT * DT * 64);  // [TG][RT][MT][16]
  float* lds_l = lds_m + TG * RT * MT * 16;
  if (TG > 1) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (lg == 0) {
        lds_m[(wave * MT + m) * 16 + li] = mx[m];
        lds_l[(wave * MT + m) * 16 + li] = sum[m];
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int slot_row = (rt * MT + m) * 16 + li;
    if (TG == 1) {
      if (live[m]) {
#pragma unroll
        for (int d = 0; d < DT; ++d) out.values(D, rid[m], slot_row, 16 * d + 4 * lg, acc[m][d], sum[m]);
        if (lg == 0) out.state(D, slot_row, mx[m], sum[m]);
      }
      continue;
    }
    float top = -FLT_MAX, total = 0.f;
    for (int g0 = 0; g0 < TG; g0 += 4) {
      float gm[4], gl[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = ((min(g0 + i, TG - 1) * RT + rt) * MT + m) * 16 + li;
        gm[i] = lds_m[at];
        gl[i] = g0 + i < TG ? lds_l[at] : 0.f;
      }
      const float high = fmaxf(fmaxf(fmaxf(gm[0], gm[1]), fmaxf(gm[2], gm[3])), top);
      total *= exp2_of(top - high);
      top = high;
#pragma unroll
      for (int i = 0; i < 4; ++i) total += gl[i] * exp2_of(gm[i] - top);
    }
    const float own = exp2_of(mx[m] - top);  // what this wave's values weigh in the sum
    if (m > 0) __syncthreads();              // the tile before is taken
#pragma unroll
    for (int d = 0; d < DT; ++d) lds_acc[(wave * DT + d) * 64 + lane] = acc[m][d] * own;
    __syncthreads();
    for (int d = tg; d < DT; d += TG) {
      f32x4 o = {0.f, 0.f, 0.f, 0.f};
      for (int g0 = 0; g0 < TG; g0 += 4) {
        f32x4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lds_acc[((min(g0 + i, TG - 1) * RT + rt) * DT + d) * 64 + lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) o += g0 + i < TG ? v[i] : f32x4{0.f, 0.f, 0.f, 0.f};
      }
      if (live[m]) out.values(D, rid[m], slot_row, 16 * d + 4 * lg, o, total);
    }
    if (live[m] && tg == 0 && lg == 0) out.state(D, slot_row, top, total);
  }
}

// A work-group's part of a call: its kv head, row block and tiles, set by set.  PAIRED: of a call that has AttnPlan::paired (a
// kernel of its own, so that others do not hold its registers).
template <int SHIFT, int SEEN, bool PAIRED, class Run>
__device__ __forceinline__ void part_of(const AttnArgs& a, const Run& run) {
  constexpr bool SEL = SEEN == LISTED;
  const int lane = threadIdx.x & 63;
  // work-group -> (run, kv head, row block); the row blocks of one run sit on one XCD (its L2 then serves all but
  // the first), the last one, which sees the most positions, ahead (a prompt of 2,048 tokens, 32 heads of 128 over 8:
  // int8 82 against 104 us; of 4,096 in BF16 307 against 411)
  int RB = a.plan.row_blocks;
  const int turn = blockIdx.x / XCDS;
  int rb = RB - 1 - turn % RB;
  const int u = PAIRED ? blockIdx.x : turn / RB * XCDS + blockIdx.x % XCDS;
  const int h = u % a.c.kv_heads;
  int item = u / a.c.kv_heads;
  Cut cut;
  Set set;
  int entry = 0, begin = 0;
  size_t slot = (size_t)h * attn_slots(a.plan);
  const size_t slots = (size_t)a.c.kv_heads * attn_slots(a.plan);
  bool pairs = false;  // cut EVEN or APART
  if constexpr (PAIRED) {
    if (item >= a.plan.paired) return;
    const Seq s0 = lane_seq(a.b, 0, lane);
    const PairCut c = cut_of_pairs<SHIFT>(a, s0, lane);
    if (!a.plan.whole && blockIdx.x == 0) leave_cut<SHIFT>(a, c, s0, lane, slots);
    if (c.kind == ALIKE) {
      RB = c.blocks;
      rb = RB - 1 - item % RB;
      item /= RB;
    } else {
      if (c.kind == EVEN && item >= a.plan.shares) return;
      const Pair p = find_pair<SHIFT>(a, c, s0, item, 0, 0, lane);
      pairs = true;
      set = p.set;
      rb = p.rb;
      if (c.kind == EVEN) {
        begin = item * c.run;
        cut = Cut{c.run, false};
        slot += part_slot(item, c.run, set.first);
      } else {
        begin = p.part * p.each;
        cut = Cut{p.each, true};
        slot += p.slot + p.part * p.step;
      }
    }
  }
  const Count<SEEN, SHIFT> tiles_of(a, rb);
  if (!pairs) {
    if (item >= a.plan.items) return;
    if (SEL) {
      const Lists<SHIFT> lists(a);
      const int row = item / lists.runs;
      if (row >= a.b.n_tokens) return;
      begin = item * lists.run;
      cut = Cut{lists.run, true};
      // the list's load goes out beside the sequence's, one wait less (4 tokens, 64 pages
      // of 64, D = 256: 28.7 against 29.7 us)
      entry = listed(a, row, h, ((begin - row * lists.runs * lists.run) >> (a.c.shift - SHIFT)) + lane);
      set = lists.set(a, row, lane);
    } else if (!PAIRED && a.plan.whole) {
      set = seq_set(a.b, item, tiles_of);
      cut = Cut{set.tiles, true};
    } else {
      set = find_seq(a.b, item, 0, lane, a.plan, tiles_of, &cut);
      begin = item * cut.run;
    }
    slot += (size_t)rb * a.plan.items * 2 + part_slot(item, cut.run, set.first);
  }
  while (set.b >= 0) {
    const int lo = max(begin - set.first, 0), hi = min(begin + cut.run - set.first, set.tiles);
    const Out out{a, lo == 0 && hi == set.tiles, slot, slots};
    run(set, h, rb, lo, hi, entry, out);
    if (SEL || cut.apart || set.first + set.tiles >= begin + cut.run) break;
    if (PAIRED && pairs)
      set = next_pair<SHIFT>(a, set, rb, lane);
    else
      set = next_seq<SEEN>(a, set, lane, tiles_of);
    slot |= 1;        // of the sets that begin behind the run's first tile
    __syncthreads();  // the LDS of the set before is free
  }
}

// Over codes a work-group has one row wave (more rows share theirs) and so eight waves at most: held to the registers of
// 16, D = 64 spilled (E4M3, 64 of up to 8,192 77 us against 70, windows of 4,096 63 against 49).
template <int D, int MT, int SEEN, bool ONCE, int CODE, bool PAIRED>
__global__ __launch_bounds__(64 * (CODE == HCR_BF16 ? attn_waves(D, MT) : 8)) void attn_part(AttnArgs a) {
  extern __shared__ uint4 lds[];
  part_of<Format<CODE, D>::SHIFT, SEEN, PAIRED>(
      a, [&](const Set& set, int h, int rb, int lo, int hi, int entry, const Out& out) {
        attn_run<D, MT, SEEN, ONCE, CODE>(a, set, h, rb, lo, hi, entry, out, lds);
      });
}

// One row's parts joined: D / 4 lanes hold a row of 4 values each, the groups of lanes take the parts in turn and
// join in LDS, in a fixed order.
template <int D, int SEEN, int SHIFT, bool PAIRED>
__global__ __launch_bounds__(256) void attn_join(AttnArgs a) {
  constexpr bool SEL = SEEN == LISTED;
  constexpr int LANES = D / 4;
  const int GROUPS = blockDim.x / LANES;
  const int l = threadIdx.x % LANES, grp = threadIdx.x / LANES, lane = threadIdx.x & 63;
  const int hq = blockIdx.x % a.heads, row = blockIdx.x / a.heads;
  const int h = hq / a.group, g0 = hq % a.group;
  const int slot_rows = attn_rows(a.plan);
  Cut cut;
  Set set;
  int rb = 0;  // through a window a row block counts its own tiles
  size_t slot = (size_t)h * attn_slots(a.plan);
  const size_t slots = (size_t)a.c.kv_heads * attn_slots(a.plan);
  int n = 0, step = 0;  // of pairs APART: a row's parts, and how far they are from each other
  bool pairs = false;
  if constexpr (PAIRED) {
    const int* at = reinterpret_cast<const int*>(a.part + slots * slot_rows * (D + 2));  // what the other launch went by
    const PairCut c{__builtin_amdgcn_readfirstlane(at[0]), __builtin_amdgcn_readfirstlane(at[1]), 0, 0};
    if (!__builtin_amdgcn_readfirstlane(at[3])) return;
    if (c.kind != ALIKE) {
      const Pair p = find_pair<SHIFT>(a, c, lane_seq(a.b, 0, lane), -1, row, g0, lane);
      pairs = true;
      set = p.set;
      cut = Cut{c.run, false};
      if (c.kind == APART) {
        n = p.parts;
        slot += p.slot;
        step = p.step;
      }
    }
  }
  if (!pairs) {
    if (SEEN == WINDOW && a.plan.row_blocks > 1) {
      const RowOf of = seq_of_row(a.b, row, lane);
      if (of.b < 0) return;
      rb = (of.token * a.group + g0) / slot_rows;
    }
    const Count<SEEN, SHIFT> tiles_of(a, rb);
    set = SEL ? Lists<SHIFT>(a).set(a, row, lane) : find_seq(a.b, -1, row, lane, a.plan, tiles_of, &cut);
  }
  if (set.b < 0) return;
  const int run = SEL ? Lists<SHIFT>(a).run : cut.run;
  const int r = SEL ? g0 : (row - set.seq.row) * a.group + g0;  // of the set's rows
  const int part0 = set.first / run;
  if (!n) n = run_parts(set.first, set.tiles, run);
  if (n == 1) return;  // the row is out already
  if (!pairs) slot += (size_t)(r / slot_rows) * a.plan.items * 2;
  const float* pa = a.part + (slot * slot_rows + r % slot_rows) * D + 4 * l;
  const float* ml = a.part + slots * slot_rows * D + (slot * slot_rows + r % slot_rows) * 2;
  float mx = -FLT_MAX, sum = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = grp; s0 < n; s0 += 4 * GROUPS) {
    f32x2 v[4];
    f32x4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // four at a time on their way; past the end the last one, as nothing
      const int s = s0 + i * GROUPS;
      const int part = min(s, n - 1);
      const size_t to = (size_t)(PAIRED && step ? part * step : part_slot(part0 + part, run, set.first)) * slot_rows;
      v[i] = ld2(ml + to * 2);
      o[i] = ld4(pa + to * D);
      if (s >= n) v[i] = f32x2{-FLT_MAX, 0.f};
    }
    float now = mx;
#pragma unroll
    for (int i = 0; i < 4; ++i) now = fmaxf(now, v[i][0]);
    const float f = exp2_of(mx - now);
    mx = now;
    sum *= f;
    acc *= f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float w = s0 + i * GROUPS < n ? exp2_of(v[i][0] - now) : 0.f;
      sum += v[i][1] * w;
      acc += o[i] * w;
    }
  }
  __shared__ f32x4 lds_acc[256];
  __shared__ f32x2 lds_ml[256 / LANES];
  lds_acc[threadIdx.x] = acc;
  if (l == 0) lds_ml[grp] = f32x2{mx, sum};
  __syncthreads();
  if (grp != 0) return;
  mx = -FLT_MAX;
  for (int g = 0; g < GROUPS; ++g) mx = fmaxf(mx, lds_ml[g][0]);
  sum = 0.f;
  acc = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int g = 0; g < GROUPS; ++g) {
    const float f = exp2_of(lds_ml[g][0] - mx);
    sum += lds_ml[g][1] * f;
    acc += lds_acc[g * LANES + l] * f;
  }
  const float f = sum > 0.f ? 1.f / sum : 0.f;
  store4(a.out, a.out_type, ((size_t)row * a.heads + hq) * D + 4 * l, acc * f);
}

}  // namespace hcr
