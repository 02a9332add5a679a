// Attention of a decode window over the paged cache, gfx950 (MI355X):
//   out[n] = sum_p softmax_p(scale q[n] . k[p]) v[p],   p <= the token's position
// for every page of a sequence, or for the pages listed per token and kv head.
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
// Work: the tiles of all sequences, one behind the other, are cut into equal runs, one for each work-group that the
// chip holds at once (AttnPlan), so that unlike lengths and loose bounds cost nothing; a run goes from one sequence
// on to the next.  The waves of a work-group take its tiles in turn and join in LDS; sequences that lie in several
// runs are joined by a second launch; each join is (m, l, O) -> (max, sum of l 2^(m - max), sum of O 2^(m - max)),
// in a fixed order.  Where the chip is full of sequences or they are short, a work-group takes a whole one instead and
// nothing is left to join (there a long one among short ones, or a bound far above them, does cost: the plan's rule
// keeps that to sequences of 4,096).
//
// Bound by the bytes of keys and values.  Measured on MI355X (graphs of calls, inputs rotated): one sequence of
// 420,000 positions, 48 heads of 256 over 8, 2 tokens: 505 us, 6.8 TB/s (a 4 GiB device copy moves 4.8); 64 sequences
// of 1,000 to 8,192, 32 heads of 128 over 8: 194 us, 6.2 TB/s.  36 rows of 4 sequences of up to 9,001: 51 us, 3.3 TB/s:
// a work-group has 10 tiles behind 6 us of first loads, three row waves share each of them, so that a CU has 64 KB on
// their way where it has 256 KB with one row wave, and the second launch takes 7.

#include <float.h>
#include <math.h>
#include <hip/hip_runtime.h>

#include "hcr_paged_device.h"

namespace hcr {

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

__device__ __forceinline__ int tiles_of(const Seq& s) {
  return s.tokens ? max(ceil_div(s.first + s.tokens, TILE), 1) : 0;
}
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
__device__ __forceinline__ Set find_seq(const BatchArgs& b, int x, int row, int lane, const AttnPlan& p, Cut* cut) {
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
__device__ __forceinline__ Set seq_set(const BatchArgs& b, int i) {
  const Seq q = wave_seq(b, i);
  return Set{q, q.tokens ? i : -1, 0, 0, tiles_of(q)};
}
// Listed pages: every token's list in `runs` runs of `run` tiles, whole ones as one.
struct Lists {
  int tiles, run, runs;
  __device__ __forceinline__ explicit Lists(const AttnArgs& a)
      : tiles(a.n_sel << (a.c.shift - TILE_SHIFT)),
        run(a.plan.whole ? tiles : run_tiles_listed(a.plan, tiles, a.b.n_tokens)), runs(ceil_div(tiles, run)) {}
  __device__ __forceinline__ Set set(const AttnArgs& a, int row, int lane) const {
    const RowOf r = seq_of_row(a.b, row, lane);
    return Set{r.seq, r.b, r.token, row * runs * run, tiles};
  }
};
// The sequence with new tokens behind this one, its tiles next (tiles 0: none); 64 looked at together, since a padded
// batch may hold many without.
__device__ __forceinline__ Set next_seq(const AttnArgs& a, const Set& s, int lane) {
  const int first = s.first + s.tiles;
  for (int b = s.b + 1; b < a.b.n_seqs; b += 64) {
    const Seq q = lane_seq(a.b, b, lane);
    const unsigned long long at = __ballot(q.tokens > 0);
    if (at) {
      const int l = __ffsll(at) - 1;
      const Seq found = of_lane(q, l);
      return Set{found, b + l, 0, first, tiles_of(found)};
    }
  }
  return Set{Seq{0, 0, 0}, -1, 0, first, 0};
}

// The rows of a set that a work-group takes, and which positions they see: [0, len).
struct Rows {
  int first, count;      // of the set's rows; the work-group's first one, the set's number
  int len_min, len_max;  // of the work-group's rows
  __device__ __forceinline__ Rows(const AttnArgs& a, const Set& set, bool listed, int rb) {
    first = rb * attn_rows(a.plan);
    count = listed ? a.group : set.seq.tokens * a.group;
    const int last = min(first + attn_rows(a.plan), count) - 1;
    len_min = set.seq.first + (listed ? set.token : first / a.group) + 1;
    len_max = set.seq.first + (listed ? set.token : last / a.group) + 1;
  }
};

// Entry idx of a row's list of pages (behind its end the last one, which no tile takes).
__device__ __forceinline__ int listed(const AttnArgs& a, int row, int h, int idx) {
  return a.sel[((size_t)row * a.c.kv_heads + h) * a.n_sel + min(idx, a.n_sel - 1)];
}

// The tiles of a set from `tile` to `hi`, every `step`-th, those without a visible position left out.  Lane l holds
// entry `from` + l of the page list, as the page's number (any: the table's) and its index in the sequence.
template <int D, bool SEL>
struct Tiles {
  const AttnArgs& a;
  const Set& set;
  const int h, len_max, lane, psh, hi, step;
  int tile, from, number, index;
  int p0;               // of the tile found: its first position,
  const char *kp, *vp;  // its keys and values (the same for the whole wave)
  __device__ __forceinline__ Tiles(const AttnArgs& a_, const Set& set_, int h_, int len, int lane_, int lo, int hi_,
                                   int skip, int step_, int entry)
      : a(a_), set(set_), h(h_), len_max(len), lane(lane_), psh(a_.c.shift - TILE_SHIFT), hi(hi_), step(step_),
        tile(lo + skip), from(lo >> psh), number(-1), index(-1), p0(0), kp(nullptr), vp(nullptr) {
    list(entry);
  }
  // Raw entries, not looked at before find(): the query rows' loads go out behind these without a wait.  entry: of a
  // list of pages, loaded before.
  __device__ __forceinline__ void list(int entry) {
    if (len_max <= 0) return;  // nothing to see; the table may have no columns
    const int* table = a.b.table + (size_t)set.b * a.b.table_stride;
    if (SEL) {
      const bool in = entry >= 0 && entry <= (len_max - 1) >> a.c.shift;
      number = table[in ? entry : 0];
      index = in ? entry : 1 << 30 >> a.c.shift;  // at positions that no row sees
    } else {
      number = table[min(from + lane, a.b.table_stride - 1)];
    }
  }
  __device__ __forceinline__ bool find() {
    for (; tile < hi; tile += step) {
      if ((tile >> psh) - from >= 64) {
        from = tile >> psh;
        list(SEL ? listed(a, set.seq.row + set.token, h, from + lane) : 0);
        asm volatile("" : "+v"(number), "+v"(index));  // waited for here, not by every tile behind the branch
      }
      const int at = (tile >> psh) - from;
      const int pn = page_or_none(__builtin_amdgcn_readlane(number, at), a.c.n_pages);
      const int off = (tile << TILE_SHIFT) & ((1 << a.c.shift) - 1);
      p0 = SEL ? (__builtin_amdgcn_readlane(index, at) << a.c.shift) + off : tile << TILE_SHIFT;
      if (pn < 0 || p0 >= len_max) continue;
      const size_t base = head_base(a.c, pn, h);
      kp = reinterpret_cast<const char*>(a.c.k + base + off * 8);
      vp = reinterpret_cast<const char*>(a.c.v + base + off * D);
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
// Ones at the positions, of 8 from p on, that a row of length len sees.
__device__ __forceinline__ uint4 seen8(int p, int len) {
  return visible8(make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u), p, len);
}

// The lane's 8 products s of one row as probabilities against the row's running maximum; its sum and values follow
// where the maximum moves.  p0: the position of the first of 8; whole: every row sees all of them.
template <int DT>
__device__ __forceinline__ void probabilities(const AttnArgs& a, const f32x4 (&s)[2], bool whole, int p0, int len,
                                              float& mx, float& sum, f32x4 (&acc)[DT], float (&p)[8]) {
  float y[8];  // as exponents of two
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = s[i >> 2][i & 3] * a.scale_hi;
  if (!whole) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = p0 + i < len ? y[i] : -INFINITY;
  }
  float top = fmaxf(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), fmaxf(fmaxf(y[4], y[5]), fmaxf(y[6], y[7])));
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
  for (int i = 0; i < 8; ++i) {
    const float v = s[i >> 2][i & 3];
    p[i] = exp2_of(__builtin_fmaf(v, a.scale_lo, __builtin_fmaf(v, a.scale_hi, -mx)));
  }
  if (!whole) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = p0 + i < len ? p[i] : 0.f;
  }
  sum += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
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
template <int D, int MT, bool SEL, bool ONCE>
__device__ __forceinline__ void attn_run(const AttnArgs& a, const Set& set, int h, int rb, int lo, int hi,
                                         int entry, const Out& out, uint4* lds) {
  constexpr int KS = D / 32, DT = D / 16;
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int RT = a.plan.row_waves, TG = a.plan.groups;  // waves: TG groups over the tiles x RT over the rows
  const int rt = wave % RT, tg = wave / RT;
  const int G = a.group;
  const Rows rows(a, set, SEL, rb);
  if (rows.first >= rows.count) return;
  // a wave behind the last row takes the last row again, and stores nothing
  const int r0 = rows.first + rt * 16 * MT;
  const bool idle = r0 >= rows.count;
  Tiles<D, SEL> tiles(a, set, h, rows.len_max, lane, lo, hi, tg, TG, entry);

  // Keys of the next tile are loaded behind their last use in this one, values likewise.  Loads return in order and a
  // wait counts the loads issued behind the one it is for: behind a branch there is no count, and the wait for the keys
  // covers the values too.  BLIND: no branch, past the last tile every lane asks for the tile's first 16 bytes again.
  // Taken where several row waves of D = 64, or of two tiles of D = 256, share the tiles: 60 rows of D = 64 over 50,000
  // 69 against 81 us, over 20,000 39 against 43, 64 of D = 256 over 16,400 49 against 51 (1,000 and 300 positions, 256
  // rows of D = 64: 1 % slower).  Not elsewhere, where the loads for nothing cost as much as they gain: 60 rows of
  // D = 128 110 against 107, 96 of D = 256 362 against 339, one row over 700 9.6 against 9.1, over 420,000 536 against
  // 529; for 36 rows of D = 256 49.7 against 50.7.
  constexpr bool BLIND = !ONCE && !SEL && (D == 64 || (D == 256 && MT == 2));
  const uint32_t k_lane = ((uint32_t)(lg << a.c.shift) + 8 * (li >> 2) + (li & 3)) * 16;  // key tile 0's row li
  const uint32_t v_lane = (uint32_t)(lg * D + li) * 16;
  const uint32_t k_step = 4u << a.c.shift << 4;  // 32 dimensions on
  uint4 kf[2][KS], vf[DT];
  auto load_keys = [&](uint32_t on) {
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const char* at = tiles.kp + (k * k_step & on);
      kf[0][k] = ld_kv<ONCE>(at + (k_lane & on));
      kf[1][k] = ld_kv<ONCE>(at + (k_lane & on) + (4 * 16 & on));
    }
  };
  auto load_values = [&](uint32_t on) {
#pragma unroll
    for (int d = 0; d < DT; ++d) vf[d] = ld_kv<ONCE>(tiles.vp + (v_lane & on) + (16 * 16 * d & on));
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
      for (int k = 0; k < KS; ++k) qf[m][k] = ld16(a.q + (size_t)rid[m] * D + 8 * lg + 32 * k);
    }
  }
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
    const bool whole = now + TILE <= rows.len_min;
    f32x4 s[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      s[m][0] = s[m][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint4 qk = lds_q[(m * KS + k) * 64];
#pragma unroll
        for (int t = 0; t < 2; ++t) s[m][t] = mfma(kf[t][k], qk, s[m][t]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    more = tiles.find();
    if (together) __builtin_amdgcn_s_barrier();
    const uint32_t on = !BLIND || more ? ~0u : 0u;
    if (BLIND || more) load_keys(on);
    __builtin_amdgcn_sched_barrier(0);

    if (!whole) {
#pragma unroll
      for (int d = 0; d < DT; ++d) vf[d] = visible8(vf[d], now + 8 * lg, rows.len_max);
    }
    // A value that is no number and that only later tokens see: zero times it would reach the earlier ones' rows.  It
    // leaves the product, and its dimension of the rows that see it becomes NaN: those where a product of such places
    // with the rows' visible ones is not zero.
    if (!SEL && !whole && rows.len_min < rows.len_max && any_odd(vf)) {
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const uint4 at = drop_odd(vf[d], now + 8 * lg, rows.len_min);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const f32x4 met = mfma(at, seen8(now + 8 * lg, len[m]), f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][d][i] = met[i] > 0.f ? NAN : acc[m][d][i];
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float p[8];
      probabilities<DT>(a, s[m], whole, now + 8 * lg, len[m], mx[m], sum[m], acc[m], p);
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

template <int D, int MT, bool SEL, bool ONCE>
__global__ __launch_bounds__(64 * attn_waves(D, MT)) void attn_part(AttnArgs a) {
  extern __shared__ uint4 lds[];
  const int lane = threadIdx.x & 63;
  // work-group -> (run, kv head, row block); the row blocks of one run sit on one XCD (its L2 then serves all but
  // the first)
  const int RB = a.plan.row_blocks;
  const int turn = blockIdx.x / XCDS;
  const int rb = turn % RB;
  const int u = turn / RB * XCDS + blockIdx.x % XCDS;
  const int h = u % a.c.kv_heads, item = u / a.c.kv_heads;
  if (item >= a.plan.items) return;
  Cut cut;
  Set set;
  int entry = 0, begin = 0;
  if (SEL) {
    const Lists lists(a);
    const int row = item / lists.runs;
    if (row >= a.b.n_tokens) return;
    begin = item * lists.run;
    cut = Cut{lists.run, true};
    // the list's load goes out beside the sequence's, one wait less (4 tokens, 64 pages
    // of 64, D = 256: 28.7 against 29.7 us)
    entry = listed(a, row, h, ((begin - row * lists.runs * lists.run) >> (a.c.shift - TILE_SHIFT)) + lane);
    set = lists.set(a, row, lane);
  } else if (a.plan.whole) {
    set = seq_set(a.b, item);
    cut = Cut{set.tiles, true};
  } else {
    set = find_seq(a.b, item, 0, lane, a.plan, &cut);
    begin = item * cut.run;
  }
  const size_t slots = (size_t)a.c.kv_heads * RB * a.plan.items * 2;
  const size_t slot = ((size_t)h * RB + rb) * a.plan.items * 2;
  while (set.b >= 0) {
    const int lo = max(begin - set.first, 0), hi = min(begin + cut.run - set.first, set.tiles);
    const Out out{a, lo == 0 && hi == set.tiles, slot + part_slot(item, cut.run, set.first), slots};
    attn_run<D, MT, SEL, ONCE>(a, set, h, rb, lo, hi, entry, out, lds);
    if (SEL || cut.apart || set.first + set.tiles >= begin + cut.run) break;
    set = next_seq(a, set, lane);
    __syncthreads();  // the LDS of the set before is free
  }
}

// One row's parts joined: D / 4 lanes hold a row of 4 values each, the groups of lanes take the parts in turn and
// join in LDS, in a fixed order.
template <int D, bool SEL>
__global__ __launch_bounds__(256) void attn_join(AttnArgs a) {
  constexpr int LANES = D / 4;
  const int GROUPS = blockDim.x / LANES;
  const int l = threadIdx.x % LANES, grp = threadIdx.x / LANES, lane = threadIdx.x & 63;
  const int hq = blockIdx.x % a.heads, row = blockIdx.x / a.heads;
  Cut cut;
  const Set set = SEL ? Lists(a).set(a, row, lane) : find_seq(a.b, -1, row, lane, a.plan, &cut);
  if (set.b < 0) return;
  const int run = SEL ? Lists(a).run : cut.run, n = run_parts(set.first, set.tiles, run);
  if (n == 1) return;  // the row is out already
  const int h = hq / a.group, g0 = hq % a.group;
  const int r = SEL ? g0 : (row - set.seq.row) * a.group + g0;  // of the set's rows
  const int slot_rows = attn_rows(a.plan);
  const size_t slots = (size_t)a.c.kv_heads * a.plan.row_blocks * a.plan.items * 2;
  const size_t slot = ((size_t)h * a.plan.row_blocks + r / slot_rows) * a.plan.items * 2;
  const int part0 = set.first / run;
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
      const size_t to = (size_t)part_slot(part0 + min(s, n - 1), run, set.first) * slot_rows;
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

namespace {

template <int D, int MT, bool SEL>
void run_part(const AttnArgs& a, int grid, hipStream_t st) {
  const dim3 threads(64 * a.plan.row_waves * a.plan.groups);
  const int lds = attn_lds(D, a.plan);
  // one wave's rows, and not several tokens' lists, which mostly name the same pages
  if (a.plan.row_waves * a.plan.row_blocks == 1 && (!SEL || a.b.max_tokens == 1))
    hipLaunchKernelGGL((attn_part<D, MT, SEL, true>), dim3(grid), threads, lds, st, a);
  else
    hipLaunchKernelGGL((attn_part<D, MT, SEL, false>), dim3(grid), threads, lds, st, a);
}
template <int D, bool SEL>
void run_attn(const AttnArgs& a, int grid, int join_grid, hipStream_t st) {
  // a wave a row where rows have few parts, four where many
  const int join = a.plan.items > 2 * (SEL ? a.b.n_tokens : a.b.n_seqs) ? 256 : 64;
  if (a.plan.q_tiles == 1) {
    run_part<D, 1, SEL>(a, grid, st);
  } else if constexpr (D != 64) {
    run_part<D, 2, SEL>(a, grid, st);
  }
  if (join_grid) hipLaunchKernelGGL((attn_join<D, SEL>), dim3(join_grid), dim3(join), 0, st, a);
}

}  // namespace

int launch_attn(const AttnArgs& a, void* stream) {
  const AttnPlan& p = a.plan;
  const int grid = ceil_div(p.items * a.c.kv_heads, XCDS) * XCDS * p.row_blocks;
  const int join_grid = attn_joins(p) ? a.b.n_tokens * a.heads : 0;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  switch (a.c.head_dim) {
    case 64: a.sel ? run_attn<64, true>(a, grid, join_grid, st) : run_attn<64, false>(a, grid, join_grid, st); break;
    case 128: a.sel ? run_attn<128, true>(a, grid, join_grid, st) : run_attn<128, false>(a, grid, join_grid, st); break;
    default: a.sel ? run_attn<256, true>(a, grid, join_grid, st) : run_attn<256, false>(a, grid, join_grid, st);
  }
  return hipGetLastError() == hipSuccess ? HCR_OK : HCR_EHIP;
}

}  // namespace hcr
