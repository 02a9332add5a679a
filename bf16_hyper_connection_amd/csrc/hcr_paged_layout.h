// Index arithmetic of the paged cache, shared by its kernels, the C ABI and a host-compiled test: where a
// position's keys and values lie, which rows and positions a sequence has, how attention is split.
// Host and device code include it.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "hcr_layout.h"
#include "hcr_paged.h"
#include "hcr_paged_q8.h"

#if defined(__HIPCC__)
#define HCR_HD __host__ __device__ inline __attribute__((always_inline))
#else
#define HCR_HD inline
#endif

namespace hcr {

// ---- geometry
constexpr int GROUP_MAX = 64;  // heads of one kv head
HCR_HD bool page_ok(int page) { return page == 32 || page == 64 || page == 128 || page == 256; }
HCR_HD bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }
HCR_HD int log2_of(int pow2) {
  int s = 0;
  while ((1 << s) < pow2) ++s;
  return s;
}

// What the kernels take of a cache and of a batch (by value).
struct CacheArgs {
  uint16_t* k;  // BF16 bits
  uint16_t* v;
  uint16_t* means;
  int n_pages, kv_heads, head_dim, shift;  // page = 1 << shift
};
// What they take besides of a cache of codes (code HCR_BF16: none, BF16 pages).
struct CodeArgs {
  float* k_scales;
  float* v_scales;
  int code;
};
HCR_HD bool coded(const CodeArgs& x) { return x.code == HCR_INT8 || x.code == HCR_E4M3; }
// The positions that a token sees: all up to its own (size 0), or its last `size` and the first `first`.
struct WindowArgs {
  int size, first;
};
struct BatchArgs {
  const int* q_start;
  const int* ctx_len;
  const int* table;
  int table_stride, n_seqs, n_tokens, max_tokens, max_ctx;
};

// First element of head h of a page (k_pages and v_pages alike; 64 bits: a cache passes 2^31 elements).
HCR_HD size_t head_base(const CacheArgs& c, int page, int h) {
  return ((size_t)page * c.kv_heads + h) * ((size_t)c.head_dim << c.shift);
}
// Element of dimension d of slot s within a head's page.
HCR_HD int k_at(int shift, int s, int d) { return (((d >> 3) << shift) + s) * 8 + (d & 7); }
HCR_HD int v_at(int head_dim, int s, int d) { return ((s >> 3) * head_dim + d) * 8 + (s & 7); }
// The same for codes, 16 in the place of 8, and a slot's scale.
HCR_HD int k_code_at(int shift, int s, int d) { return (((d >> 4) << shift) + s) * 16 + (d & 15); }
HCR_HD int v_code_at(int head_dim, int s, int d) { return ((s >> 4) * head_dim + d) * 16 + (s & 15); }
HCR_HD size_t scale_base(const CacheArgs& c, int page, int h) { return ((size_t)page * c.kv_heads + h) << c.shift; }

// A sequence's rows [row, row + tokens) and the position of its first new token (negative where the sequence is
// shorter than its window), held to the bounds of the batch whatever q_start and ctx_len say.
struct Seq {
  int row, tokens, first;
};
HCR_HD Seq seq_of(const BatchArgs& b, int s0, int s1, int ctx) {
  Seq q{0, 0, 0};
  if (s0 < 0 || s0 >= b.n_tokens || s1 <= s0) return q;
  q.row = s0;
  q.tokens = s1 - s0;
  const int room = b.n_tokens - s0;
  if (q.tokens > room) q.tokens = room;
  if (q.tokens > b.max_tokens) q.tokens = b.max_tokens;
  if (ctx > b.max_ctx) ctx = b.max_ctx;
  if (ctx < 0) ctx = 0;
  q.first = ctx - q.tokens;
  return q;
}
// A table entry as a page of the cache, -1 where it is none.
HCR_HD int page_or_none(int page, int n_pages) { return page >= 0 && page < n_pages ? page : -1; }

HCR_HD int ceil_div(int a, int b) { return (a + b - 1) / b; }

// ---- attention: 16-row tiles of a unit's rows (a sequence's window x group, or one token's group for listed
// pages), tiles of 32 positions, and splits of the length into chunks of tiles
constexpr int TILE = 32;
constexpr int TILE_SHIFT = 5;
// A wave's tile of codes has 64 positions, so that it has as many bytes on their way as of BF16 (and 32 of D = 256, whose
// accumulators leave no room for more): 64 sequences of up to 8,192 positions, D = 128, whole, 108 us where tiles of 32
// took 143.
constexpr int tile_shift(bool codes, int D) { return codes && D != 256 ? TILE_SHIFT + 1 : TILE_SHIFT; }
// Tiles of work-groups whose four waves share their rows (hcr_attn_rows.h): 16 keys a wave.
constexpr int ROWS_SHIFT = 6;
// Pages of codes hold a tile of either kind at least.
HCR_HD bool code_page_ok(int page) { return page_ok(page) && page >= 64; }
// Waves of a work-group at most: what its registers leave room for on a CU (one 16-row tile of D = 256 takes 249
// of 512 registers of a lane, two 334; of D = 128 153 and 207; of D = 64 105).
constexpr int attn_waves(int D, int q_tiles) { return D == 64 ? 16 : D == 256 && q_tiles > 1 ? 4 : 8; }
// Work-groups of four waves that share their rows, on a CU: the registers are held to that.  As many as spill no more
// than a dozen of them (measured, codes: D = 128, 20 rows of 200,000 positions 103 us with four, 113 with two; D = 64 70
// against 84, 64 rows through a window of 1,024 68 with four, 77 with three).  D = 256 of three row tiles: with three
// work-groups E4M3 spills 27 (36 rows, two against three: 4 sequences of up to 9,001 38 and 47, one of 100,000 100 and
// 114, of 400,000 359 both), int8 none, which gains by the third only over long sequences (42 and 44, 115 and 111, 399
// and 383): two for both.
constexpr int rows_held(int D, int q_tiles) { return D == 256 ? (q_tiles > 2 ? 2 : 3) : D == 128 && q_tiles > 2 ? 3 : 4; }

// How a call is cut.  Its sets of rows (a sequence's window; one token for listed pages) have their tiles one set
// behind the other, and the work-groups of a kv head and row block take equal runs of them: as many work-groups as
// the chip holds at once, none with much more to do than another, however unlike the lengths are and however far
// below the bounds.  The host fixes the number of work-groups, the device the run's length.  Where the work-groups
// suffice, every set begins a run of its own (a second set costs a work-group the wait for its first loads again);
// else a run goes on from one set to the next.
// Sets of more rows than a work-group takes may have unlike numbers of row blocks (a prompt many, a single token one),
// which the host does not know: with several of them the device counts the pairs of a set and a row block (pair_cut).
struct AttnPlan {
  int q_tiles;     // 16-row tiles a wave holds
  int row_waves;   // waves of a work-group over the rows
  int groups;      // waves of a work-group over its tiles, for each of them
  int row_blocks;  // work-groups over a set's rows
  int items;       // work-groups over the tiles
  int least;       // tiles that are worth a work-group
  int whole;       // a work-group for each set instead, with all of its tiles: nothing to join
  int shared;      // the work-group's four waves share q_tiles row tiles, and tiles of 64 positions
  int paired;      // work-groups of a kv head over the pairs of a set and a row block; 0: they are not counted
  int shares;      // work-groups of a kv head that the chip holds at once
};
HCR_HD int attn_rows(const AttnPlan& p) { return p.row_waves * p.q_tiles * 16; }  // of a work-group
// Tiles of one run, from those of all sets (every set has one at least: a set without positions writes its zeros).
HCR_HD int run_tiles(const AttnPlan& p, int tiles_of_all) {
  const int even = ceil_div(tiles_of_all, p.items);
  return even > p.least ? even : p.least;
}
// The same with each of `sets` sets beginning a run: at most so many runs more; 0 where that makes them longer by
// more than a sixteenth.
HCR_HD int run_tiles_apart(const AttnPlan& p, int tiles_of_all, int sets) {
  if (sets >= p.items) return 0;
  const int even = ceil_div(tiles_of_all, p.items - sets);
  const int run = even > p.least ? even : p.least;
  return 16ll * run <= 17ll * run_tiles(p, tiles_of_all) ? run : 0;
}
// Listed pages: every token's list in as many runs.
HCR_HD int run_tiles_listed(const AttnPlan& p, int list_tiles, int n_tokens) {
  const int even = ceil_div(list_tiles, p.items / n_tokens);
  return even > p.least ? even : p.least;
}
// The runs that a set's tiles [first, first + tiles) lie in: a row's parts, to be joined where there are several.
// A run has two places for parts: of the set that began before it, and of the set that goes on behind it.
HCR_HD int run_parts(int first, int tiles, int run) { return (first + tiles - 1) / run - first / run + 1; }
HCR_HD int part_slot(int run_index, int run, int first) { return 2 * run_index + (first >= run_index * run); }
// Row blocks of a set of `rows` rows, and how many pairs there are at most.
HCR_HD int set_blocks(const AttnPlan& p, int rows) { return ceil_div(rows, attn_rows(p)); }
HCR_HD long long pairs_bound(const AttnPlan& p, long long sets, long long rows_of_all) {
  const long long each = sets * p.row_blocks, all = sets + rows_of_all / attn_rows(p);
  return each < all ? each : all;
}
// How pairs are cut, from the tiles of all of them, their number, that of the sets, and the row blocks of those that have
// rows:
//   ALIKE  as many row blocks each, more runs than one of each row block, or (of more than 64 sets, which take a work-group
//          longer to look through than to go through) enough row blocks for the chip: each row block's tiles as one row
//          block's sets are cut, in `items` equal runs that may go on from one set to the next
//   EVEN   no more pairs than the chip's share for a kv head: the tiles of all pairs, one behind the other, in one equal
//          run for each share
//   APART  more of them: each by itself, what is longer than half a share and than the average pair (by a sixteenth: what
//          is not much longer stays whole) in several runs
enum PairKind { ALIKE, EVEN, APART };
struct PairCut {
  int kind, run, blocks;  // ALIKE: row blocks of a set
  int joins;              // whether a pair has several parts
};
HCR_HD PairCut pair_cut(const AttnPlan& p, long long tiles, int pairs, int sets, int fewest_blocks, int most_blocks) {
  constexpr long long MOST = 1 << 26;  // a pair has 2^25 at most
  if (p.whole || pairs == 0) return PairCut{APART, (int)MOST, 0, 0};
  if (fewest_blocks == most_blocks && (p.items > 1 || (sets > 64 && most_blocks >= p.shares)))
    return PairCut{ALIKE, 0, most_blocks, p.items > 1};
  const bool even = pairs <= p.shares && tiles < 1 << 30;
  const int parts = even ? p.shares : 2 * p.shares < pairs ? 2 * p.shares : pairs;
  long long run = (tiles + parts - 1) / parts;
  if (!even) run += run / 16;
  run = run > p.least ? run : p.least;
  return PairCut{even ? EVEN : APART, (int)(run < MOST ? run : MOST), 0, 1};
}
// A pair APART in even runs: `parts` of `each` tiles (the last may be shorter).  One that is cut has less than twice
// tiles / run parts, all of them together less than four for each share.
struct PairRuns {
  int parts, each;
};
HCR_HD PairRuns pair_runs(int tiles, int run) {
  const int each = ceil_div(tiles, ceil_div(tiles, run));
  return PairRuns{ceil_div(tiles, each), each};
}
// Work-groups of a call.
HCR_HD long long attn_grid(const CacheArgs& c, const AttnPlan& p) {
  const long long items = (long long)(p.paired ? p.paired : p.items) * c.kv_heads;
  return (items + XCDS - 1) / XCDS * XCDS * (p.paired ? 1 : p.row_blocks);
}
// Places for parts of a kv head.
HCR_HD long long attn_slots(const AttnPlan& p) {
  return p.paired ? 4ll * p.shares : 2ll * p.items * p.row_blocks;
}
// Whether a set may have several parts, to be joined by a second launch.
HCR_HD bool attn_joins(const AttnPlan& p) { return !p.whole && (p.paired || p.items > 1); }
// Bytes of LDS of a work-group: its query rows, in their place what its groups join in, a 16-row tile of each wave
// at a time, and the groups' (m, l).
HCR_HD int attn_lds(int D, const AttnPlan& p) {
  const int rows = attn_rows(p);
  return p.groups > 1 ? p.groups * (p.row_waves * 16 * D * 4 + rows * 8) : rows * D * 2;
}
AttnPlan attn_plan(const CacheArgs& c, const BatchArgs& b, int heads, int n_sel);
// The plan over codes or over a window.
AttnPlan attn_plan_more(const CacheArgs& c, const CodeArgs& x, const WindowArgs& w, const BatchArgs& b, int heads,
                        int n_sel);

// The tiles that rows of lengths len_min to len_max (a row's position + 1; 0 and less: it sees nothing) see through a
// window: the first `firsts`, then those from tile `low` on.
struct WindowTiles {
  int firsts, low, tiles;
};
HCR_HD WindowTiles window_tiles(const WindowArgs& w, int len_min, int len_max, int shift) {
  const int start = len_min > w.size ? len_min - w.size : 0;
  WindowTiles t;
  t.low = start >> shift;
  t.firsts = (w.first + (1 << shift) - 1) >> shift;
  if (t.firsts > t.low) t.firsts = t.low;
  t.tiles = t.firsts + (len_max > 0 ? ((len_max - 1) >> shift) + 1 - t.low : 0);
  if (t.tiles < 1) t.tiles = 1;
  return t;
}

// Tiles that rows of `tokens` consecutive tokens see at most, none of them past position max_ctx (size 0: all).
HCR_HD int window_bound(const WindowArgs& w, int max_ctx, long long tokens, int shift) {
  const long long one = 1ll << shift, all = (max_ctx + one - 1) >> shift;
  if (!w.size) return (int)all;
  const long long most = ((w.first + one - 1) >> shift) + ((w.size + tokens + one - 2) >> shift) + 1;
  return (int)(all < most ? all : most);
}
// The tiles that each of a set's row blocks counts as, where pairs are counted: those of the block that has most (one at least).
HCR_HD int pair_tiles(const AttnPlan& p, const WindowArgs& w, const Seq& s, int group, int shift) {
  const int len = s.first + s.tokens, block = ceil_div(attn_rows(p), group) + 1;  // tokens of a row block
  const int tiles = len > 0 ? window_bound(w, len, block < s.tokens ? block : s.tokens, shift) : 0;
  return tiles > 1 ? tiles : 1;
}

struct AttnArgs {
  CacheArgs c;
  BatchArgs b;
  const uint16_t* q;
  const int* sel;  // null: every page
  int n_sel, heads, group, out_type;
  float scale_hi, scale_lo;  // scale / ln 2 (probabilities are powers of two) in two parts
  void* out;
  float* part;  // [kv_heads][slots][rows][D], then (m, l) pairs [kv_heads][slots][rows]; slots: [row_blocks][items][2], or
                // of cut pairs alone; behind them the PairCut that the join goes by
  AttnPlan plan;
  CodeArgs code;
  WindowArgs window;
};
int launch_attn(const AttnArgs& a, void* stream);  // of every kind: takes those below
int launch_attn_window(const AttnArgs& a, void* stream);
int launch_attn_int8(const AttnArgs& a, void* stream);
int launch_attn_e4m3(const AttnArgs& a, void* stream);

// ---- append
// Aligned parts of `1 << shift` positions that so many consecutive ones can touch.
HCR_HD int parts_touched(int tokens, int shift) { return ((tokens - 1 + (1 << shift) - 1) >> shift) + 1; }
struct AppendArgs {
  CacheArgs c;
  BatchArgs b;
  hcr_rows q, k, v;
  int heads, type;
  const float *q_norm, *k_norm, *rope;
  float eps;
  int rope_dim, rope_style;
  uint16_t* q_out;
  CodeArgs code;
};
int launch_append(const AppendArgs& a, void* stream);  // of either kind
int launch_append_q8(const AppendArgs& a, void* stream);
constexpr int APPEND_THREADS = 256;
constexpr int APPEND_EACH = 4;  // tokens of a work-group of query heads, one where there are few
HCR_HD int append_each(const BatchArgs& b) { return b.max_tokens >= 32 ? APPEND_EACH : 1; }
// Work-groups: first those of (sequence, page, kv head, k or v), then those of (sequence, tokens, query heads).
struct AppendGrid {
  int pages, passes;  // pages that a window can touch; work-groups over the query heads
  long long kv_groups, groups;
};
HCR_HD AppendGrid append_grid(const CacheArgs& c, const BatchArgs& b, int heads) {
  AppendGrid g;
  g.pages = parts_touched(b.max_tokens, c.shift);
  g.passes = ceil_div(heads, APPEND_THREADS / (c.head_dim / 8));
  g.kv_groups = (long long)b.n_seqs * g.pages * c.kv_heads * 2;
  g.groups = g.kv_groups + (long long)b.n_seqs * ceil_div(b.max_tokens, append_each(b)) * g.passes;
  return g;
}

// ---- read back
struct ReadArgs {
  CacheArgs c;
  CodeArgs code;
  BatchArgs b;
  int out_type;
  void *k_out, *v_out;  // either may be null
};
int launch_read(const ReadArgs& a, void* stream);
constexpr int READ_THREADS = 256;
constexpr int READ_SHIFT = 6;
constexpr int READ_SLOTS = 1 << READ_SHIFT;  // positions of a work-group
// The aligned position that a sequence's parts begin at (negative for a padded one), and the parts of READ_SLOTS that its
// rows can touch.
HCR_HD int read_start(int first) { return first & ~(READ_SLOTS - 1); }
HCR_HD int read_parts(const BatchArgs& b) { return parts_touched(b.max_tokens, READ_SHIFT); }

// ---- scores and selection
struct ScoreArgs {
  CacheArgs c;
  BatchArgs b;
  const uint16_t* q;
  int heads, group;
  float* scores;
  int stride;
};
int launch_block_scores(const ScoreArgs& a, void* stream);

struct TopkArgs {
  BatchArgs b;
  const float* scores;
  int stride, kv_heads, shift, n_sel, n_first, n_last;
  int* sel;
};
int launch_block_topk(const TopkArgs& a, void* stream);

}  // namespace hcr
