// Index arithmetic of the paged cache, shared by its kernels, the C ABI and a host-compiled test: where a
// position's keys and values lie, which rows and positions a sequence has, how attention is split.
// Host and device code include it.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "hcr_layout.h"
#include "hcr_paged.h"

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
// Waves of a work-group at most: what its registers leave room for on a CU (one 16-row tile of D = 256 takes 249
// of 512 registers of a lane, two 334; of D = 128 153 and 207; of D = 64 105).
constexpr int attn_waves(int D, int q_tiles) { return D == 64 ? 16 : D == 256 && q_tiles > 1 ? 4 : 8; }

// How a call is cut.  Its sets of rows (a sequence's window; one token for listed pages) have their tiles one set
// behind the other, and the work-groups of a kv head and row block take equal runs of them: as many work-groups as
// the chip holds at once, none with much more to do than another, however unlike the lengths are and however far
// below the bounds.  The host fixes the number of work-groups, the device the run's length.  Where the work-groups
// suffice, every set begins a run of its own (a second set costs a work-group the wait for its first loads again);
// else a run goes on from one set to the next.
struct AttnPlan {
  int q_tiles;     // 16-row tiles a wave holds
  int row_waves;   // waves of a work-group over the rows
  int groups;      // waves of a work-group over its tiles, for each of them
  int row_blocks;  // work-groups over a set's rows
  int items;       // work-groups over the tiles
  int least;       // tiles that are worth a work-group
  int whole;       // a work-group for each set instead, with all of its tiles: nothing to join
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
// Whether a set may have several parts, to be joined by a second launch.
HCR_HD bool attn_joins(const AttnPlan& p) { return p.items > 1 && !p.whole; }
// Bytes of LDS of a work-group: its query rows, in their place what its groups join in, a 16-row tile of each wave
// at a time, and the groups' (m, l).
HCR_HD int attn_lds(int D, const AttnPlan& p) {
  const int rows = attn_rows(p);
  return p.groups > 1 ? p.groups * (p.row_waves * 16 * D * 4 + rows * 8) : rows * D * 2;
}
AttnPlan attn_plan(const CacheArgs& c, const BatchArgs& b, int heads, int n_sel);

struct AttnArgs {
  CacheArgs c;
  BatchArgs b;
  const uint16_t* q;
  const int* sel;  // null: every page
  int n_sel, heads, group, out_type;
  float scale_hi, scale_lo;  // scale / ln 2 (probabilities are powers of two) in two parts
  void* out;
  float* part;  // [kv_heads][row_blocks][items][2][rows][D], then (m, l) pairs [kv_heads][row_blocks][items][2][rows]
  AttnPlan plan;
};
int launch_attn(const AttnArgs& a, void* stream);

// ---- append
struct AppendArgs {
  CacheArgs c;
  BatchArgs b;
  hcr_rows q, k, v;
  int heads, type;
  const float *q_norm, *k_norm, *rope;
  float eps;
  int rope_dim, rope_style;
  uint16_t* q_out;
};
int launch_append(const AppendArgs& a, void* stream);
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
  g.pages = ((b.max_tokens - 1) >> c.shift) + 2;
  g.passes = ceil_div(heads, APPEND_THREADS / (c.head_dim / 8));
  g.kv_groups = (long long)b.n_seqs * g.pages * c.kv_heads * 2;
  g.groups = g.kv_groups + (long long)b.n_seqs * ceil_div(b.max_tokens, append_each(b)) * g.passes;
  return g;
}

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
