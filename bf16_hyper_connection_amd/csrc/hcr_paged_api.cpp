// C ABI of the paged cache: argument checks, the handle and the plan of an attention call.  Every check runs on
// the host before any HIP call.

#include <float.h>
#include <math.h>
#include <stdint.h>
#include <stdlib.h>

#include "hcr_paged_check.h"

namespace hcr {

namespace {

size_t scratch_of(const CacheArgs& c, const AttnPlan& p) {
  if (!attn_joins(p)) return 0;
  return align256((size_t)c.kv_heads * attn_slots(p) * attn_rows(p) * (c.head_dim + 2) * 4 +
                  (p.paired ? sizeof(PairCut) : 0));
}

// The plan of any kind of call.
AttnPlan plan_of(const hcr_cache& h, const BatchArgs& b, int heads, int n_sel, const WindowArgs& w) {
  return coded(h.code) || w.size ? attn_plan_more(h.args, h.code, w, b, heads, n_sel)
                                 : attn_plan(h.args, b, heads, n_sel);
}
// A window held to the longest sequence: no sum with a position passes 32 bits.
WindowArgs held(WindowArgs w, const BatchArgs& b) {
  const int most = b.max_ctx > 1 ? b.max_ctx : 1;
  if (w.size > most) w.size = most;
  if (w.first > most) w.first = most;
  return w;
}

}  // namespace

int attn(hcr_cache_t h, const hcr_batch* batch, int heads, double scale, const void* q, const int* sel, int n_sel,
         const WindowArgs& w, int out_type, void* out, void* scratch, size_t scratch_bytes, void* stream) {
  if (!h) return HCR_EINVAL;
  const CacheArgs& c = h->args;
  AttnArgs a{};
  a.c = c;
  const int rc = check_bounds(c, batch, heads, &a.b);
  if (rc < 0) return rc;
  if (out_type != HCR_F32 && out_type != HCR_BF16) return HCR_EINVAL;
  if (!(scale > -1e30 && scale < 1e30)) return HCR_EINVAL;  // NaN and infinite too
  if (!lists_fit(c, a.b, n_sel)) return HCR_EINVAL;
  if (rc == 1) return HCR_OK;
  if (!q || !out) return HCR_EINVAL;
  if (const int e = check_arrays(a.b)) return e;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(sel, 4) || !aligned(scratch, 256)) return HCR_EALIGN;
  a.code = h->code;
  a.window = held(w, a.b);
  a.plan = plan_of(*h, a.b, heads, n_sel, a.window);
  if (attn_grid(c, a.plan) * 64 * 16 > THREADS_MAX || (long long)a.b.n_tokens * heads * 256 > THREADS_MAX)
    return HCR_EINVAL;
  const size_t need = scratch_of(c, a.plan);
  if (need && (!scratch || scratch_bytes < need)) return HCR_ESCRATCH;
  const size_t values = (size_t)a.b.n_tokens * heads * c.head_dim;
  const Span so = span(out, values * (out_type == HCR_F32 ? 4 : 2)), sq = span(q, values * 2);
  const Span ss = need ? span(scratch, need) : Span{0, 0};
  const Span sl = span(sel, (size_t)a.b.n_tokens * c.kv_heads * n_sel * 4);
  const Span written[] = {so, ss};
  if (overlap(so, ss)) return HCR_EALIAS;
  for (const Span& s : written)
    if (overlap(s, sq) || overlap(s, sl) || overlap_any(s, cache_spans(*h)) || overlap_any(s, batch_spans(a.b)))
      return HCR_EALIAS;
  a.q = static_cast<const uint16_t*>(q);
  a.sel = sel;
  a.n_sel = n_sel;
  a.heads = heads;
  a.group = heads / c.kv_heads;
  a.out_type = out_type;
  const double log2e = scale * 1.4426950408889634;
  // both parts of one sign, neither zero (the least FP32 value if need be): a product of -inf stays -inf and weighs
  // nothing
  a.scale_hi = (float)log2e;
  if (fabs(a.scale_hi) >= fabs(log2e)) a.scale_hi = nextafterf(a.scale_hi, 0.f);
  a.scale_lo = (float)(log2e - a.scale_hi);
  // (over codes and windows for a scale of zero too: what a row does not see is hidden ahead of the product)
  if (scale != 0 || coded(a.code) || a.window.size) {
    const float least = copysignf(FLT_TRUE_MIN, (float)scale);
    if (a.scale_hi == 0.f) a.scale_hi = least;
    if (a.scale_lo == 0.f) a.scale_lo = least;
  }
  a.out = out;
  a.part = static_cast<float*>(scratch);
  return launch_attn(a, stream);
}

size_t attn_scratch(hcr_cache_t h, const hcr_batch* batch, int heads, int n_sel, const WindowArgs& w) {
  BatchArgs b;
  if (!h || check_bounds(h->args, batch, heads, &b) != HCR_OK || !lists_fit(h->args, b, n_sel)) return 0;
  return scratch_of(h->args, plan_of(*h, b, heads, n_sel, held(w, b)));
}

int check_cache(const CacheArgs& c, const CodeArgs& x) {
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.means, 16) || !aligned(x.k_scales, 16) ||
      !aligned(x.v_scales, 16))
    return HCR_EALIGN;
  const CacheSpans s = cache_spans(c, x);
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(s.s[i], s.s[j])) return HCR_EALIAS;
  return HCR_OK;
}

int new_cache(const CacheArgs& c, const CodeArgs& x, hcr_cache_t* out) {
  hcr_cache* h = static_cast<hcr_cache*>(malloc(sizeof(hcr_cache)));
  if (!h) return HCR_EINVAL;
  h->args = c;
  h->code = x;
  *out = h;
  return HCR_OK;
}

// Several sets of several row blocks: the device counts the pairs of a set and a row block (pair_cut).  Where the bounds
// would have a work-group take 2,048 positions and more (the search takes each about 3 us: 40 sequences of up to 9 tokens, 32
// heads of 64 over 2, BF16 (int8): at up to 2,500 positions 37.9 us without it, 39.6 with it (42.7, 47.4), at 9,000 75.7 and
// 71.0 (80.4 and 77.3)); of whole sets where there would be several rounds of work-groups, less than half of them with
// rows.  fill: work-groups that the chip holds at once.
// Measured (us a call, D = 128, 32 heads over 8, against a plan in which each row block of the longest prompt takes runs
// over all sets):
//   a prompt of 2,048 and 63 single tokens of up to 8,192: int8 331 against 7,730, BF16 801 against 14,420, through a window
//   of 5,000 330 against 6,220; of up to 4,096 (whole) int8 225 against 467, BF16 448 against 1,262.  300 sequences of
//   5,000, 3 prompts of 700 among them, D = 64: int8 608 against 16,100; 512 tokens at 60,000 beside three single ones
//   1,051 against 2,360; 3 prompts of 1,000 to 1 through a window of 6,000 298 against 400; 4 of 300 at 9,000 (BF16, D =
//   64) 609 against 781.  Alike sets pay for the count (3 of 128 at 9,000 141 against 138, 200 of 30 at
//   5,000, D = 64 1,504 against 1,493, BF16 1,650 against 1,588)
static void plan_pairs(AttnPlan& p, const CacheArgs& c, const BatchArgs& b, int group, int fill, long long span) {
  if (p.row_blocks == 1 || b.n_seqs == 1 || (!p.whole && b.n_seqs * span < 2048ll * p.items)) return;
  const long long pairs = pairs_bound(p, b.n_seqs, (long long)b.n_tokens * group);
  const long long each = (long long)b.n_seqs * p.row_blocks;
  if (p.whole && (2 * pairs >= each || each * c.kv_heads < 4096)) return;
  const int shares = fill / c.kv_heads > 1 ? fill / c.kv_heads : 1;
  const long long paired = pairs + (p.whole ? 0 : 2 * shares);
  if ((paired + XCDS) * c.kv_heads * 1024 > THREADS_MAX) return;  // what a launch does not hold is cut as it was
  p.shares = shares;
  p.paired = (int)paired;
}

// Measured on MI355X, 8 kv heads, graphs of calls on rotated inputs (us a call), lengths from an eighth of the
// longest up to it:
//   row tiles  two 16-row tiles a wave from 17 rows on.  D = 128: 24 rows 154 against 160, 64 rows 161 against 185.
//              D = 256 up to 32 rows, a wave a SIMD: 24 rows of 4 sequences of 90,010 260 against 302, of 64 of
//              4,000 197 against 257.  49 to 64 rows too, in two row waves, where there are tiles for them: 64 rows of
//              16,400 50 against 58, 4 sequences of 60,000 233 against 258, but 32 of 700 71 against 61, one of 9,001 36
//              against 35 (36 rows level, 54 against 52 at 9,001).  Not D = 64 (92 against 90), nor three for D = 256
//              (36 rows 283 against 303, but 57 against 51 at 9,001: the accumulators no longer fit beside the operands)
//   rows       several row waves, D = 256: one group, as many work-groups as fit a CU (36 rows: 314 against 432
//              with two groups), four row waves at most (96 rows: 484 against 544 with six in one work-group)
//   whole      a work-group a set and no join, where the chip is full of them or they end soon.  512 work-groups,
//              D = 128: up to 300 positions 14 against 28, 700 24 against 33, 4,000 93 against 104; 256: 700 16
//              against 28, 2,000 35 against 39 (D = 256 66 against 64), 8,192 127 against 101; 8: 300 7.1 against
//              9.7, 700 9.2 against 9.7, 1,200 11.4 against 9.6 (earlier for D = 256, whose tiles are twice the
//              bytes: a CU alone takes about 35 GB/s).  36 rows of D = 256: 700 63 against 74, 2,000 158 against
//              153.  Beyond 4,096 the runs stay, although lengths as even as these would still gain 5 % (8,192: 184
//              against 194): one long sequence among short ones would hold a single CU for the whole call
//   apart      every set begins a run of its own where runs get no more than a sixteenth longer by it (run_tiles_apart;
//              a quarter was slower for a few long sequences): 12 single tokens over up to 3,127 positions 19.0 against
//              22.9
//   least      a run has a tile for each of its waves, and a sixteenth as many tiles as rows, whose part is written and
//              read again (37 windows of 224 rows of D = 256 over up to 249: 24.4 against 34.6 with a tile a run); but
//              fewer, down to a tile (two for up to 16 rows), where that leaves no more runs than CUs: 56 rows of 2
//              sequences of 483 12.1 against 15.4, 128 rows of 328 18.3 against 20.5, 2 single tokens over 4,988
//              (D = 128) 11.1 against 12.5; without that bound 40 single tokens over up to 2,050 19.3 against 15.9
//   waves      16 for D = 64 with more than 64 rows (42 windows of 192 rows over up to 913 positions: 23 against 32
//              with 8).  Else 8 a work-group, one work-group a CU, for long sequences (D = 256, one of 420,000: 568
//              against 575 with 4); 4, two work-groups a CU, for runs where no sequence is longer than 2,048 (one of
//              2,000, D = 256: 13.4 against 14.5) and for many sets of up to 512 (300: 14 against 17), since a short
//              one is mostly the wait for its first loads
// The bounds are in positions, whatever a tile has (BF16 and codes of D = 256 32, codes of D <= 128 64).
// Over codes (the same calls, whole or with four waves against the other):
//   whole      fewer sets than CUs: a set in one work-group takes longer with its length, in runs with the number of sets,
//              more past 64, which a wave does not see at once.  One, D = 128, three caches in turn: 640 positions 9.9
//              against 10.3, 768 9.7 against 10.4, 832 11.9 against 10.6; a call that is not in a graph takes 2.5 more for
//              the second launch.  D = 64: 768 8.4 against 10.1, 1,024 9.8 against 10.0; D = 256: 384 10.8 against 11.4,
//              448 12.4 against 11.2.  128 work-groups (16 sets of 8 heads, rotated caches), D = 128: 1,200 16.7 against
//              17.4, 1,600 20.2 against 17.9; 192: 2,200 25.4 against 33.8, 3,000 32.7 against 34.7; D = 256 128: 700 19.9
//              against 19.2, 192: 1,600 35.7 against 35.6; D = 64 128: 2,200 16.8 against 20.0.  72 sets of one head, D =
//              128: 1,200 16.3 against 20.2, 2,200 23.7 against 23.3
//              32 sets, D = 128: of 3,000 33.5 against 38.9, 4,096 42 against 43; D = 256: 3,000 64 against 57.  64
//              and more to 4,096 as above: one of 8,192 beside 63 of 100 takes 24 in runs, 66 whole, one of 5,000 28
//              and 45 (lengths from an eighth of 8,192 up to it 114 and 105, all of 8,192 174 and 177)
//   waves      four for 64 and more whole sets of up to 1,024 (D = 256, 64 of 700 29.8 against 32.4, 128 47.9 against 60.4),
//              for runs of few sets up to 4,096 (8 of 4,096 20.3 against 23.3), and for runs of more than CUs' sets of any
//              length: 64 of up to 8,192 115 against 128 with eight, 12,000 156 against 168, 20,000 246 against 253
static AttnPlan plan_for(const CacheArgs& c, const BatchArgs& b, int heads, int n_sel, int tiles, int shift, bool one_tile,
                         bool codes) {
  constexpr int CUS = 256;
  AttnPlan p{};
  const int group = heads / c.kv_heads;
  const int rows = n_sel ? group : b.max_tokens * group;
  const bool wide = c.head_dim == 256;
  const long long sets = n_sel ? b.n_tokens : b.n_seqs;
  const long long span = (long long)tiles << shift;  // positions of a set at most
  const bool lengthy = rows > 48 && rows <= 64 && span >= 8192 && sets * span >= 16384;
  p.q_tiles = !one_tile && rows > 16 && (c.head_dim == 128 || (wide && (rows <= 32 || lengthy))) ? 2 : 1;
  const int row_tiles = ceil_div(rows, 16 * p.q_tiles);
  p.row_blocks = ceil_div(row_tiles, wide ? 4 : 8);
  p.row_waves = ceil_div(row_tiles, p.row_blocks);
  const bool alone = wide && p.row_waves > 1;  // row waves fill a work-group
  // waves of a work-group: 8, more where many row waves of D = 64 leave room, 4 of two wide row tiles
  const int room = attn_waves(c.head_dim, p.q_tiles);
  const int waves = room > 8 && p.row_waves <= 4 ? 8 : room;
  const int most_groups = alone ? 1 : waves / p.row_waves;

  const int units = c.kv_heads * p.row_blocks;
  const long long full = sets * units;  // work-groups of whole sets
  // positions up to which a work-group takes a whole set, and up to which four waves a work-group do
  long long whole_to, few_to;
  if (full < CUS) {
    whole_to = wide ? (rows > 16 ? 192 : 384) : 96 * most_groups;
    if (codes) {
      const long long over = full > 64 ? full - 64 : 0, most = wide ? 2048 : 4096;
      whole_to = (c.head_dim == 64 ? 1024 : whole_to) * (sets > 64 ? 2 : 1) * (4096 + over * over) / 4096;
      if (whole_to > most) whole_to = most;
    }
  } else if (n_sel) {
    whole_to = span;  // lists are alike
  } else if (alone) {
    whole_to = 1024;
  } else {
    whole_to = full < 2 * CUS && !(codes && !wide) ? 2048 : 4096;
  }
  p.whole = span <= whole_to;
  if (p.whole)
    few_to = full < 2 * CUS ? -1 : codes ? 1024 : 512;
  else
    few_to = n_sel ? -1 : !codes ? 2048 : full < CUS ? 4096 : span;
  const bool few = span <= few_to;
  p.groups = few && p.row_waves <= 4 && most_groups > 4 / p.row_waves ? 4 / p.row_waves : most_groups;
  if (p.groups > tiles) p.groups = tiles;
  if (p.groups < 1) p.groups = 1;

  // tiles that are worth a work-group, fewer where there are work-groups to spare
  const int part_rows = rows < attn_rows(p) ? rows : attn_rows(p);
  const int worth = p.groups > part_rows / 16 ? p.groups : part_rows / 16;
  const long long even = (sets * units * tiles + CUS - 1) / CUS;
  p.least = even < worth ? (int)even : worth;
  if (p.least < (rows > 16 ? 1 : 2)) p.least = rows > 16 || worth == 1 ? 1 : 2;
  const int held = (room < 8 ? room : 8) / (p.row_waves * p.groups);  // work-groups of a CU
  const int fill = CUS * (held > 1 ? held : 1);
  const long long runs = ceil_div(tiles > 0 ? tiles : 1, p.least);  // of a set at most
  long long items = fill / units;
  if (n_sel) {
    items /= sets;
    items = (items > runs ? runs : items > 1 ? items : 1) * sets;
  } else if (items > runs * sets) {
    items = runs * sets;
  }
  p.items = p.whole ? (int)sets : items > 1 ? (int)items : 1;
  if (!n_sel) plan_pairs(p, c, b, group, fill, span);
  return p;
}

AttnPlan attn_plan(const CacheArgs& c, const BatchArgs& b, int heads, int n_sel) {
  return plan_for(c, b, heads, n_sel, n_sel ? n_sel << (c.shift - TILE_SHIFT) : ceil_div(b.max_ctx, TILE), TILE_SHIFT,
                  false, false);
}

// Work-groups of four waves that share their rows (hcr_attn_rows.h), up to four row tiles each.  As few row blocks as hold
// the rows, each with as few row tiles: a block reads the set's keys and values once.  Measured (us a call, graphs):
//   most       prompts whose blocks of 64 rows are fewer than two a CU (by the tokens there are, whatever the bounds): blocks
//              of 32, where those then take whole sets; a work-group alone on a CU is mostly waits.  Int8, 32 heads over 8:
//              one prompt of 512 15.5 against 20.9, of 1,000 28 against 36, 4 of up to 256 behind 2,048 48 against 63, one
//              of 512 through a window of 1,024 (BF16) 31 against 69.  Not where the chip is full of them (2 of 1,024 at
//              4,096, D = 256: 332 against 303) or where runs are cut (256 at 8,192: 106 against 93)
//   whole      a work-group a set where sets fill the chip and end soon.  D = 128, 24 rows: 64 sequences of 700 21
//              against 34, of 4,000 97 against 87, 128 of 4,000 121 against 155; 36 rows of D = 256: 32 of 700 33 against
//              36, 32 of 2,000 84 against 67, 16 of 700 32 against 27.  8 prompts of up to 512 at 4,096 200 against 295.
//              Never beyond 4,096 positions, as above
//   fill       work-groups a CU, by the tiles there are for each: one for up to 7, two for up to 15 (D = 256 31), three
//              for up to 31, else what registers leave room for; fewer, longer runs leave less to join and wait for their
//              first loads less often.  36 rows of D = 256: 16 of 700 23.5 with one, 28 with two; 16 of 2,000 38 with two,
//              42 with one, 40 with three; one of 60,000 78 with two, 80 with three.  24 rows: D = 128, one of 4,000 12.7
//              with one, 14.0 with two; 4 of 9,000 21.1 with three, 22.3 with two; one of 80,000 48.1 with four, 51.5 with
//              three; D = 64, 4 of 9,000 18.7 with three, 20.5 with two.  24 rows through a window of 8,192 21.5 with one,
//              23 with three
static AttnPlan rows_plan(const CacheArgs& c, const WindowArgs& w, const BatchArgs& b, int group, int n_sel) {
  constexpr int CUS = 256;
  AttnPlan p{};
  p.shared = 1;
  const int rows = n_sel ? group : b.max_tokens * group;
  const int row_tiles = ceil_div(rows, 16);
  const long long sets = n_sel ? b.n_tokens : b.n_seqs;
  const auto full_of = [&](int most) { return sets * c.kv_heads * ceil_div(row_tiles, most); };  // work-groups of whole sets
  const auto tiles_of = [&](int row_blocks) {
    const int block = ceil_div(16 * ceil_div(row_tiles, row_blocks), group) + 1;  // tokens of a row block
    return n_sel ? n_sel << (c.shift - ROWS_SHIFT)
                 : window_bound(w, b.max_ctx, block < b.max_tokens ? block : b.max_tokens, ROWS_SHIFT);
  };
  const auto whole_of = [&](long long full, int tiles) {
    return full < CUS ? tiles <= 4 : full < 2 * CUS ? tiles <= 16 : full < 4 * CUS ? tiles <= 32 : tiles <= 64;
  };
  int most = 4;
  if (!n_sel && row_tiles > 4 && (long long)c.kv_heads * ceil_div(b.n_tokens * group, 64) < 2 * CUS &&
      full_of(2) >= 2 * CUS && whole_of(full_of(2), tiles_of(ceil_div(row_tiles, 2))))
    most = 2;
  p.row_blocks = ceil_div(row_tiles, most);
  p.q_tiles = ceil_div(row_tiles, p.row_blocks);
  p.row_waves = p.groups = 1;
  const int tiles = tiles_of(p.row_blocks);
  const long long units = (long long)c.kv_heads * p.row_blocks, full = sets * units;
  p.whole = whole_of(full, tiles);
  const long long even = (full * tiles + CUS - 1) / CUS;  // of a CU
  p.least = 1;
  const int held = rows_held(c.head_dim, p.q_tiles);
  const int fill = CUS * (even < 8 ? 1 : even < 16 || (c.head_dim == 256 && even < 32) ? 2 : even < 32 ? 3 : held);
  const long long runs = tiles > 0 ? tiles : 1;
  long long items = fill / units;
  if (n_sel) {
    items /= sets;
    items = (items > runs ? runs : items > 1 ? items : 1) * sets;
  } else if (items > runs * sets) {
    items = runs * sets;
  }
  p.items = p.whole ? (int)sets : items > 1 ? (int)items : 1;
  if (!n_sel) plan_pairs(p, c, b, group, fill, (long long)tiles << ROWS_SHIFT);
  return p;
}

// Over codes and windows rows that fill more than one tile share a work-group's four waves: a row tile a wave would read
// (and widen) every page once a tile.  Measured, 8 kv heads (us, shared against a tile a wave): D = 256, 36 rows over
// 100,000 positions of int8 115 against 185, of E4M3 100 against 152; D = 128 over 200,000: 20 rows 97 against 119, 48
// 124 against 185, 64 147 against 200; D = 64, 20 rows 67 against 78; prompts of BF16 through a window 82 against 92.  Its
// tiles have 64 positions, so pages of 32 (BF16 through a window) keep a tile a wave
// (a prompt of 1,024, D = 128: through a window of 1,024 64 where pages of 64 take 46, of 5,000 227 and 120).  Up to 16 rows one wave has all of
// a tile's operands as loaded, with no barrier in its loop.
AttnPlan attn_plan_more(const CacheArgs& c, const CodeArgs& x, const WindowArgs& w, const BatchArgs& b, int heads,
                        int n_sel) {
  const int group = heads / c.kv_heads, rows = (n_sel ? 1 : b.max_tokens) * group;
  if (rows > 16 && c.shift >= ROWS_SHIFT) return rows_plan(c, w, b, group, n_sel);
  const int shift = tile_shift(coded(x), c.head_dim);
  const int tiles = n_sel ? n_sel << (c.shift - shift) : window_bound(w, b.max_ctx, b.max_tokens, shift);
  AttnPlan p = plan_for(c, b, heads, n_sel, tiles, shift, true, coded(x));
  // Windows of 4,096 are whole sets too, although the ends of their tiles are more: four waves, two work-groups a CU.  Sequences
  // longer than the window are then as long as each other: 64 windows of 4,096 of BF16 D = 128 165 us, in runs 175, D =
  // 64 84 against 96, D = 256 320 against 335, int8 94 against 98, 128 of them 178 against 192.  Those that are shorter
  // are not (one of 4,196 beside 63 of 200: 62 against 35), so that no longer window is: of 5,000 in runs 210 against 200,
  // 8,192 330 against 323, one of 5,100 beside 63 of 200 35 against 75.
  if (w.size && !p.whole && p.row_waves == 1 && p.groups >= 4 && ((long long)tiles << shift) <= 4096 + 256 &&
      (long long)b.n_seqs * c.kv_heads >= 512) {
    p.whole = 1;
    p.groups = 4;
    p.items = b.n_seqs;
  }
  return p;
}

}  // namespace hcr

using namespace hcr;

extern "C" {

size_t hcr_cache_pages_bytes(int n_pages, int kv_heads, int head_dim, int page) {
  if (n_pages < 1 || kv_heads < 1 || !head_dim_ok(head_dim) || !page_ok(page)) return 0;
  return (size_t)n_pages * kv_heads * head_dim * page * 2;
}

int hcr_cache_create(void* k_pages, void* v_pages, void* k_means, int n_pages, int kv_heads, int head_dim, int page,
                     hcr_cache_t* out) {
  if (!out) return HCR_EINVAL;
  *out = nullptr;
  if (!k_pages || !v_pages || n_pages < 1 || kv_heads < 1 || kv_heads > 4096 || !head_dim_ok(head_dim) ||
      !page_ok(page))
    return HCR_EINVAL;
  const CacheArgs c{static_cast<uint16_t*>(k_pages), static_cast<uint16_t*>(v_pages), static_cast<uint16_t*>(k_means),
                    n_pages, kv_heads, head_dim, log2_of(page)};
  const CodeArgs none{nullptr, nullptr, HCR_BF16};
  if (const int e = check_cache(c, none)) return e;
  return new_cache(c, none, out);
}

void hcr_cache_destroy(hcr_cache_t c) { free(c); }

int hcr_cache_append(hcr_cache_t h, const hcr_batch* batch, int heads, int type, const hcr_rows* q, const hcr_rows* k,
                     const hcr_rows* v, const float* q_norm, const float* k_norm, float eps, const float* rope,
                     int rope_rows, int rope_dim, int rope_style, void* q_out, void* stream) {
  if (!h) return HCR_EINVAL;
  const CacheArgs& c = h->args;
  AppendArgs a{};
  a.c = c;
  const int rc = check_bounds(c, batch, heads, &a.b);
  if (rc < 0) return rc;
  if (type != HCR_F32 && type != HCR_BF16) return HCR_EINVAL;
  if (!(eps >= 0.f) || eps - eps != 0.f) return HCR_EINVAL;
  if (rope_dim < 0 || rope_dim > c.head_dim || rope_dim % 16 || (rope_dim && !rope) ||
      (rope_dim && rope_rows < a.b.max_ctx) ||
      (rope_style != HCR_ROPE_HALVES && rope_style != HCR_ROPE_PAIRS))
    return HCR_EINVAL;
  if (rc == 1) return HCR_OK;
  if (!q_out) return HCR_EINVAL;
  if (const int e = check_arrays(a.b)) return e;
  if (!aligned(q_out, 16) || !aligned(q_norm, 16) || !aligned(k_norm, 16) || !aligned(rope, 16)) return HCR_EALIGN;
  Span in[6];
  if (const int e = check_rows(q, type, a.b.n_tokens, heads, c.head_dim, &in[0])) return e;
  if (const int e = check_rows(k, type, a.b.n_tokens, c.kv_heads, c.head_dim, &in[1])) return e;
  if (const int e = check_rows(v, type, a.b.n_tokens, c.kv_heads, c.head_dim, &in[2])) return e;
  in[3] = span(q_norm, (size_t)c.head_dim * 4);
  in[4] = span(k_norm, (size_t)c.head_dim * 4);
  in[5] = span(rope_dim ? rope : nullptr, (size_t)rope_rows * rope_dim * 4);
  if (append_grid(c, a.b, heads).groups * APPEND_THREADS > THREADS_MAX) return HCR_EINVAL;
  const Span so = span(q_out, (size_t)a.b.n_tokens * heads * c.head_dim * 2);
  const CacheSpans sc = cache_spans(*h);
  if (overlap_any(so, sc) || overlap_any(so, batch_spans(a.b))) return HCR_EALIAS;
  for (const Span& s : in)
    if (overlap(so, s) || overlap_any(s, sc)) return HCR_EALIAS;
  for (const Span& s : batch_spans(a.b).s)
    if (overlap_any(s, sc)) return HCR_EALIAS;
  a.q = *q;
  a.k = *k;
  a.v = *v;
  a.heads = heads;
  a.type = type;
  a.q_norm = q_norm;
  a.k_norm = k_norm;
  a.rope = rope;
  a.eps = eps;
  a.rope_dim = rope_dim;
  a.rope_style = rope_style;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.code = h->code;
  return launch_append(a, stream);
}

size_t hcr_attn_scratch_bytes(hcr_cache_t h, const hcr_batch* batch, int heads, int n_sel) {
  return attn_scratch(h, batch, heads, n_sel, WindowArgs{0, 0});
}

int hcr_attn(hcr_cache_t c, const hcr_batch* batch, int heads, double scale, const void* q, int out_type, void* out,
             void* scratch, size_t scratch_bytes, void* stream) {
  return attn(c, batch, heads, scale, q, nullptr, 0, WindowArgs{0, 0}, out_type, out, scratch, scratch_bytes, stream);
}

int hcr_attn_blocks(hcr_cache_t c, const hcr_batch* batch, int heads, double scale, const void* q, const int* sel,
                    int n_sel, int out_type, void* out, void* scratch, size_t scratch_bytes, void* stream) {
  if (n_sel < 1 || !sel) return HCR_EINVAL;
  return attn(c, batch, heads, scale, q, sel, n_sel, WindowArgs{0, 0}, out_type, out, scratch, scratch_bytes, stream);
}

int hcr_block_scores(hcr_cache_t h, const hcr_batch* batch, int heads, const void* q, float* scores, int scores_stride,
                     void* stream) {
  if (!h || !h->args.means) return HCR_EINVAL;
  const CacheArgs& c = h->args;
  ScoreArgs a{};
  a.c = c;
  const int rc = check_bounds(c, batch, heads, &a.b);
  if (rc < 0) return rc;
  const int pages = a.b.max_ctx > 0 ? (a.b.max_ctx - 1) >> c.shift : 0;  // that a token can score
  if (scores_stride < 0 || scores_stride < pages) return HCR_EINVAL;
  if (rc == 1 || pages == 0) return HCR_OK;
  if (!q || !scores) return HCR_EINVAL;
  if (const int e = check_arrays(a.b)) return e;
  if (!aligned(q, 16) || !aligned(scores, 16)) return HCR_EALIGN;
  if ((long long)a.b.n_seqs * c.kv_heads * (pages / 64 + 1) * 256 > THREADS_MAX) return HCR_EINVAL;
  const Span so = span(scores, (size_t)a.b.n_tokens * c.kv_heads * scores_stride * 4);
  if (overlap(so, span(q, (size_t)a.b.n_tokens * heads * c.head_dim * 2)) || overlap_any(so, cache_spans(*h)) ||
      overlap_any(so, batch_spans(a.b)))
    return HCR_EALIAS;
  a.q = static_cast<const uint16_t*>(q);
  a.heads = heads;
  a.group = heads / c.kv_heads;
  a.scores = scores;
  a.stride = scores_stride;
  return launch_block_scores(a, stream);
}

int hcr_block_topk(hcr_cache_t h, const hcr_batch* batch, const float* scores, int scores_stride, int n_sel,
                   int n_first, int n_last, int* sel, void* stream) {
  if (!h) return HCR_EINVAL;
  const CacheArgs& c = h->args;
  TopkArgs a{};
  const int rc = check_bounds(c, batch, c.kv_heads, &a.b);
  if (rc < 0) return rc;
  const int pages = a.b.max_ctx > 0 ? (a.b.max_ctx - 1) >> c.shift : 0;
  // n_sel: the kernel's lanes step through a list in 32 bits
  if (n_sel < 1 || n_sel > ROWS_MAX || n_first < 0 || n_last < 1 || n_first > n_sel || n_last > n_sel - n_first)
    return HCR_EINVAL;
  if (scores_stride < 0 || scores_stride < pages) return HCR_EINVAL;
  if (rc == 1) return HCR_OK;
  if (!sel || (!scores && pages)) return HCR_EINVAL;
  if (const int e = check_arrays(a.b)) return e;
  if (!aligned(scores, 16) || !aligned(sel, 4)) return HCR_EALIGN;
  const size_t rows = (size_t)a.b.n_tokens * c.kv_heads;
  if (rows * 1024 > (size_t)THREADS_MAX) return HCR_EINVAL;
  const Span so = span(sel, rows * n_sel * 4);
  if (overlap(so, span(scores, rows * scores_stride * 4)) || overlap_any(so, cache_spans(*h)) ||
      overlap_any(so, batch_spans(a.b)))
    return HCR_EALIAS;
  a.scores = scores;
  a.stride = scores_stride;
  a.kv_heads = c.kv_heads;
  a.shift = c.shift;
  a.n_sel = n_sel;
  a.n_first = n_first;
  a.n_last = n_last;
  a.sel = sel;
  return launch_block_topk(a, stream);
}

}  // extern "C"
