// C ABI of the paged cache: argument checks, the handle and the plan of an attention call.  Every check runs on
// the host before any HIP call.

#include <float.h>
#include <math.h>
#include <stdint.h>
#include <stdlib.h>

#include "hcr_paged_layout.h"

struct hcr_cache {
  hcr::CacheArgs args;
};

namespace hcr {

namespace {

struct Span {
  uintptr_t lo, hi;  // [lo, hi); lo == hi: absent
};
Span span(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return p ? Span{a, a + bytes} : Span{0, 0};
}
bool overlap(Span a, Span b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr long long ROWS_MAX = 1ll << 30;  // rows of heads of a call, positions, tiles: 32 bits hold them
constexpr long long THREADS_MAX = (1ll << 32) - 1;  // of a launch

size_t pages_elements(const CacheArgs& c) {
  return ((size_t)c.n_pages * c.kv_heads * c.head_dim) << c.shift;
}
size_t means_elements(const CacheArgs& c) { return (size_t)c.n_pages * c.kv_heads * c.head_dim; }

// The device arrays of a batch, which no output may overlap.
struct BatchSpans {
  Span s[3];
};
BatchSpans batch_spans(const BatchArgs& b) {
  return BatchSpans{{span(b.q_start, ((size_t)b.n_seqs + 1) * 4), span(b.ctx_len, (size_t)b.n_seqs * 4),
                     span(b.table, (size_t)b.n_seqs * b.table_stride * 4)}};
}
struct CacheSpans {
  Span s[3];
};
CacheSpans cache_spans(const CacheArgs& c) {
  return CacheSpans{{span(c.k, pages_elements(c) * 2), span(c.v, pages_elements(c) * 2),
                     span(c.means, means_elements(c) * 2)}};
}
template <typename T>
bool overlap_any(Span o, const T& t) {
  for (const Span& s : t.s)
    if (overlap(o, s)) return true;
  return false;
}

// The ints of a batch against a cache and a number of heads; *b takes them.  1: nothing to do.
int check_bounds(const CacheArgs& c, const hcr_batch* in, int heads, BatchArgs* b) {
  if (!in) return HCR_EINVAL;
  if (heads < 1 || heads % c.kv_heads || heads / c.kv_heads > GROUP_MAX) return HCR_EINVAL;
  if (in->n_seqs < 0 || in->n_tokens < 0 || in->max_tokens < 0 || in->max_ctx < 0 || in->table_stride < 0)
    return HCR_EINVAL;
  if ((long long)in->table_stride << c.shift < in->max_ctx || in->max_ctx > 1 << 30) return HCR_EINVAL;
  *b = BatchArgs{in->q_start, in->ctx_len,  in->block_table, in->table_stride,
                 in->n_seqs,  in->n_tokens, in->max_tokens,  in->max_ctx};
  if (b->max_tokens > b->n_tokens) b->max_tokens = b->n_tokens;
  if (b->n_seqs == 0 || b->max_tokens == 0) return 1;
  // rows and work-groups stay inside 32 bits
  if ((long long)b->n_tokens * heads > ROWS_MAX || (long long)b->n_seqs * b->max_tokens > ROWS_MAX / heads ||
      (long long)b->n_seqs * ceil_div(b->max_ctx, TILE) > ROWS_MAX)
    return HCR_EINVAL;
  return HCR_OK;
}
// Page lists whose positions and tiles (all tokens' together) 32 bits hold.
bool lists_fit(const CacheArgs& c, const BatchArgs& b, int n_sel) {
  return n_sel >= 0 && (long long)n_sel << c.shift <= ROWS_MAX &&
         ((long long)n_sel << (c.shift - TILE_SHIFT)) * b.n_tokens <= ROWS_MAX;
}
int check_arrays(const BatchArgs& b) {
  if (!b.q_start || !b.ctx_len || (!b.table && b.table_stride)) return HCR_EINVAL;
  if (!aligned(b.q_start, 4) || !aligned(b.ctx_len, 4) || !aligned(b.table, 4)) return HCR_EALIGN;
  return HCR_OK;
}

// Rows of heads of one input: their span, or an error.
int check_rows(const hcr_rows* r, int type, int n_tokens, int heads, int head_dim, Span* s) {
  if (!r || !r->data) return HCR_EINVAL;
  const long long unit = type == HCR_F32 ? 4 : 8, size = type == HCR_F32 ? 4 : 2;
  const long long most = 1ll << 48;  // elements on the way to the last row
  if (r->token_stride < 0 || r->head_stride < 0 || r->token_stride > most / n_tokens || r->head_stride > most / heads)
    return HCR_EINVAL;
  if (!aligned(r->data, 16) || r->token_stride % unit || r->head_stride % unit) return HCR_EALIGN;
  const long long last = (n_tokens - 1) * r->token_stride + (heads - 1) * r->head_stride + head_dim;
  *s = span(r->data, (size_t)last * size);
  return HCR_OK;
}

long long attn_grid(const CacheArgs& c, const AttnPlan& p) {
  return ((long long)p.items * c.kv_heads + XCDS - 1) / XCDS * XCDS * p.row_blocks;
}

size_t scratch_of(const CacheArgs& c, const AttnPlan& p) {
  if (!attn_joins(p)) return 0;
  return align256((size_t)c.kv_heads * p.row_blocks * p.items * 2 * attn_rows(p) * (c.head_dim + 2) * 4);
}

int attn(hcr_cache_t h, const hcr_batch* batch, int heads, double scale, const void* q, const int* sel, int n_sel,
         int out_type, void* out, void* scratch, size_t scratch_bytes, void* stream) {
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
  a.plan = attn_plan(c, a.b, heads, n_sel);
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
  for (const Span& w : written)
    if (overlap(w, sq) || overlap(w, sl) || overlap_any(w, cache_spans(c)) || overlap_any(w, batch_spans(a.b)))
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
  if (scale != 0) {
    const float least = copysignf(FLT_TRUE_MIN, (float)scale);
    if (a.scale_hi == 0.f) a.scale_hi = least;
    if (a.scale_lo == 0.f) a.scale_lo = least;
  }
  a.out = out;
  a.part = static_cast<float*>(scratch);
  return launch_attn(a, stream);
}

}  // namespace

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
AttnPlan attn_plan(const CacheArgs& c, const BatchArgs& b, int heads, int n_sel) {
  constexpr int CUS = 256;
  AttnPlan p{};
  const int group = heads / c.kv_heads;
  const int rows = n_sel ? group : b.max_tokens * group;
  const bool wide = c.head_dim == 256;
  const int tiles = n_sel ? n_sel << (c.shift - TILE_SHIFT) : ceil_div(b.max_ctx, TILE);
  const long long sets = n_sel ? b.n_tokens : b.n_seqs;
  const bool lengthy = rows > 48 && rows <= 64 && tiles >= 256 && sets * tiles >= 512;
  p.q_tiles = rows > 16 && (c.head_dim == 128 || (wide && (rows <= 32 || lengthy))) ? 2 : 1;
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
  p.whole = full < CUS              ? tiles <= (wide ? (rows > 16 ? 6 : 12) : 3 * most_groups)
            : n_sel                 ? 1  // lists are alike
            : alone                 ? tiles <= 32
            : full < 2 * CUS        ? tiles <= 64
                                    : tiles <= 128;
  const bool few = p.whole ? full >= 2 * CUS && tiles <= 16 : !n_sel && tiles <= 64;
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
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(k_means, 16)) return HCR_EALIGN;
  const CacheArgs c{static_cast<uint16_t*>(k_pages), static_cast<uint16_t*>(v_pages), static_cast<uint16_t*>(k_means),
                    n_pages, kv_heads, head_dim, log2_of(page)};
  const CacheSpans s = cache_spans(c);
  if (overlap(s.s[0], s.s[1]) || overlap(s.s[0], s.s[2]) || overlap(s.s[1], s.s[2])) return HCR_EALIAS;
  hcr_cache* h = static_cast<hcr_cache*>(malloc(sizeof(hcr_cache)));
  if (!h) return HCR_EINVAL;
  h->args = c;
  *out = h;
  return HCR_OK;
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
  const CacheSpans sc = cache_spans(c);
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
  return launch_append(a, stream);
}

size_t hcr_attn_scratch_bytes(hcr_cache_t h, const hcr_batch* batch, int heads, int n_sel) {
  BatchArgs b;
  if (!h || check_bounds(h->args, batch, heads, &b) != HCR_OK || !lists_fit(h->args, b, n_sel)) return 0;
  return scratch_of(h->args, attn_plan(h->args, b, heads, n_sel));
}

int hcr_attn(hcr_cache_t c, const hcr_batch* batch, int heads, double scale, const void* q, int out_type, void* out,
             void* scratch, size_t scratch_bytes, void* stream) {
  return attn(c, batch, heads, scale, q, nullptr, 0, out_type, out, scratch, scratch_bytes, stream);
}

int hcr_attn_blocks(hcr_cache_t c, const hcr_batch* batch, int heads, double scale, const void* q, const int* sel,
                    int n_sel, int out_type, void* out, void* scratch, size_t scratch_bytes, void* stream) {
  if (n_sel < 1 || !sel) return HCR_EINVAL;
  return attn(c, batch, heads, scale, q, sel, n_sel, out_type, out, scratch, scratch_bytes, stream);
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
  if (overlap(so, span(q, (size_t)a.b.n_tokens * heads * c.head_dim * 2)) || overlap_any(so, cache_spans(c)) ||
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
  if (overlap(so, span(scores, rows * scores_stride * 4)) || overlap_any(so, cache_spans(c)) ||
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
