// Argument checks that the paged cache's entry points share: the handle, spans of memory, bounds of a batch.  Host only;
// every check runs before any HIP call.
#pragma once

#include <stdint.h>

#include "hcr_paged_layout.h"

struct hcr_cache {
  hcr::CacheArgs args;
  hcr::CodeArgs code;
};

namespace hcr {

struct Span {
  uintptr_t lo, hi;  // [lo, hi); lo == hi: absent
};
inline Span span(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return p ? Span{a, a + bytes} : Span{0, 0};
}
inline bool overlap(Span a, Span b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }
inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr long long ROWS_MAX = 1ll << 30;  // rows of heads of a call, positions, tiles: 32 bits hold them
constexpr long long THREADS_MAX = (1ll << 32) - 1;  // of a launch

inline size_t pages_elements(const CacheArgs& c) {
  return ((size_t)c.n_pages * c.kv_heads * c.head_dim) << c.shift;
}
inline size_t means_elements(const CacheArgs& c) { return (size_t)c.n_pages * c.kv_heads * c.head_dim; }

// The device arrays of a batch, which no output may overlap.
struct BatchSpans {
  Span s[3];
};
inline BatchSpans batch_spans(const BatchArgs& b) {
  return BatchSpans{{span(b.q_start, ((size_t)b.n_seqs + 1) * 4), span(b.ctx_len, (size_t)b.n_seqs * 4),
                     span(b.table, (size_t)b.n_seqs * b.table_stride * 4)}};
}
struct CacheSpans {
  Span s[5];
};
inline CacheSpans cache_spans(const CacheArgs& c, const CodeArgs& x) {
  const size_t pages = pages_elements(c) * (coded(x) ? 1 : 2), scales = pages_elements(c) / c.head_dim * 4;
  return CacheSpans{{span(c.k, pages), span(c.v, pages), span(c.means, means_elements(c) * 2), span(x.k_scales, scales),
                     span(x.v_scales, scales)}};
}
inline CacheSpans cache_spans(const hcr_cache& h) { return cache_spans(h.args, h.code); }
template <typename T>
bool overlap_any(Span o, const T& t) {
  for (const Span& s : t.s)
    if (overlap(o, s)) return true;
  return false;
}

// The ints of a batch against a cache and a number of heads; *b takes them.  1: nothing to do.
inline int check_bounds(const CacheArgs& c, const hcr_batch* in, int heads, BatchArgs* b) {
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
inline bool lists_fit(const CacheArgs& c, const BatchArgs& b, int n_sel) {
  return n_sel >= 0 && (long long)n_sel << c.shift <= ROWS_MAX &&
         ((long long)n_sel << (c.shift - TILE_SHIFT)) * b.n_tokens <= ROWS_MAX;
}
inline int check_arrays(const BatchArgs& b) {
  if (!b.q_start || !b.ctx_len || (!b.table && b.table_stride)) return HCR_EINVAL;
  if (!aligned(b.q_start, 4) || !aligned(b.ctx_len, 4) || !aligned(b.table, 4)) return HCR_EALIGN;
  return HCR_OK;
}

// Rows of heads of one input: their span, or an error.
inline int check_rows(const hcr_rows* r, int type, int n_tokens, int heads, int head_dim, Span* s) {
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

// hcr_attn and its kinds, after their own arguments' checks.
int attn(hcr_cache_t h, const hcr_batch* batch, int heads, double scale, const void* q, const int* sel, int n_sel,
         const WindowArgs& w, int out_type, void* out, void* scratch, size_t scratch_bytes, void* stream);
size_t attn_scratch(hcr_cache_t h, const hcr_batch* batch, int heads, int n_sel, const WindowArgs& w);
// Pages and means of a new cache; 0 or an error.
int check_cache(const CacheArgs& c, const CodeArgs& x);
int new_cache(const CacheArgs& c, const CodeArgs& x, hcr_cache_t* out);

}  // namespace hcr
