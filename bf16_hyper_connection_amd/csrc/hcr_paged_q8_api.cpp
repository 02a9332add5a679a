// C ABI of the paged cache's other forms (include/hcr_paged_q8.h): pages of codes, reading a cache back, attention over
// a sliding window.  Every check runs on the host before any HIP call.

#include "hcr_paged_check.h"

using namespace hcr;

extern "C" {

size_t hcr_cache_pages_bytes_q8(int n_pages, int kv_heads, int head_dim, int page) {
  if (n_pages < 1 || kv_heads < 1 || !head_dim_ok(head_dim) || !code_page_ok(page)) return 0;
  return (size_t)n_pages * kv_heads * head_dim * page;
}

int hcr_cache_create_q8(void* k_pages, void* v_pages, float* k_scales, float* v_scales, void* k_means, int code,
                        int n_pages, int kv_heads, int head_dim, int page, hcr_cache_t* out) {
  if (!out) return HCR_EINVAL;
  *out = nullptr;
  if (!k_pages || !v_pages || !k_scales || !v_scales || n_pages < 1 || kv_heads < 1 || kv_heads > 4096 ||
      !head_dim_ok(head_dim) || !code_page_ok(page) || (code != HCR_INT8 && code != HCR_E4M3))
    return HCR_EINVAL;
  const CacheArgs c{static_cast<uint16_t*>(k_pages), static_cast<uint16_t*>(v_pages), static_cast<uint16_t*>(k_means),
                    n_pages, kv_heads, head_dim, log2_of(page)};
  const CodeArgs x{k_scales, v_scales, code};
  if (const int e = check_cache(c, x)) return e;
  return new_cache(c, x, out);
}

int hcr_cache_read(hcr_cache_t h, const hcr_batch* batch, int out_type, void* k_out, void* v_out, void* stream) {
  if (!h) return HCR_EINVAL;
  const CacheArgs& c = h->args;
  ReadArgs a{};
  a.c = c;
  a.code = h->code;
  const int rc = check_bounds(c, batch, c.kv_heads, &a.b);
  if (rc < 0) return rc;
  if (out_type != HCR_F32 && out_type != HCR_BF16) return HCR_EINVAL;
  if (rc == 1) return HCR_OK;
  if (!k_out && !v_out) return HCR_EINVAL;
  if (const int e = check_arrays(a.b)) return e;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return HCR_EALIGN;
  if ((long long)a.b.n_seqs * read_parts(a.b) * c.kv_heads * READ_THREADS > THREADS_MAX) return HCR_EINVAL;
  const size_t bytes = (size_t)a.b.n_tokens * c.kv_heads * c.head_dim * (out_type == HCR_F32 ? 4 : 2);
  const Span sk = span(k_out, bytes), sv = span(v_out, bytes);
  if (overlap(sk, sv)) return HCR_EALIAS;
  const Span written[] = {sk, sv};
  for (const Span& s : written)
    if (overlap_any(s, cache_spans(*h)) || overlap_any(s, batch_spans(a.b))) return HCR_EALIAS;
  a.out_type = out_type;
  a.k_out = k_out;
  a.v_out = v_out;
  return launch_read(a, stream);
}

size_t hcr_attn_window_scratch_bytes(hcr_cache_t h, const hcr_batch* batch, int heads, int window, int n_first) {
  if (window < 1 || n_first < 0) return 0;
  return attn_scratch(h, batch, heads, 0, WindowArgs{window, n_first});
}

int hcr_attn_window(hcr_cache_t c, const hcr_batch* batch, int heads, double scale, const void* q, int window,
                    int n_first, int out_type, void* out, void* scratch, size_t scratch_bytes, void* stream) {
  if (window < 1 || n_first < 0) return HCR_EINVAL;
  return attn(c, batch, heads, scale, q, nullptr, 0, WindowArgs{window, n_first}, out_type, out, scratch, scratch_bytes,
              stream);
}

}  // extern "C"
