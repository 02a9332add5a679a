/*
 * hcr_paged_q8.h -- C ABI of the paged cache's other forms, beside hcr_paged.h: pages of
 * 8-bit codes, reading a cache back, and attention over a sliding window.
 *
 * A cache of codes (the engine's int8 key-value cache, Strata PR #2072, setup) has half
 * the bytes of a BF16 one.  hcr_cache_append writes it: with y a head's key after norm
 * and rotation, or its value, in FP32, and top the largest code,
 *
 *   scale = max |y| / top        FP32, one for each position and kv head
 *   code  = y / scale, to the nearest code, ties to the even one;  it stands for code * scale
 *
 * (both quotients are FP32's, correctly rounded; codes stop at top), so that what a position
 * holds depends on that position alone, however windows were cut and whatever was written
 * over.  A head that holds a value that is not finite has the scale NaN and stands for NaN as
 * a whole; zeros, and heads whose scale rounds to 0, have the scale 0.  hcr_attn and
 * hcr_attn_blocks attend over what the codes stand for, in FP32 (a probability takes its value's
 * scale along into its BF16 parts: of scales under 2^-100 low bits are lost); hcr_block_scores and
 * hcr_block_topk take such a cache as any other (mean keys are of what the codes stand for).
 * Pages that were filled otherwise may hold any codes and scales: a key that is no number (the
 * E4M3 codes 0x7F and 0xFF, a scale of NaN) makes every output NaN of the rows that see it, a
 * value's code that is none its own dimension of them, a value's scale that is not finite all
 * of theirs no numbers; rows that do not see it take nothing from it.
 *
 * Pages hold 64, 128 or 256 positions:
 *   k_pages  : codes [n_pages][kv_heads][D / 16][page][16]   16 dimensions together
 *   v_pages  : codes [n_pages][kv_heads][page / 16][D][16]   16 positions together
 *   k_scales, v_scales : float [n_pages][kv_heads][page]
 *   k_means  : BF16 [n_pages][kv_heads][D]
 *
 * Everything that hcr_paged.h says of batches, bounds, rows, padded tokens, streams,
 * graphs and errors holds here too.
 */
#ifndef HCR_PAGED_Q8_H
#define HCR_PAGED_Q8_H

#include "hcr_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  HCR_INT8 = 2, /* whole numbers -127..127, top 127 (-128 in a page stands for -128) */
  HCR_E4M3 = 3  /* 8-bit floats of 4 exponent and 3 mantissa bits, no infinities, top 448 */
};

/* Create a handle for one layer's cache of codes (HCR_INT8 or HCR_E4M3); hcr_cache_destroy
 * ends it.  Host-only; k_means may be NULL.
 * Errors: HCR_EINVAL (NULL, a geometry that is not listed above), HCR_EALIGN (16 bytes),
 * HCR_EALIAS (overlapping buffers). */
int hcr_cache_create_q8(void* k_pages, void* v_pages, float* k_scales, float* v_scales, void* k_means, int code,
                        int n_pages, int kv_heads, int head_dim, int page, hcr_cache_t* out);

/* Bytes of k_pages of a cache of codes (v_pages has as many); 0 for a geometry that is not listed above.
 * Its k_scales take 4 / head_dim of that. */
size_t hcr_cache_pages_bytes_q8(int n_pages, int kv_heads, int head_dim, int page);

/* Read back keys and values of either kind of cache: row n, the i-th of the T_b tokens of
 * sequence b, is position p = ctx_len[b] - T_b + i (T_b = ctx_len[b] reads a sequence whole).
 *   k_out, v_out  float or BF16 (out_type) [n_tokens][kv_heads][D], 16-byte aligned; one
 *                 may be NULL.  A code times its scale in FP32, rounded once.
 * Tokens at negative positions and positions whose page is none: zeros.
 * Errors: HCR_EINVAL, HCR_EALIGN, HCR_EALIAS, HCR_EHIP. */
int hcr_cache_read(hcr_cache_t c, const hcr_batch* batch, int out_type, void* k_out, void* v_out, void* stream);

/* Bytes of scratch that hcr_attn_window needs, as hcr_attn_scratch_bytes. */
size_t hcr_attn_window_scratch_bytes(hcr_cache_t c, const hcr_batch* batch, int heads, int window, int n_first);

/* hcr_attn over a sliding window, for either kind of cache: token n at position p sees the
 * positions p - window + 1 .. p and, besides, 0 .. n_first - 1 (up to p; a position in both
 * counts once).  window >= 1, n_first >= 0.  Table entries of pages that no token sees are
 * not read as pages: they may be -1.
 * Errors: as hcr_attn. */
int hcr_attn_window(hcr_cache_t c, const hcr_batch* batch, int heads, double scale, const void* q, int window,
                    int n_first, int out_type, void* out, void* scratch, size_t scratch_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HCR_PAGED_Q8_H */
