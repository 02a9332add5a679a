/*
 * hcr_paged.h -- C ABI of the paged key-value cache of the decode window, in
 * libhcr.so beside the hyper-connection read and the skinny matvec (hcr.h).
 *
 * What follows the attn_q projection in a verify window (Strata PR #2221, first
 * comment) and, at long contexts, the selection of blocks (Strata PR #2072, first
 * comment: block scores and a top-k over 420,000 cells).  With n the i-th of the
 * T_b new tokens of sequence b, its position is p = ctx_len[b] - T_b + i:
 *
 *   hcr_cache_append   q, k normalised per head, rotated, k and v into the pages
 *   hcr_attn           out[n] = softmax(scale q[n] . k[0..p]) v[0..p], per head
 *   hcr_block_scores   s[n,h,j] = max over the heads g of kv head h of q[n,g] . mean_j
 *   hcr_block_topk     which pages token n attends to, from the scores
 *   hcr_attn_blocks    hcr_attn over the listed pages alone
 *
 * Memory. Every pointer but the hcr_batch, hcr_rows and handles themselves is a
 * device pointer the caller owns.  Pages hold `page` positions of every kv head,
 * in the order in which the matrix cores take them (16 contiguous bytes are one
 * operand of a lane), D = head_dim:
 *   k_pages : BF16 [n_pages][kv_heads][D / 8][page][8]   8 dimensions together
 *   v_pages : BF16 [n_pages][kv_heads][page / 8][D][8]   8 positions together
 *   k_means : BF16 [n_pages][kv_heads][D]                mean key of a complete page
 * head_dim is 64, 128 or 256; page is 32, 64, 128 or 256.
 * Position p of sequence b lives in slot p % page of page
 * block_table[b * table_stride + p / page].  Pages may be shared by sequences
 * that read them; a page that hcr_cache_append writes belongs to one sequence.
 *
 * Bounds that the kernels hold themselves, since they read the batch on the
 * device: a page number outside 0..n_pages-1 is a page without positions (nothing
 * is written to it, attention skips it, its score is -inf); ctx_len is taken as
 * at most max_ctx, a sequence's new tokens as at most max_tokens and inside
 * 0..n_tokens-1.  A token at a negative position (a padded sequence of length 0)
 * appends nothing and its row of every output is zeros (scores: nothing; topk:
 * -1).  Rows behind the last sequence's (from q_start[n_seqs]) are left as they
 * were.  A row whose q or keys are not finite is not either; a value that is not
 * finite makes its own dimension of the rows that see it so.  No other row depends on
 * them, nor on what else lies in a page (behind the last position, NaN included), with
 * one exception: a key whose product with q is -inf weighs nothing.
 *
 * Every call is asynchronous on `stream`, makes no allocation, synchronisation or
 * memset and can be captured into a HIP graph; its lengths and pages are read when
 * the graph runs, within the bounds it was captured with.  Sums have a fixed
 * order: a call is bitwise reproducible.
 *
 * Errors as in hcr.h: HCR_OK or a negative code, every check before any HIP call.
 */
#ifndef HCR_PAGED_H
#define HCR_PAGED_H

#include "hcr.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { HCR_F32 = 0, HCR_BF16 = 1 };              /* element types of rows and outputs */
enum { HCR_ROPE_HALVES = 0, HCR_ROPE_PAIRS = 1 }; /* rotated pairs: (j, j + r/2) or (2j, 2j + 1) */

typedef struct hcr_cache* hcr_cache_t;

/* The sequences of one call (a host struct; its pointers are device memory, 4-byte
 * aligned int32). */
typedef struct hcr_batch {
  int n_seqs;             /* sequences */
  int n_tokens;           /* rows of q, k, v, out, scores and sel */
  int max_tokens;         /* no sequence has more new tokens */
  int max_ctx;            /* no sequence is longer; at most table_stride * page */
  int table_stride;       /* entries of a row of block_table */
  const int* q_start;     /* [n_seqs + 1] first row of each sequence, ascending */
  const int* ctx_len;     /* [n_seqs] positions of each sequence, its new tokens included */
  const int* block_table; /* [n_seqs][table_stride] page numbers */
} hcr_batch;

/* Rows of heads: element (n, h, d) at data[n * token_stride + h * head_stride + d],
 * strides in elements and multiples of 16 bytes. */
typedef struct hcr_rows {
  const void* data;
  long long token_stride;
  long long head_stride;
} hcr_rows;

/* Create a handle for one layer's cache.  Host-only; k_means may be NULL (then
 * hcr_cache_append keeps no means and hcr_block_scores refuses the cache).
 * Errors: HCR_EINVAL (NULL, a geometry that is not listed above), HCR_EALIGN
 * (16 bytes), HCR_EALIAS (overlapping buffers). */
int hcr_cache_create(void* k_pages, void* v_pages, void* k_means, int n_pages, int kv_heads, int head_dim, int page,
                     hcr_cache_t* out);
void hcr_cache_destroy(hcr_cache_t c);

/* Bytes of k_pages (v_pages has as many); 0 for a geometry that is not listed above. */
size_t hcr_cache_pages_bytes(int n_pages, int kv_heads, int head_dim, int page);

/* Append a window: per head x of q and k (each D values, all of one type)
 *   y = x * w / sqrt(mean(x^2) + eps)      (w NULL: y = x)
 * then the first rope_dim values rotated by the angles of the token's position,
 * (a, b) -> (a cos - b sin, b cos + a sin), in FP32, rounded once to BF16: q to
 * q_out [n_tokens][heads][D], k and v (v as it is) to the pages.  Where a new token
 * fills the last slot of its page, the page's mean key is written to k_means: the
 * FP32 mean of its BF16 keys, rounded to BF16.
 *   heads      a multiple of kv_heads, at most 64 times it
 *   type       HCR_F32 or HCR_BF16, of q, k and v
 *   q_norm, k_norm  float [D] or NULL; eps >= 0
 *   rope       float [rope_rows][rope_dim]: cos of rope_dim / 2 angles, then their
 *              sin; row p for position p, rope_rows >= max_ctx.  NULL with rope_dim 0
 *   rope_dim   0..D, a multiple of 16;  rope_style HCR_ROPE_HALVES or HCR_ROPE_PAIRS
 * Rows of q, k and v may lie side by side in one projection's output.  The window's
 * rows must not overlap the cache or q_out.
 * Errors: HCR_EINVAL, HCR_EALIGN, HCR_EALIAS, HCR_EHIP. */
int hcr_cache_append(hcr_cache_t c, const hcr_batch* batch, int heads, int type, const hcr_rows* q, const hcr_rows* k,
                     const hcr_rows* v, const float* q_norm, const float* k_norm, float eps, const float* rope,
                     int rope_rows, int rope_dim, int rope_style, void* q_out, void* stream);

/* Bytes of scratch that hcr_attn (n_sel 0) or hcr_attn_blocks (n_sel of the call)
 * needs for a batch of these bounds (only the ints of `batch` are read); 0 where the
 * call would be refused or needs none. */
size_t hcr_attn_scratch_bytes(hcr_cache_t c, const hcr_batch* batch, int heads, int n_sel);

/* Attention of a window over its sequences' pages: the window's own keys and values
 * are in the cache already (hcr_cache_append), token n sees positions 0..p.
 *   q    BF16 [n_tokens][heads][D]       out  float or BF16 (out_type) [n_tokens][heads][D]
 *   scratch  hcr_attn_scratch_bytes, 256-byte aligned; calls that share one, replays of
 *            graphs among them, must be ordered on one stream.  NULL where 0 bytes are needed
 * Products of BF16 values in FP32 on the matrix cores; probabilities in two BF16 parts
 * (2^-17), in three for a float `out`.  A row that sees no position is zeros.  |scale|
 * < 1e30.
 * Errors: HCR_EINVAL, HCR_EALIGN, HCR_ESCRATCH, HCR_EALIAS, HCR_EHIP. */
int hcr_attn(hcr_cache_t c, const hcr_batch* batch, int heads, double scale, const void* q, int out_type, void* out,
             void* scratch, size_t scratch_bytes, void* stream);

/* The same over listed pages: sel int32 [n_tokens][kv_heads][n_sel] holds page indices
 * of the token's sequence (position / page), in any order; entries outside the sequence
 * (-1) are skipped, positions behind p are not seen, an index listed twice counts
 * twice.  n_sel >= 1. */
int hcr_attn_blocks(hcr_cache_t c, const hcr_batch* batch, int heads, double scale, const void* q, const int* sel,
                    int n_sel, int out_type, void* out, void* scratch, size_t scratch_bytes, void* stream);

/* Scores of the complete pages before each token's own (j < p / page) from their mean
 * keys: scores[n][h][j], float [n_tokens][kv_heads][scores_stride], 16-byte aligned,
 * scores_stride >= (max_ctx - 1) / page; the other entries are left as they were.  A
 * score is NaN where one of its products is, -inf where the page is none.
 * Errors: HCR_EINVAL (a cache without means too), HCR_EALIGN, HCR_EALIAS, HCR_EHIP. */
int hcr_block_scores(hcr_cache_t c, const hcr_batch* batch, int heads, const void* q, float* scores, int scores_stride,
                     void* stream);

/* Selection: of the pages 0..p / page of each token and kv head, the first n_first, the
 * last n_last (the token's own among them) and, up to n_sel in all, those of the
 * highest scores between (level scores: the lowest index first; NaN ranks as -inf), as
 * ascending indices in sel [n_tokens][kv_heads][n_sel], -1 behind them.  n_first >= 0,
 * n_last >= 1, n_first + n_last <= n_sel <= 2^30.  scores as hcr_block_scores leaves
 * them.
 * Errors: HCR_EINVAL, HCR_EALIGN, HCR_EALIAS, HCR_EHIP. */
int hcr_block_topk(hcr_cache_t c, const hcr_batch* batch, const float* scores, int scores_stride, int n_sel,
                   int n_first, int n_last, int* sel, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HCR_PAGED_H */
