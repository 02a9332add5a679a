// Selection of pages for a decode window, gfx950 (MI355X): scores of every complete page by its mean key, and the
// pages of the highest scores.

#include <float.h>
#include <hip/hip_runtime.h>

#include "hcr_device.h"
#include "hcr_paged_layout.h"

namespace hcr {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;

// ---- scores: s[n][h][j] = max over the group's heads of q . mean_j, FP32 sums of BF16 products on the matrix
// cores.  A wave takes 16 pages of one kv head as the rows of A (16 contiguous bytes of a mean per lane) and
// the window's query rows as columns of B, each token's heads padded to 2^k <= 16 columns (or to whole tiles of
// 16) by repeating its last head, which leaves the maximum as it is: the maximum over a token's heads is then a
// butterfly inside a row of 16 lanes.  Bound by the means' bytes, read once per column tile from L2 after the
// first.
constexpr int SCORE_WAVES = 4;

__device__ __forceinline__ float max_dpp(float v, int width) {  // over aligned runs of `width` lanes of a row
  if (width >= 2) v = fmaxf(v, dpp<0xB1>(v));
  if (width >= 4) v = fmaxf(v, dpp<0x4E>(v));
  if (width >= 8) v = fmaxf(v, dpp<0x141>(v));
  if (width >= 16) v = fmaxf(v, dpp<0x140>(v));
  return v;
}

template <int D>
__global__ __launch_bounds__(64 * SCORE_WAVES) void block_scores(ScoreArgs a, int width, int tiles_per_token,
                                                                 int chunks) {
  constexpr int KS = D / 32;
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = threadIdx.x >> 6;
  int u = blockIdx.x;
  const int h = u % a.c.kv_heads;
  u /= a.c.kv_heads;
  const int b = u % a.b.n_seqs;
  const int j0 = (u / a.b.n_seqs * SCORE_WAVES + wave) * 16;
  const Seq seq = seq_of(a.b, a.b.q_start[b], a.b.q_start[b + 1], a.b.ctx_len[b]);
  if (seq.tokens == 0) return;
  const int before = max(seq.first + seq.tokens - 1, 0) >> a.c.shift;  // pages that the last token scores
  if (j0 >= before) return;

  const int number = page_or_none(a.b.table[(size_t)b * a.b.table_stride + min(j0 + li, before - 1)], a.c.n_pages);
  const uint16_t* mp = a.c.means + ((size_t)max(number, 0) * a.c.kv_heads + h) * D + 8 * lg;
  uint4 mf[KS];
#pragma unroll
  for (int k = 0; k < KS; ++k) mf[k] = *reinterpret_cast<const uint4*>(mp + 32 * k);
  bool none[4];  // of the lane's result rows, the pages that are none
#pragma unroll
  for (int i = 0; i < 4; ++i) none[i] = __shfl(number, 4 * lg + i) < 0;

  const int tokens_per_tile = 16 / width;  // width 16: one token, in tiles_per_token tiles
  for (int t0 = 0; t0 < seq.tokens; t0 += tokens_per_tile) {
    const int t = min(t0 + li / width, seq.tokens - 1);
    const size_t n = seq.row + t;
    f32x4 best = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    for (int tt = 0; tt < tiles_per_token; ++tt) {
      const int g = min(16 * tt + li % width, a.group - 1);
      const uint16_t* qp = a.q + (n * a.heads + h * a.group + g) * D + 8 * lg;
      f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, mf[k]),
                                                    *reinterpret_cast<const bf16x8*>(qp + 32 * k), c, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) best[i] = fmaxf(best[i], c[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) best[i] = max_dpp(best[i], width);
    const int last = max(seq.first + t, 0) >> a.c.shift;  // this token scores the pages before it
    if (li % width == 0 && t0 + li / width < seq.tokens) {
      float* out = a.scores + (n * a.c.kv_heads + h) * a.stride;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + 4 * lg + i;
        if (j < last) out[j] = none[i] ? -INFINITY : best[i];
      }
    }
  }
}

template <int D>
void run_scores(const ScoreArgs& a, hipStream_t st) {
  int width = 1;
  while (width < a.group && width < 16) width *= 2;
  const int chunks = ceil_div((a.b.max_ctx - 1) >> a.c.shift, 16 * SCORE_WAVES);
  hipLaunchKernelGGL((block_scores<D>), dim3(chunks * a.b.n_seqs * a.c.kv_heads), dim3(64 * SCORE_WAVES), 0, st, a,
                     width, ceil_div(a.group, 16), chunks);
}

int launch_block_scores(const ScoreArgs& a, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (a.c.head_dim == 64)
    run_scores<64>(a, st);
  else if (a.c.head_dim == 128)
    run_scores<128>(a, st);
  else
    run_scores<256>(a, st);
  return hipGetLastError() == hipSuccess ? HCR_OK : HCR_EHIP;
}

// ---- selection: one work-group per token and kv head.  The scores between the first and the last pages become
// keys whose order as whole numbers is theirs; three histograms (11, 11 and 10 bits, from the top) narrow the
// smallest selected key down to its value; the pages above it, and as many level with it as are left to take,
// lowest index first, go out in ascending order behind one prefix sum.
constexpr int TOPK_THREADS = 1024;
constexpr int TOPK_BINS = 2048;

// -0 as +0, NaN as -inf; larger scores have larger keys
__device__ __forceinline__ uint32_t order_key(float s) {
  if (!(s == s)) s = -INFINITY;
  const uint32_t u = __float_as_uint(s + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum over the work-group's threads, and the total.  tmp: 16 values.
__device__ __forceinline__ uint32_t prefix(uint32_t v, uint32_t* tmp, uint32_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const uint32_t y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // tmp may still be read from before
  if (lane == 63) tmp[wave] = x;
  __syncthreads();
  uint32_t base = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < TOPK_THREADS / 64; ++w) {
    if (w < wave) base += tmp[w];
    total += tmp[w];
  }
  return base + x - v;
}

__global__ __launch_bounds__(TOPK_THREADS) void block_topk(TopkArgs a) {
  __shared__ uint32_t bins[TOPK_BINS];
  __shared__ uint32_t tmp[TOPK_THREADS / 64];
  __shared__ uint32_t found[2];  // the digit, and how many keys lie above it
  const int tid = threadIdx.x;
  const int h = blockIdx.x % a.kv_heads;
  const int bt = blockIdx.x / a.kv_heads;
  const int t = bt % a.b.max_tokens, b = bt / a.b.max_tokens;
  const Seq seq = seq_of(a.b, a.b.q_start[b], a.b.q_start[b + 1], a.b.ctx_len[b]);
  if (t >= seq.tokens) return;
  const size_t row = (size_t)(seq.row + t) * a.kv_heads + h;
  const int pos = seq.first + t;
  const int count = pos < 0 ? 0 : (pos >> a.shift) + 1;  // pages up to the token's own
  int* sel = a.sel + row * a.n_sel;
  if (count <= a.n_sel) {
    for (int i = tid; i < a.n_sel; i += TOPK_THREADS) sel[i] = i < count ? i : -1;
    return;
  }
  const int m = count - a.n_first - a.n_last;  // between the first and the last, more than are wanted
  const uint32_t want = a.n_sel - a.n_first - a.n_last;
  const float* s = a.scores + row * a.stride + a.n_first;
  for (int i = tid; i < a.n_first; i += TOPK_THREADS) sel[i] = i;
  for (int i = tid; i < a.n_last; i += TOPK_THREADS) sel[a.n_sel - a.n_last + i] = count - a.n_last + i;
  if (want == 0) return;

  uint32_t key = 0, mask = 0, left = want;  // keys with these top bits hold the smallest selected one
#pragma unroll
  for (int round = 0; round < 3; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
    const uint32_t digit = round == 2 ? 1023 : 2047;
    for (int i = tid; i < TOPK_BINS; i += TOPK_THREADS) bins[i] = 0;
    __syncthreads();
    for (int i = tid; i < m; i += TOPK_THREADS) {
      const uint32_t k = order_key(s[i]);
      if ((k & mask) == key) atomicAdd(&bins[(k >> shift) & digit], 1u);
    }
    __syncthreads();
    // thread t counts the bins from the top: 2047 - 2 t and the one below
    const int top = TOPK_BINS - 1 - 2 * tid;
    const uint32_t c0 = bins[top], c1 = bins[top - 1];
    uint32_t total;
    const uint32_t above = prefix(c0 + c1, tmp, total);
    if (above < left && left <= above + c0) {
      found[0] = top;
      found[1] = above;
    } else if (above + c0 < left && left <= above + c0 + c1) {
      found[0] = top - 1;
      found[1] = above + c0;
    }
    __syncthreads();
    key |= found[0] << shift;
    mask |= digit << shift;
    left -= found[1];
    __syncthreads();
  }

  // thread t takes consecutive pages, so that ranks follow the index
  const int each = ceil_div(m, TOPK_THREADS);
  const int i0 = min(tid * each, m), i1 = min(i0 + each, m);
  uint32_t level = 0, over = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = order_key(s[i]);
    over += k > key;
    level += k == key;
  }
  uint32_t total;
  uint32_t levels = prefix(level, tmp, total);  // level keys before this thread's: the first `left` are taken
  const uint32_t mine = levels >= left ? 0 : min(level, left - levels);
  uint32_t at = a.n_first + prefix(over + mine, tmp, total);
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = order_key(s[i]);
    bool take = k > key;
    if (k == key) take = levels++ < left;
    if (take) sel[at++] = a.n_first + i;
  }
}

int launch_block_topk(const TopkArgs& a, void* stream) {
  (void)hipGetLastError();
  hipLaunchKernelGGL(block_topk, dim3(a.b.n_seqs * a.b.max_tokens * a.kv_heads), dim3(TOPK_THREADS), 0,
                     reinterpret_cast<hipStream_t>(stream), a);
  return hipGetLastError() == hipSuccess ? HCR_OK : HCR_EHIP;
}

}  // namespace hcr
