// Selection of pages for a decode window, gfx950 (MI355X): scores of every complete page by its mean key, and the
// pages of the highest scores.

#include <float.h>
#include <hip/hip_runtime.h>

#include "hcr_paged_device.h"

namespace hcr {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;

// ---- scores: s[n][h][j] = max over the group's heads of q . mean_j, FP32 sums of BF16 products on the matrix
// cores.  A wave takes 16 pages of one kv head as the rows of A (16 contiguous bytes of a mean per lane) and
// the window's query rows as columns of B, each token's heads padded to 2^k <= 16 columns (or to whole tiles of
// 16) by repeating its last head, which leaves the maximum as it is: the maximum over a token's heads is then a
// butterfly inside a row of 16 lanes.  Bound by the means' bytes, read once per column tile from L2 after the
// first, and by two waits (the page's number, its mean) and the launch, as long as the bytes: 27.8 MB of 6,562 pages,
// 8 heads of 256, 4 tokens in 10.5 us.
constexpr int SCORE_WAVES = 4;

// The larger one, NaN where one is NaN (one instruction, v_maximum3_f32; fmaxf would drop a head that is no number).
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float max_dpp(float v, int width) {  // over aligned runs of `width` lanes of a row
  if (width >= 2) v = larger(v, dpp<0xB1>(v));
  if (width >= 4) v = larger(v, dpp<0x4E>(v));
  if (width >= 8) v = larger(v, dpp<0x141>(v));
  if (width >= 16) v = larger(v, dpp<0x140>(v));
  return v;
}

// TILES 16-page tiles a wave; with one, `each` of the window's column tiles a work-group
template <int D, int TILES>
__global__ __launch_bounds__(64 * SCORE_WAVES) void block_scores(ScoreArgs a, int width, int tiles_per_token,
                                                                 int each) {
  constexpr int KS = D / 32;
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int u = blockIdx.x;
  const int h = u % a.c.kv_heads;
  u /= a.c.kv_heads;
  const int b = u % a.b.n_seqs;
  const int j0 = (u / a.b.n_seqs * SCORE_WAVES + wave) * 16 * TILES;
  // the pages' numbers and the sequence come together; entries behind the sequence's are not used
  int number[TILES];
#pragma unroll
  for (int p = 0; p < TILES; ++p)
    number[p] = a.b.table[(size_t)b * a.b.table_stride + min(j0 + 16 * p + li, a.b.table_stride - 1)];
  const Seq seq = wave_seq(a.b, b);
  if (seq.tokens == 0) return;
  const int before = max(seq.first + seq.tokens - 1, 0) >> a.c.shift;  // pages that the last token scores
  if (j0 >= before) return;

  uint4 mf[TILES][KS];
  bool none[TILES][4];  // of the lane's result rows, the pages that are none
#pragma unroll
  for (int p = 0; p < TILES; ++p) {
    number[p] = page_or_none(number[p], a.c.n_pages);
    const uint16_t* mp = a.c.means + ((size_t)max(number[p], 0) * a.c.kv_heads + h) * D + 8 * lg;
#pragma unroll
    for (int k = 0; k < KS; ++k) mf[p][k] = *reinterpret_cast<const uint4*>(mp + 32 * k);
#pragma unroll
    for (int i = 0; i < 4; ++i) none[p][i] = __shfl(number[p], 4 * lg + i) < 0;
  }

  // column tiles of the window: tokens_per_tile tokens in one, or one token in tiles_per_token; the next one's
  // rows are loaded while this one is multiplied
  const int tokens_per_tile = 16 / width;
  const int first = TILES == 1 ? blockIdx.y * each : 0;
  int tiles = ceil_div(seq.tokens, tokens_per_tile) * tiles_per_token;
  if (TILES == 1) tiles = min(first + each, tiles);
  if (first >= tiles) return;
  uint4 qf[KS];
  auto load = [&](int tile) {
    const int t = min(tile / tiles_per_token * tokens_per_tile + li / width, seq.tokens - 1);
    const int g = min(16 * (tile % tiles_per_token) + li % width, a.group - 1);
    const uint16_t* qp = a.q + ((size_t)(seq.row + t) * a.heads + h * a.group + g) * D + 8 * lg;
#pragma unroll
    for (int k = 0; k < KS; ++k) qf[k] = *reinterpret_cast<const uint4*>(qp + 32 * k);
  };
  load(first);
  const f32x4 lowest = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  f32x4 best[TILES];
#pragma unroll
  for (int p = 0; p < TILES; ++p) best[p] = lowest;
  for (int tile = first; tile < tiles; ++tile) {
    f32x4 c[TILES] = {};
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int p = 0; p < TILES; ++p)
        c[p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, mf[p][k]),
                                                       __builtin_bit_cast(bf16x8, qf[k]), c[p], 0, 0, 0);
    if (tile + 1 < tiles) load(tile + 1);
#pragma unroll
    for (int p = 0; p < TILES; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) best[p][i] = larger(best[p][i], c[p][i]);
    if ((tile + 1) % tiles_per_token) continue;
    const int t = tile / tiles_per_token * tokens_per_tile + li / width;
    const int last = max(seq.first + t, 0) >> a.c.shift;  // this token scores the pages before it
    float* out = a.scores + ((size_t)(seq.row + min(t, seq.tokens - 1)) * a.c.kv_heads + h) * a.stride;
#pragma unroll
    for (int p = 0; p < TILES; ++p) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s = max_dpp(best[p][i], width);
        const int j = j0 + 16 * p + 4 * lg + i;
        if (li % width == 0 && t < seq.tokens && j < last) out[j] = none[p][i] ? -INFINITY : s;
      }
      best[p] = lowest;
    }
  }
}

template <int D, int TILES>
void run_scores(const ScoreArgs& a, int pages, hipStream_t st) {
  int width = 1;
  while (width < a.group && width < 16) width *= 2;
  const int grid = ceil_div(pages, 16 * TILES * SCORE_WAVES) * a.b.n_seqs * a.c.kv_heads;
  // a wide window's column tiles side by side while they fit the chip at two work-groups a CU (each reads the means
  // again, from L2).  Measured on MI355X: 16 tokens of 12 heads, 16 sequences of 127 pages, 4 kv heads
  // 7.6 us against 15.2, 4 tokens of 64 heads, 2 of 281 5.0 against 10.8
  const int tiles = ceil_div(a.b.max_tokens, 16 / width), room = TILES == 1 ? 512 / grid : 1;
  const int each = ceil_div(tiles, room < 1 ? 1 : room);
  hipLaunchKernelGGL((block_scores<D, TILES>), dim3(grid, ceil_div(tiles, each)), dim3(64 * SCORE_WAVES), 0, st, a,
                     width, ceil_div(a.group, 16), each * ceil_div(a.group, 16));
}
template <int D>
void run_scores(const ScoreArgs& a, hipStream_t st) {
  const int pages = (a.b.max_ctx - 1) >> a.c.shift;
  // Two tiles of pages a wave, which share its query rows' way from L2, where one each would fill the chip twice (2
  // waves a SIMD).  Measured on MI355X, 8 kv heads, one and two tiles: 6,562 pages, D = 256, 4 tokens 13.1 and 11.4
  // us, 1 token 10.1 and 9.3; 656 pages 5.1 and 6.9, 4.2 and 5.4; 32 sequences of 512 pages, D = 128, 10.9 and 9.4
  if ((long long)pages * a.b.n_seqs * a.c.kv_heads >= 2ll * 1024 * 16)
    run_scores<D, 2>(a, pages, st);
  else
    run_scores<D, 1>(a, pages, st);
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
// keys whose order as whole numbers is theirs, held in registers (up to 8 a lane; longer rows are read again for
// each pass).  Three histograms of their digits (11, 11 and 10 bits, from the top) narrow the smallest selected key
// down to its value; the pages above it, and as many level with it as are left to take, lowest index first, go out
// in ascending order: a wave holds consecutive pages, so ranks are counted from ballots.  A few thousand scores are
// nothing for the memory: the time is the launch, the first loads and the histograms' barriers.  Measured on MI355X
// (graphs of calls): 64 of 6,562 pages for 32 rows 8.7 us, 32 of 512 for 256 rows 6.9 (12.0 and 7.4 with the scores
// read again in every pass and ranks from two prefix sums over the work-group).
constexpr int TOPK_BINS = 2048;
constexpr int TOPK_KEYS = 8;  // of a lane

// -0 as +0, NaN as -inf; larger scores have larger keys
__device__ __forceinline__ uint32_t order_key(float s) {
  if (!(s == s)) s = -INFINITY;
  const uint32_t u = __float_as_uint(s + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Inclusive prefix sum over the lanes of a wave: inside rows of 16, then over the rows.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or_0(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_prefix(uint32_t v) {
  v += dpp_or_0<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
  v += dpp_or_0<0x112, 0xF>(v);
  v += dpp_or_0<0x114, 0xF>(v);
  v += dpp_or_0<0x118, 0xF>(v);
  v += dpp_or_0<0x142, 0xA>(v);  // row_bcast 15 into rows 1 and 3, 31 into rows 2 and 3
  v += dpp_or_0<0x143, 0xC>(v);
  return v;
}

template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void block_topk(TopkArgs a) {
  constexpr int THREADS = 64 * WAVES, PART = THREADS * TOPK_KEYS, PER = TOPK_BINS / THREADS;
  __shared__ uint32_t bins[3][TOPK_BINS];
  __shared__ uint32_t sums[3][WAVES];
  __shared__ uint32_t counts[2][WAVES];
  __shared__ uint32_t found[3][2];  // the digit, and how many keys lie above it
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const RowOf of = seq_of_row(a.b, blockIdx.x / a.kv_heads, lane);
  if (of.b < 0) return;
  const size_t row = blockIdx.x;  // of scores and sel: token and kv head
  const int pos = of.seq.first + of.token;
  const int count = pos < 0 ? 0 : (pos >> a.shift) + 1;  // pages up to the token's own
  int* sel = a.sel + row * a.n_sel;
  if (count <= a.n_sel) {
    for (int i = tid; i < a.n_sel; i += THREADS) sel[i] = i < count ? i : -1;
    return;
  }
  const int m = count - a.n_first - a.n_last;  // between the first and the last, more than are wanted
  const uint32_t want = a.n_sel - a.n_first - a.n_last;
  const float* s = a.scores + row * a.stride + a.n_first;

  // the lane's keys of a part: wave w holds pages [512 w, 512 w + 512) of it, lane l every 64th from l on
  uint32_t keys[TOPK_KEYS];
  auto load = [&](int part) {
#pragma unroll
    for (int e = 0; e < TOPK_KEYS; ++e) {
      const int i = part + (wave * TOPK_KEYS + e) * 64 + lane;
      keys[e] = i < m ? order_key(s[i]) : 0;  // 0: below every score's key
    }
  };
  const bool once = m <= PART;
  if (once) load(0);
  for (int i = tid; i < 3 * TOPK_BINS; i += THREADS) bins[0][i] = 0;
  for (int i = tid; i < a.n_first; i += THREADS) sel[i] = i;
  for (int i = tid; i < a.n_last; i += THREADS) sel[a.n_sel - a.n_last + i] = count - a.n_last + i;
  if (want == 0) return;
  __syncthreads();

  uint32_t key = 0, mask = 0, left = want;  // keys with these top bits hold the smallest selected one
#pragma unroll
  for (int round = 0; round < 3; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
    const uint32_t digit = round == 2 ? 1023 : 2047;
    for (int part = 0; part < m; part += PART) {
      if (!once) load(part);
#pragma unroll
      for (int e = 0; e < TOPK_KEYS; ++e)
        if (keys[e] && (keys[e] & mask) == key) atomicAdd(&bins[round][(keys[e] >> shift) & digit], 1u);
    }
    __syncthreads();
    // bins counted from the top, PER a thread, the waves' sums joined
    uint32_t c[PER], all = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      c[i] = bins[round][TOPK_BINS - 1 - (tid * PER + i)];
      all += c[i];
    }
    const uint32_t upto = wave_prefix(all);
    if (lane == 63) sums[round][wave] = upto;
    __syncthreads();
    uint32_t above = upto - all;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) above += w < wave ? sums[round][w] : 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (above < left && left <= above + c[i]) {
        found[round][0] = TOPK_BINS - 1 - (tid * PER + i);
        found[round][1] = above;
      }
      above += c[i];
    }
    __syncthreads();
    key |= found[round][0] << shift;
    mask |= digit << shift;
    left -= found[round][1];
  }

  uint32_t at = a.n_first, levels = 0;  // where this part's pages go, level ones before it
  for (int part = 0; part < m; part += PART) {
    if (!once) load(part);
    uint32_t over = 0, level = 0;  // of this wave
#pragma unroll
    for (int e = 0; e < TOPK_KEYS; ++e) {
      over += __popcll(__ballot(keys[e] > key));
      level += __popcll(__ballot(keys[e] == key));
    }
    if (lane == 0) {
      counts[0][wave] = over;
      counts[1][wave] = level;
    }
    __syncthreads();
    uint32_t o = 0, v = levels, part_over = 0, part_level = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const uint32_t co = counts[0][w], cl = counts[1][w];
      o += w < wave ? co : 0;
      v += w < wave ? cl : 0;
      part_over += co;
      part_level += cl;
    }
    uint32_t to = at + o + min(v, left) - min(levels, left);
    const unsigned long long below = (1ull << lane) - 1;
#pragma unroll
    for (int e = 0; e < TOPK_KEYS; ++e) {
      const unsigned long long bl = __ballot(keys[e] == key);
      const uint32_t mine = v + __popcll(bl & below);  // level keys before this one
      const bool take = keys[e] > key || (keys[e] == key && mine < left);
      const unsigned long long taken = __ballot(take);
      if (take) sel[to + __popcll(taken & below)] = a.n_first + part + (wave * TOPK_KEYS + e) * 64 + lane;
      to += __popcll(taken);
      v += __popcll(bl);
    }
    at += part_over + min(levels + part_level, left) - min(levels, left);
    levels += part_level;
    if (!once) __syncthreads();  // counts are read
  }
}

int launch_block_topk(const TopkArgs& a, void* stream) {
  (void)hipGetLastError();
  const dim3 grid(a.b.n_tokens * a.kv_heads);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  // as many waves as hold every score of the longest row
  if (a.b.max_ctx >> a.shift <= 4 * 64 * TOPK_KEYS)
    hipLaunchKernelGGL((block_topk<4>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((block_topk<16>), grid, dim3(1024), 0, st, a);
  return hipGetLastError() == hipSuccess ? HCR_OK : HCR_EHIP;
}

}  // namespace hcr
