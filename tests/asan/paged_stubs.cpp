// Host-only stand-ins for the paged cache's launchers, and a program's worth of checks of its index arithmetic, so
// that hcr_paged_api.cpp can be built with the host compiler under AddressSanitizer and
// UndefinedBehaviorSanitizer.  The launchers return HCR_EHIP: a call that the argument checks let through shows.
#define __host__
#define __device__
#include <stdio.h>
#include <string.h>
#include <vector>

#include "hcr_paged_layout.h"

namespace hcr {
int launch_attn(const AttnArgs&, void*) { return HCR_EHIP; }
int launch_append(const AppendArgs&, void*) { return HCR_EHIP; }
int launch_block_scores(const ScoreArgs&, void*) { return HCR_EHIP; }
int launch_block_topk(const TopkArgs&, void*) { return HCR_EHIP; }
}  // namespace hcr

using namespace hcr;

#define CHECK(x)                                             \
  do {                                                       \
    if (!(x)) {                                              \
      snprintf(why, sizeof(why), "%s line %d", #x, __LINE__); \
      return why;                                            \
    }                                                        \
  } while (0)

static char why[256];

// Whatever q_start and ctx_len hold, a sequence's rows and positions stay inside the batch's bounds.
static const char* check_sequences() {
  const int odd[] = {-2147483647 - 1, -7, -1, 0, 1, 2, 5, 16, 17, 100, 4096, 1 << 30, 2147483647};
  for (int n_tokens : {1, 5, 100})
    for (int max_tokens : {1, 4, 16})
      for (int max_ctx : {0, 1, 100, 4096})
        for (int s0 : odd)
          for (int s1 : odd)
            for (int ctx : odd) {
              const BatchArgs b{nullptr, nullptr, nullptr, 1, 1, n_tokens, max_tokens, max_ctx};
              const Seq q = seq_of(b, s0, s1, ctx);
              CHECK(q.tokens >= 0 && q.tokens <= max_tokens && q.row >= 0);
              if (q.tokens == 0) continue;
              CHECK(q.row == s0 && q.row + q.tokens <= n_tokens && q.row + q.tokens <= (long long)s1);
              CHECK(q.first + q.tokens >= 0 && q.first + q.tokens <= max_ctx);
              if (ctx >= 0 && ctx <= max_ctx) CHECK(q.first + q.tokens == ctx);
            }
  for (int p : odd) CHECK(page_or_none(p, 7) == (p >= 0 && p < 7 ? p : -1));
  return nullptr;
}

// Each cell of a page has one place, inside the page.
static const char* check_cells() {
  for (int D : {64, 128, 256})
    for (int page : {32, 64, 128, 256}) {
      const int shift = log2_of(page);
      CHECK(1 << shift == page && page_ok(page) && head_dim_ok(D));
      std::vector<char> k(D * page), v(D * page);
      for (int s = 0; s < page; ++s)
        for (int d = 0; d < D; ++d) {
          const int a = k_at(shift, s, d), b = v_at(D, s, d);
          CHECK(a >= 0 && a < D * page && b >= 0 && b < D * page && !k[a] && !v[b]);
          k[a] = v[b] = 1;
        }
      const CacheArgs c{nullptr, nullptr, nullptr, 1 << 20, 16, D, shift};
      CHECK(head_base(c, 0, 0) == 0 && head_base(c, 0, 1) == size_t(D) * page);
      CHECK(head_base(c, (1 << 20) - 1, 15) == ((size_t(1) << 24) - 1) * D * page);
    }
  return nullptr;
}

// A plan covers every row and every tile, and the device's walk over it (as in the kernel) visits each tile of a
// split once, in its waves' turns, never one outside.
static const char* check_plans() {
  for (int D : {64, 128, 256})
    for (int page : {32, 64, 256})
      for (int kv : {1, 8})
        for (int group : {1, 6, 16, 33, 64})
          for (int seqs : {1, 3, 64, 1000})
            for (int tokens : {1, 4, 100})
              for (int ctx : {0, 1, 32, 33, 700, 9001, 420000})
                for (int n_sel : {0, 1, 7, 64, 1000}) {
                  const CacheArgs c{nullptr, nullptr, nullptr, 10, kv, D, log2_of(page)};
                  const BatchArgs b{nullptr, nullptr, nullptr, ctx / page + 1, seqs, seqs * tokens, tokens, ctx};
                  const AttnPlan p = attn_plan(c, b, kv * group, n_sel);
                  const int rows = n_sel ? group : tokens * group;
                  CHECK(p.q_tiles == 1 || p.q_tiles == 2 || (p.q_tiles == 4 && D != 256));
                  CHECK(p.row_blocks * p.q_tiles * 16 >= rows && (p.row_blocks - 1) * p.q_tiles * 16 < rows);
                  const int tiles = n_sel ? n_sel * (page / TILE) : (ctx + TILE - 1) / TILE;
                  CHECK(p.splits >= 1 && p.chunk >= 1 && (long long)p.splits * p.chunk >= tiles);
                  CHECK(p.splits == 1 || (p.splits - 1) * p.chunk < tiles);
                }
  for (int psh : {0, 1, 3})
    for (int chunk : {1, 3, 8, 100, 700})
      for (int tiles : {1, 5, 8, 150, 1500}) {
        std::vector<int> seen(tiles);
        for (int lo = 0; lo < tiles; lo += chunk) {
          const int hi = lo + chunk < tiles ? lo + chunk : tiles;
          for (int wave = 0; wave < ATTN_WAVES; ++wave)
            for (int pb = lo >> psh; pb << psh < hi; pb += 64) {
              const int end = hi < (pb + 64) << psh ? hi : (pb + 64) << psh;
              int tile = lo > pb << psh ? lo : pb << psh;
              tile += (wave - (tile - lo)) & (ATTN_WAVES - 1);
              for (; tile < end; tile += ATTN_WAVES) {
                const int at = (tile >> psh) - pb;
                CHECK(at >= 0 && at < 64 && tile >= lo && tile < hi && (tile - lo) % ATTN_WAVES == wave);
                ++seen[tile];
              }
            }
        }
        for (int t = 0; t < tiles; ++t) CHECK(seen[t] == 1);
      }
  return nullptr;
}

extern "C" const char* paged_index_checks(void) {
  if (const char* e = check_sequences()) return e;
  if (const char* e = check_cells()) return e;
  if (const char* e = check_plans()) return e;
  return "ok";
}
