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

// A plan covers every row; the items of any lengths fit its bound and cover every tile once; LDS fits a CU.
static const char* check_plans() {
  unsigned seed = 1;
  auto rnd = [&](int n) { return int((seed = seed * 1664525u + 1013904223u) >> 8) % n; };
  for (int D : {64, 128, 256})
    for (int page : {32, 64, 256})
      for (int kv : {1, 3, 8})
        for (int group : {1, 6, 16, 33, 64})
          for (int seqs : {1, 3, 64, 1000})
            for (int tokens : {1, 4, 100})
              for (int ctx : {0, 1, 32, 33, 700, 9001, 420000})
                for (int n_sel : {0, 1, 7, 64, 1000}) {
                  const CacheArgs c{nullptr, nullptr, nullptr, 10, kv, D, log2_of(page)};
                  const BatchArgs b{nullptr, nullptr, nullptr, ctx / page + 1, seqs, seqs * tokens, tokens, ctx};
                  const AttnPlan p = attn_plan(c, b, kv * group, n_sel);
                  const int rows = n_sel ? group : tokens * group;
                  CHECK(p.q_tiles == 1 || (p.q_tiles == 2 && D != 64));
                  CHECK(p.row_waves * p.groups <= attn_waves(D, p.q_tiles) && p.groups >= 1 && p.row_waves >= 1);
                  CHECK(p.row_blocks * attn_rows(p) >= rows && (p.row_blocks - 1) * attn_rows(p) < rows);
                  CHECK(attn_lds(D, p) <= 160 * 1024 && attn_lds(D, p) >= attn_rows(p) * D * 2);
                  CHECK(p.least >= 1 && p.items >= 1);
                  if (p.whole) {
                    CHECK(p.items == (n_sel ? seqs * tokens : seqs) && !attn_joins(p));
                    continue;
                  }
                  for (int turn = 0; turn < 3; ++turn) {  // lengths: all the longest, random, one long
                    const int sets = n_sel ? seqs * tokens : seqs;
                    if (sets > 2000) continue;
                    std::vector<int> t(sets);
                    const int most = n_sel ? n_sel * (page / TILE) : ceil_div(ctx, TILE);
                    int all = 0;
                    for (int& x : t) {
                      x = n_sel || turn == 0 ? most : turn == 1 ? rnd(most + 1) : &x == &t[0] ? most : 0;
                      if (x < 1) x = 1;
                      all += x;
                    }
                    int run = run_tiles(p, all), runs = 0;
                    CHECK(run >= 1 && (long long)run * p.items >= all);
                    for (int x : t) runs += ceil_div(x, run);
                    bool apart = sets <= 64 && runs <= p.items;
                    if (n_sel) {
                      CHECK(p.items % sets == 0);
                      run = run_tiles_listed(p, most, sets);
                      apart = true;
                    } else if (sets <= 64 && !apart && run_tiles_apart(p, all, sets) > 0) {
                      run = run_tiles_apart(p, all, sets);
                      apart = true;
                    }
                    std::vector<char> used(2 * p.items);
                    int first = 0;
                    for (int x : t) {  // every part of every set has a place of its own
                      const int n = run_parts(first, x, run);
                      CHECK(n >= 1 && (n == 1 || attn_joins(p)) && (!apart || n == ceil_div(x, run)));
                      for (int k = 0; k < n && (n > 1 || apart); ++k) {
                        const int slot = part_slot(first / run + k, run, first);
                        CHECK(slot >= 0 && slot < 2 * p.items && !used[slot]);
                        used[slot] = 1;
                      }
                      first += apart ? n * run : x;
                    }
                  }
                }
  return nullptr;
}

extern "C" const char* paged_index_checks(void) {
  if (const char* e = check_sequences()) return e;
  if (const char* e = check_cells()) return e;
  if (const char* e = check_plans()) return e;
  return "ok";
}

// Pages (entries of a table's row, or of a list) that the longest run of an attention call spans: `all` tiles of the
// sequences together, `longest` of one (dense calls).
extern "C" int paged_run_pages(int D, int kv, int page, int heads, int n_seqs, int n_tokens, int max_tokens, int max_ctx,
                               int n_sel, int all, int longest) {
  const CacheArgs c{nullptr, nullptr, nullptr, 10, kv, D, log2_of(page)};
  const BatchArgs b{nullptr, nullptr, nullptr, ceil_div(max_ctx, page), n_seqs, n_tokens, max_tokens, max_ctx};
  const AttnPlan p = attn_plan(c, b, heads, n_sel);
  const int tiles = n_sel ? n_sel << (c.shift - TILE_SHIFT) : longest;
  int run = p.whole ? tiles : n_sel ? run_tiles_listed(p, tiles, n_tokens) : run_tiles(p, all);
  if (run > tiles) run = tiles;
  return run >> (c.shift - TILE_SHIFT);
}
