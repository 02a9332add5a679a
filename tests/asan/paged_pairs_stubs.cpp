// Host checks of attention's pairs of a set and a row block (hcr_paged_layout.h, hcr_paged_api.cpp), beside paged_stubs.cpp
// and paged_q8_stubs.cpp in a build of the host code under AddressSanitizer and UndefinedBehaviorSanitizer.
#include <stdio.h>
#include <vector>

#include "hcr_paged_layout.h"

using namespace hcr;

#define CHECK(x)                                             \
  do {                                                       \
    if (!(x)) {                                              \
      snprintf(why, sizeof(why), "%s line %d", #x, __LINE__); \
      return why;                                            \
    }                                                        \
  } while (0)

static char why[256];

static AttnPlan plan_of(const CacheArgs& c, const CodeArgs& x, const WindowArgs& w, const BatchArgs& b, int heads) {
  return coded(x) || w.size ? attn_plan_more(c, x, w, b, heads, 0) : attn_plan(c, b, heads, 0);
}
static int shift_of(const CacheArgs& c, const CodeArgs& x, const AttnPlan& p) {
  return p.shared ? ROWS_SHIFT : tile_shift(coded(x), c.head_dim);
}

// What the device makes of a plan and of the sequences' tokens and lengths: the tiles of the longest run, with every
// invariant of its work-groups and parts checked (-1 and `fail` where one does not hold).
static long long longest_run(const CacheArgs& c, const CodeArgs& x, const WindowArgs& w, const BatchArgs& b, int heads,
                             const std::vector<Seq>& seqs, const AttnPlan& p, const char** fail) {
  const int group = heads / c.kv_heads, shift = shift_of(c, x, p);
  long long tiles = 0, longest = 0;
  int pairs = 0, fewest = 1 << 30, most = 0;
  for (const Seq& s : seqs) {
    const int blocks = set_blocks(p, s.tokens * group), n = pair_tiles(p, w, s, group, shift);
    pairs += blocks;
    tiles += (long long)blocks * n;
    if (blocks && blocks < fewest) fewest = blocks;
    if (blocks > most) most = blocks;
    // a row block's own tiles are no more than those that its pair counts as
    for (int rb = 0; rb < blocks; ++rb) {
      const int low = rb * attn_rows(p) / group, high = ((rb + 1) * attn_rows(p) - 1) / group;
      const int len_max = s.first + (high < s.tokens - 1 ? high : s.tokens - 1) + 1;
      const int own = w.size ? window_tiles(w, s.first + low + 1, len_max, shift).tiles
                             : ceil_div(len_max > 0 ? len_max : 0, 1 << shift);
      if (own > n) return *fail = "a row block has more tiles than its pair", -1;
    }
  }
  if (pairs > pairs_bound(p, b.n_seqs, (long long)b.n_tokens * group)) return *fail = "more pairs than the bound", -1;
  const PairCut cut = pair_cut(p, tiles, pairs, b.n_seqs, fewest, most);
  if (cut.kind == ALIKE) {  // what find_seq makes of them fits as it does without pairs
    if (cut.blocks != most || fewest != most) return *fail = "unlike sets (ALIKE)", -1;
    if ((long long)p.items * most > p.paired) return *fail = "more runs than work-groups (ALIKE)", -1;
    if (p.items > 1 && 2ll * p.items * most > attn_slots(p)) return *fail = "more parts than places (ALIKE)", -1;
    if (!attn_joins(p) || cut.joins != (p.items > 1)) return *fail = "parts without a join (ALIKE)", -1;
    return run_tiles(p, (int)(tiles / most < 1 << 30 ? tiles / most : 1 << 30));
  }
  if (cut.kind == EVEN) {
    if ((long long)p.shares * cut.run < tiles || p.shares > p.paired) return *fail = "tiles behind the last run (EVEN)", -1;
    std::vector<char> used(attn_slots(p));
    long long first = 0;
    for (const Seq& s : seqs)
      for (int rb = 0; rb < set_blocks(p, s.tokens * group); ++rb) {
        const int n = pair_tiles(p, w, s, group, shift), parts = run_parts((int)first, n, cut.run);
        for (int k = 0; k < parts && parts > 1; ++k) {
          const int slot = part_slot((int)first / cut.run + k, cut.run, (int)first);
          if (slot < 0 || slot >= attn_slots(p) || used[slot]) return *fail = "a part without a place of its own (EVEN)", -1;
          used[slot] = 1;
        }
        if (parts > 1 && !attn_joins(p)) return *fail = "parts without a join (EVEN)", -1;
        first += n;
      }
    return cut.run;
  }
  int items = 0, slots = 0;
  for (const Seq& s : seqs) {
    const int blocks = set_blocks(p, s.tokens * group), n = pair_tiles(p, w, s, group, shift);
    const PairRuns r = pair_runs(n, cut.run);
    if (r.parts < 1 || (long long)r.parts * r.each < n || (long long)(r.parts - 1) * r.each >= n)
      return *fail = "a pair's runs do not cover its tiles", -1;
    if (r.each > cut.run) return *fail = "a run is too long", -1;
    if (blocks && r.each > longest) longest = r.each;
    items += blocks * r.parts;
    if (r.parts > 1) slots += blocks * r.parts;
  }
  if (items > p.paired) return *fail = "more runs than work-groups", -1;
  if (slots > attn_slots(p)) return *fail = "more parts than places", -1;
  if (slots && !attn_joins(p)) return *fail = "parts without a join", -1;
  return longest;
}

static const char* check_pairs() {
  unsigned seed = 3;
  auto rnd = [&](int n) { return int((seed = seed * 1664525u + 1013904223u) >> 8) % n; };
  for (int code : {(int)HCR_BF16, (int)HCR_INT8, (int)HCR_E4M3})
    for (int D : {64, 128, 256})
      for (int page : {32, 64, 256})
        for (int kv : {1, 3, 8, 200})
          for (int group : {1, 4, 16, 33, 64})
            for (int count : {1, 2, 3, 64, 65, 300})
              for (int tokens : {1, 4, 100, 2000, 20000})
                for (int ctx : {0, 1, 33, 700, 4096, 9001, 420000})
                  for (int size : {0, 1, 100, 5000})
                    for (int turn = 0; turn < 4; ++turn) {  // all the longest, random, one prompt among single tokens, none
                      const CodeArgs x{nullptr, nullptr, code};
                      if (coded(x) && page == 32) continue;
                      if (count * tokens > 100000) continue;
                      const CacheArgs c{nullptr, nullptr, nullptr, 10, kv, D, log2_of(page)};
                      const WindowArgs w{size, size ? rnd(300) : 0};
                      std::vector<Seq> seqs(count);
                      int rows = 0;
                      for (Seq& s : seqs) {
                        s.row = rows;
                        s.tokens = turn == 0 ? tokens : turn == 1 ? rnd(tokens + 1) : turn == 3 ? 0 : &s == &seqs[count / 2] ? tokens : 1;
                        s.first = (turn == 0 ? ctx : rnd(ctx + 1)) - s.tokens;
                        if (turn == 2 && &s == &seqs[count / 2]) s.first = (ctx < tokens ? ctx : tokens) - tokens;
                        rows += s.tokens;
                      }
                      const BatchArgs b{nullptr, nullptr, nullptr, ctx / page + 1, count, rows, tokens, ctx};
                      const AttnPlan p = plan_of(c, x, w, b, kv * group);
                      const long long bound = pairs_bound(p, count, (long long)rows * group);
                      // counted where a work-group would go through many positions, or most work-groups have no rows
                      const int shift = shift_of(c, x, p), block = ceil_div(attn_rows(p), group) + 1;
                      const int tiles = window_bound(w, ctx, p.shared && block < tokens ? block : tokens, shift);
                      const long long each = 1ll * count * p.row_blocks;
                      const bool counted = p.row_blocks > 1 && count > 1 &&
                                           (p.whole ? 2 * bound < each && each * kv >= 4096
                                                    : ((long long)count * tiles << shift) >= 2048ll * p.items);
                      CHECK(p.paired ? counted && attn_grid(c, p) * 1024 < 1ll << 32
                                     : !counted || (bound + 4096) * kv * 1024 > (1ll << 32) - (1 << 23));
                      CHECK(!coded(x) || p.shared || p.row_waves * p.groups <= 8);  // what their kernels are held to
                      if (!p.paired) continue;
                      CHECK(p.shares >= 1 && attn_grid(c, p) >= (long long)p.paired * kv && attn_grid(c, p) % XCDS == 0);
                      const char* fail = nullptr;
                      const long long longest = longest_run(c, x, w, b, kv * group, seqs, p, &fail);
                      if (fail) {
                        snprintf(why, sizeof(why), "%s: code %d D %d page %d kv %d group %d sets %d tokens %d ctx %d size %d turn %d",
                                 fail, code, D, page, kv, group, count, tokens, ctx, size, turn);
                        return why;
                      }
                      CHECK(longest >= 0);
                    }
  return nullptr;
}

extern "C" const char* paged_pairs_checks(void) {
  if (const char* e = check_pairs()) return e;
  // the largest that the checks of a batch let through
  AttnPlan p{};
  p.least = p.shares = 1;
  CHECK(pair_cut(p, 1ll << 55, 1 << 30, 2, 1, 9).run == 1 << 26 && pair_cut(p, 0, 0, 2, 1 << 30, 0).kind == APART);
  const PairRuns r = pair_runs(1 << 25, 1 << 26), one = pair_runs(1 << 25, 1);
  CHECK(r.parts == 1 && r.each == 1 << 25 && (long long)one.parts * one.each >= 1 << 25);
  return "ok";
}

// Tiles of the longest run, or of the longest whole pair, of a batch of one prompt (tokens of its own alone) among `singles`
// single tokens at `ctx`; negative where an invariant fails.
extern "C" long long paged_pairs_longest(int code, int D, int kv, int heads, int size, int prompt, int singles, int ctx,
                                         long long* total) {
  const CodeArgs x{nullptr, nullptr, code};
  const CacheArgs c{nullptr, nullptr, nullptr, 10, kv, D, 6};
  const WindowArgs w{size, 0};
  std::vector<Seq> seqs(singles + 1, Seq{0, 1, ctx - 1});
  seqs[singles / 2] = Seq{0, prompt, 0};
  const BatchArgs b{nullptr, nullptr, nullptr, 1 << 20, singles + 1, singles + prompt, prompt, ctx > prompt ? ctx : prompt};
  const AttnPlan p = plan_of(c, x, w, b, heads);
  *total = 0;
  for (const Seq& s : seqs)
    *total += (long long)set_blocks(p, s.tokens * (heads / kv)) * pair_tiles(p, w, s, heads / kv, shift_of(c, x, p));
  if (!p.paired) return -1;
  const char* fail = nullptr;
  const long long n = longest_run(c, x, w, b, heads, seqs, p, &fail);
  return fail ? -2 : n;
}

// Whether a work-group takes a set whole, of `sets` single tokens with up to `ctx` positions in pages of 64 (size: of a window).
extern "C" int paged_plan_whole(int code, int D, int kv, int heads, int size, int sets, int ctx) {
  const CacheArgs c{nullptr, nullptr, nullptr, 10, kv, D, 6};
  const BatchArgs b{nullptr, nullptr, nullptr, 1 << 20, sets, sets, 1, ctx};
  return plan_of(c, CodeArgs{nullptr, nullptr, code}, WindowArgs{size, 0}, b, heads).whole;
}

// Pages that the longest run of an attention call over codes or through a window spans, of sequences of up to max_ctx positions
// that are all as long (n_sel: of lists); 0 where pairs are counted.
extern "C" int paged_more_run_pages(int code, int D, int kv, int page, int heads, int n_seqs, int max_tokens, int max_ctx,
                                    int n_sel, int size, int first) {
  const CodeArgs x{nullptr, nullptr, code};
  const CacheArgs c{nullptr, nullptr, nullptr, 10, kv, D, log2_of(page)};
  const WindowArgs w{size, first};
  const BatchArgs b{nullptr, nullptr, nullptr, ceil_div(max_ctx, page), n_seqs, n_seqs * max_tokens, max_tokens, max_ctx};
  const AttnPlan p = attn_plan_more(c, x, w, b, heads, n_sel);
  if (p.paired) return 0;
  const int shift = shift_of(c, x, p);
  const int low = attn_rows(p) * (p.row_blocks - 1) / (heads / kv);  // the last row block's first token
  const int tiles = n_sel ? n_sel << (c.shift - shift)
                    : size ? window_tiles(w, max_ctx - max_tokens + low + 1, max_ctx, shift).tiles
                           : ceil_div(max_ctx, 1 << shift);
  int run = p.whole ? tiles : n_sel ? run_tiles_listed(p, tiles, b.n_tokens) : run_tiles(p, n_seqs * tiles);
  if (run > tiles) run = tiles;
  return run >> (c.shift - shift);
}

// Whether a call over pages of `page` positions counts its pairs.
extern "C" int paged_plan_paired(int code, int D, int kv, int page, int heads, int size, int n_seqs, int n_tokens, int max_tokens,
                                 int max_ctx) {
  const CacheArgs c{nullptr, nullptr, nullptr, 10, kv, D, log2_of(page)};
  const BatchArgs b{nullptr, nullptr, nullptr, 1 << 20, n_seqs, n_tokens, max_tokens, max_ctx};
  return plan_of(c, CodeArgs{nullptr, nullptr, code}, WindowArgs{size, 0}, b, heads).paired > 0;
}
