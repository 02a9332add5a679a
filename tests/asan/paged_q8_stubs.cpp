// Host-only stand-ins and index checks of the paged cache's other forms (codes, windows, reading back), beside
// paged_stubs.cpp in a build of the host code under AddressSanitizer and UndefinedBehaviorSanitizer.
#include <stdio.h>
#include <vector>

#include "hcr_paged_layout.h"

namespace hcr {
int launch_read(const ReadArgs&, void*) { return HCR_EHIP; }
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

// Each cell of a page of codes has one place, inside the page, and a tile lies in one page.
static const char* check_cells() {
  for (int page : {32, 64, 128, 256}) CHECK(code_page_ok(page) == (page != 32));
  CHECK(!code_page_ok(16) && !code_page_ok(512) && !code_page_ok(96));
  for (int D : {64, 128, 256}) {
    CHECK(tile_shift(false, D) == TILE_SHIFT && tile_shift(true, D) == (D == 256 ? 5 : 6));
    for (int page : {64, 128, 256}) {
      const int shift = log2_of(page);
      std::vector<char> k(D * page), v(D * page);
      for (int s = 0; s < page; ++s)
        for (int d = 0; d < D; ++d) {
          const int a = k_code_at(shift, s, d), b = v_code_at(D, s, d);
          CHECK(a >= 0 && a < D * page && b >= 0 && b < D * page && !k[a] && !v[b]);
          k[a] = v[b] = 1;
        }
      const CacheArgs c{nullptr, nullptr, nullptr, 1 << 20, 16, D, shift};
      CHECK(scale_base(c, (1 << 20) - 1, 15) == ((size_t(1) << 24) - 1) * page);
    }
  }
  return nullptr;
}

// The operands of a tile: what a lane loads lies inside the tile, every cell is loaded once, and the positions of a
// lane's products are those of its values.
static const char* check_operands() {
  for (int D : {64, 128, 256})
    for (int page : {64, 128, 256}) {
      const int shift = log2_of(page), tile = 1 << tile_shift(true, D), each = tile / 4;
      for (int off = 0; off < page; off += tile) {
        std::vector<int> k(D * page), v(D * page);
        for (int lane = 0; lane < 64; ++lane) {
          const int li = lane & 15, lg = lane >> 4;
          for (int j = 0; j < D / 64; ++j)
            for (int t = 0; t < tile / 16; ++t) {
              const int slot = off + each * (li >> 2) + (li & 3) + 4 * t;
              const int at = off * 16 + ((lg << shift) + each * (li >> 2) + (li & 3)) * 16 + j * (4 << shift << 4) + t * 64;
              for (int e = 0; e < 16; ++e) {
                CHECK(at + e == k_code_at(shift, slot, 64 * j + 16 * lg + e));
                ++k[at + e];
              }
            }
          for (int d = 0; d < D / 16; ++d) {
            const int at = off * D + 256 * d +
                           (each == 16 ? (lg * D + li) * 16 : ((lg >> 1) * D + li) * 16 + (lg & 1) * 8);
            for (int e = 0; e < each; ++e) {
              CHECK(at + e == v_code_at(D, off + each * lg + e, 16 * d + li));
              ++v[at + e];
            }
          }
        }
        int keys = 0, values = 0;
        for (int x : k) {
          CHECK(x <= 1);
          keys += x;
        }
        for (int x : v) {
          CHECK(x <= 1);
          values += x;
        }
        CHECK(keys == tile * D && values == tile * D);
      }
      // row r of key tile t, as it comes back to lane row r / 4 in place r % 4, is that lane's product 4 t + r % 4
      for (int t = 0; t < tile / 16; ++t)
        for (int r = 0; r < 16; ++r) CHECK(each * (r >> 2) + (r & 3) + 4 * t == each * (r / 4) + (4 * t + r % 4));
    }
  return nullptr;
}

// The tiles of a window are those that some row sees a position of, each once.
static const char* check_windows() {
  for (int shift : {5, 6})
    for (int size : {1, 2, 31, 32, 33, 64, 65, 100, 1000, 1 << 30})
      for (int first : {0, 1, 4, 32, 64, 65, 200, 1 << 30})
        for (int len_min : {-70, -1, 0, 1, 2, 32, 33, 64, 65, 127, 400, 1000})
          for (int rows : {0, 1, 5, 63, 300}) {
            const WindowArgs w{size, first};
            const int len_max = len_min + rows;
            const WindowTiles t = window_tiles(w, len_min, len_max, shift);
            CHECK(t.firsts >= 0 && t.low >= t.firsts && t.tiles >= 1);
            const int end = len_max > 0 ? ((len_max - 1) >> shift) + 1 : 0;
            std::vector<int> seen(end + 1), taken(end + 1);
            for (int len = len_min; len <= len_max; ++len)
              for (int p = 0; p < len; ++p)
                if (p >= len - size || p < first) seen[p >> shift] = 1;
            for (int i = 0; i < t.tiles; ++i) {
              const int at = i < t.firsts ? i : i + t.low - t.firsts;
              CHECK(at >= 0 && (at < end || end == 0));
              ++taken[end ? at : 0];
            }
            for (int i = 0; i < end; ++i) CHECK(taken[i] <= 1 && seen[i] <= taken[i]);
          }
  return nullptr;
}

// Plans over codes and windows cover every row, and fit a CU.
static const char* check_plans() {
  for (int code : {(int)HCR_BF16, (int)HCR_INT8, (int)HCR_E4M3})
    for (int D : {64, 128, 256})
      for (int page : {32, 64, 256})
        for (int kv : {1, 3, 8})
          for (int group : {1, 6, 16, 33, 64})
            for (int seqs : {1, 3, 64, 1000})
              for (int tokens : {1, 4, 100, 2000})
                for (int ctx : {0, 1, 32, 33, 700, 9001, 420000})
                  for (int n_sel : {0, 7, 1000})
                    for (int size : {0, 1, 64, 4096}) {
                      if (n_sel && size) continue;
                      const CodeArgs x{nullptr, nullptr, code};
                      if (!coded(x) && !size) continue;
                      if (coded(x) && page == 32) continue;
                      const CacheArgs c{nullptr, nullptr, nullptr, 10, kv, D, log2_of(page)};
                      const BatchArgs b{nullptr, nullptr, nullptr, ctx / page + 1, seqs, seqs * tokens, tokens, ctx};
                      const AttnPlan p = attn_plan_more(c, x, WindowArgs{size, 4}, b, kv * group, n_sel);
                      const int rows = n_sel ? group : tokens * group;
                      CHECK(p.shared ? p.q_tiles >= 2 && p.q_tiles <= 4 && p.groups == 1 && p.row_waves == 1
                                     : p.q_tiles == 1);
                      CHECK(p.row_waves * p.groups <= attn_waves(D, p.q_tiles) && p.groups >= 1 && p.row_waves >= 1);
                      CHECK(p.row_blocks * attn_rows(p) >= rows && (p.row_blocks - 1) * attn_rows(p) < rows);
                      if (!p.shared) CHECK(attn_lds(D, p) <= 160 * 1024 && attn_lds(D, p) >= attn_rows(p) * D * 2);
                      if (p.shared) CHECK(page >= 64);
                      CHECK(p.least >= 1 && p.items >= 1);
                      if (p.whole) CHECK(p.items == (n_sel ? seqs * tokens : seqs) && !attn_joins(p));
                    }
  return nullptr;
}

// Parts of a read cover every row of any sequence.
static const char* check_reads() {
  for (int max_tokens : {1, 2, 31, 32, 33, 64, 100})
    for (int first = -70; first < 70; ++first) {
      const BatchArgs b{nullptr, nullptr, nullptr, 1, 1, 1000, max_tokens, 1000};
      const int start = read_start(first);
      CHECK(start <= first && start % READ_SLOTS == 0 && start + read_parts(b) * READ_SLOTS >= first + max_tokens);
      for (int shift : {5, 6, 8})  // pages that an append can touch, from a sequence's first new position on
        CHECK((first < 0 ? 0 : first) / (1 << shift) + parts_touched(max_tokens, shift) > (first + max_tokens - 1) / (1 << shift));
    }
  return nullptr;
}

extern "C" const char* paged_q8_index_checks(void) {
  if (const char* e = check_cells()) return e;
  if (const char* e = check_operands()) return e;
  if (const char* e = check_windows()) return e;
  if (const char* e = check_plans()) return e;
  if (const char* e = check_reads()) return e;
  return "ok";
}
