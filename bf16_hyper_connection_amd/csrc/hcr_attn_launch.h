// Launches of attention over one kind of pages (CODE) and of positions (SEEN): which kernel takes a call, by its plan.
#pragma once

#include "hcr_attn_rows.h"

namespace hcr {

template <int D, int MT, int SEEN, int CODE, bool PAIRED>
void run_part(const AttnArgs& a, int grid, hipStream_t st) {
  const dim3 threads(64 * a.plan.row_waves * a.plan.groups);
  const int lds = attn_lds(D, a.plan);
  // one wave's rows, and not several tokens' lists, which mostly name the same pages
  if constexpr (!PAIRED) {
    if (a.plan.row_waves * a.plan.row_blocks == 1 && (SEEN != LISTED || a.b.max_tokens == 1)) {
      hipLaunchKernelGGL((attn_part<D, MT, SEEN, true, CODE, false>), dim3(grid), threads, lds, st, a);
      return;
    }
  }
  hipLaunchKernelGGL((attn_part<D, MT, SEEN, false, CODE, PAIRED>), dim3(grid), threads, lds, st, a);
}
template <int D, int SEEN, int CODE, bool PAIRED>
void run_rows(const AttnArgs& a, int grid, hipStream_t st) {
  const dim3 threads(64 * ROWS_WAVES);
  switch (a.plan.q_tiles) {
    case 2: hipLaunchKernelGGL((attn_rows_part<D, 2, SEEN, CODE, PAIRED>), dim3(grid), threads, 0, st, a); break;
    case 3: hipLaunchKernelGGL((attn_rows_part<D, 3, SEEN, CODE, PAIRED>), dim3(grid), threads, 0, st, a); break;
    default: hipLaunchKernelGGL((attn_rows_part<D, 4, SEEN, CODE, PAIRED>), dim3(grid), threads, 0, st, a);
  }
}
template <int D, int SEEN, int CODE, bool PAIRED>
void run_attn(const AttnArgs& a, int grid, int join_grid, hipStream_t st) {
  // a wave a row where rows have few parts, four where many
  const int join = a.plan.items > 2 * (SEEN == LISTED ? a.b.n_tokens : a.b.n_seqs) ? 256 : 64;
  constexpr bool BOTH = CODE != HCR_BF16 || SEEN == WINDOW;  // kernels: a wave's rows, or four waves' together
  // (a plan of row blocks over codes has those rows shared: it has pages of a tile at least)
  if constexpr (BOTH) {
    if (a.plan.shared) {
      run_rows<D, SEEN, CODE, PAIRED>(a, grid, st);
      if (join_grid) hipLaunchKernelGGL((attn_join<D, SEEN, ROWS_SHIFT, PAIRED>), dim3(join_grid), dim3(join), 0, st, a);
      return;
    }
  }
  if constexpr (!PAIRED || CODE == HCR_BF16) {
    if constexpr (BOTH || D == 64) {
      run_part<D, 1, SEEN, CODE, PAIRED>(a, grid, st);
    } else {
      a.plan.q_tiles == 1 ? run_part<D, 1, SEEN, CODE, PAIRED>(a, grid, st) : run_part<D, 2, SEEN, CODE, PAIRED>(a, grid, st);
    }
    if (join_grid)
      hipLaunchKernelGGL((attn_join<D, SEEN, Format<CODE, D>::SHIFT, PAIRED>), dim3(join_grid), dim3(join), 0, st, a);
  }
}
template <int D, int SEEN, int CODE>
void run_kind(const AttnArgs& a, int grid, int join_grid, hipStream_t st) {
  if constexpr (SEEN != LISTED) {
    if (a.plan.paired) return run_attn<D, SEEN, CODE, true>(a, grid, join_grid, st);
  }
  run_attn<D, SEEN, CODE, false>(a, grid, join_grid, st);
}
template <int SEEN, int CODE>
int launch_seen(const AttnArgs& a, void* stream) {
  const AttnPlan& p = a.plan;
  const int grid = (int)attn_grid(a.c, p);
  const int join_grid = attn_joins(p) ? a.b.n_tokens * a.heads : 0;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  switch (a.c.head_dim) {
    case 64: run_kind<64, SEEN, CODE>(a, grid, join_grid, st); break;
    case 128: run_kind<128, SEEN, CODE>(a, grid, join_grid, st); break;
    default: run_kind<256, SEEN, CODE>(a, grid, join_grid, st);
  }
  return hipGetLastError() == hipSuccess ? HCR_OK : HCR_EHIP;
}

}  // namespace hcr
