// Attention of many query rows over the same keys, gfx950 (MI355X): the same sums as hcr_attn_device.h, cut otherwise.
//
// A work-group of four waves takes RT tiles of 16 rows and, one after another, tiles of 64 positions.  Each wave owns 16
// of a tile's keys and a quarter of its values' dimensions, so that every byte of a page is loaded (and, of codes,
// widened) by one wave alone, however many the rows:
//   S^T = K Q^T : a wave's 16 keys with every row tile (query rows in LDS, one copy for the four waves),
//   where a row's maximum may move the maxima over the four waves through LDS; the probabilities' BF16 parts into LDS as
//   operands,
//   O^T += V^T P^T : a wave's dimensions with every row tile, all 64 positions.
// A wave's accumulators are the outputs of its dimensions: nothing is joined but the sums.  Two barriers a tile, of LDS
// alone, behind the first tile of whole sequences a third where a maximum moves: keys of the next tile are on their way behind this one's products, values behind theirs.
//
// Bound by the vector units beside the matrix cores, and by waits where a work-group is alone on its CU: of prompts through
// a window of 1,024 (32 heads of 128 over 8, BF16, 64 rows a work-group) a tile takes one 2.4 us alone and three of them
// 2.4 together, vector instructions being issued in three quarters of the clocks; over codes widening comes on top (E4M3 2
// instructions for 4 codes, int8 6), exponents and the three BF16 parts of float outputs.  Measured on MI355X: those
// prompts (2,049 tokens, 34.5 GFLOP) 82 us, 0.42 PFLOP/s; 36 rows of 4 sequences of up to 9,001 (int8, D = 256, float
// outputs) 30 us, 2.9 TB/s, and 7 for the join: 9 tiles a work-group behind the waits for its first loads; of one of
// 100,000 115 us, 3.6 TB/s (24 rows 94; E4M3 100); 24 rows through a window of 8,192 17 us and 4 for the join.
#pragma once

#include "hcr_attn_device.h"

namespace hcr {

constexpr int ROWS_WAVES = 4;

// Waits for every load, in a form that the compiler's own count of them sees.
__device__ __forceinline__ void loads_done() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// Every line of the arguments asked for at once: the compiler loads each where it is first needed, and the first of a
// line waits for memory (24 rows through a window of 8,192 22.2 -> 21.4 us; level in the kernels of single row tiles).
__device__ __forceinline__ void arguments_near(const AttnArgs& a) {
  asm volatile("" ::"s"(a.c.shift), "s"(a.n_sel), "s"(a.plan.items), "s"(a.window.size));
}

template <int CODE>
struct RowsFormat {
  static constexpr bool CODED = CODE != HCR_BF16;
  static constexpr int SHIFT = ROWS_SHIFT;
  static constexpr int TILE = 1 << SHIFT;
  static constexpr int BYTES = CODED ? 1 : 2;
};

template <int D, int RT>
struct RowsLds {
  uint4 q[RT][D / 32][64];        // query rows, as operands
  uint4 p[3][RT][4][2][16];       // parts of probabilities: of 16 keys (a wave's) 8 and 8, of a row each
  f32x4 tops[RT * 16];            // the rows' largest products of a tile, of each wave
  f32x4 sums[RT * 16];            // the rows' sums, of each wave
  int len[RT * 16], rid[RT * 16];  // the rows' lengths, and their rows of q and out (-1: none)
  int risen;                       // the last tile (counted from 1) in which a row's maximum may move
};

// A set's tiles [lo, hi) (counted from its own first): its rows' part of the softmax.
template <int D, int RT, int SEEN, int CODE>
__device__ __forceinline__ void rows_run(const AttnArgs& a, const Set& set, int h, int rb, int lo, int hi, int entry,
                                         const Out& out, RowsLds<D, RT>& lds) {
  using F = RowsFormat<CODE>;
  constexpr int KS = D / 32;                       // operands of a key
  constexpr int HALVES = F::CODED ? 2 : 1;         // in 16 bytes
  constexpr int KL = KS / HALVES;                  // loads of a key
  constexpr int DL = D / 64;                       // 16 dimensions each, of a wave
  constexpr int VL = F::CODED ? 1 : 2;             // loads of their values: 16 positions or 8 in 16 bytes
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.group;
  const Rows<SEEN> rows(a, set.seq, set.token, rb);
  if (rows.first >= rows.count) return;
  Tiles<D, SEEN, F> tiles(a, set, h, rows, lane, lo, hi, 0, 1, entry);

  const uint32_t k_lane = ((uint32_t)(lg << a.c.shift) + 16 * w + li) * 16;
  const uint32_t k_step = 4u << a.c.shift << 4;  // 4 groups of dimensions on
  const uint32_t v_lane = (uint32_t)(lg * D + 16 * DL * w + li) * 16;
  uint4 kf[KL], vf[DL][VL];
  f32x4 ks = {1.f, 1.f, 1.f, 1.f}, vs_next = ks;  // codes: scales of the lane's 4 positions
  // No branch around the loads of the next tile, so that each wait counts those behind it exactly: past the last tile it
  // is loaded again, and not waited for.
  const auto load_keys = [&] {
    if constexpr (F::CODED) {  // ahead of the keys: the wait for those covers both
      const int at = 16 * w + 4 * lg;
      ks = ld4(a.code.k_scales + tiles.scales + at);
      vs_next = ld4(a.code.v_scales + tiles.scales + at);
    }
#pragma unroll
    for (int k = 0; k < KL; ++k) kf[k] = ld16(tiles.kp + k * k_step + k_lane);
  };
  const auto load_values = [&] {
#pragma unroll
    for (int d = 0; d < DL; ++d) {
#pragma unroll
      for (int u = 0; u < VL; ++u) vf[d][u] = ld16(tiles.vp + v_lane + (64 * u * D + 256 * d));
    }
  };

  const auto row_reach = [&](int m) {
    const int len = lds.len[16 * m + li];
    return Reach{SEEN == WINDOW ? len - a.window.size : 0, len, SEEN == WINDOW ? a.window.first : 0};
  };
  // The query rows are on their way beside the table's entries, and go into LDS behind the first tile's loads: a run
  // begins after two trips to memory, however many its rows.
  constexpr int QL = (KS + ROWS_WAVES - 1) / ROWS_WAVES;  // a wave takes the operands w, w + 4, ...
  uint4 query[RT][QL];
#pragma unroll
  for (int m = 0; m < RT; ++m) {
    const int r = min(rows.first + 16 * m + li, rows.count - 1);  // behind the last row the last one again, not stored
    const int t = SEEN == LISTED ? set.token : r / G, g = SEEN == LISTED ? r : r % G;
    const int rid = (set.seq.row + t) * a.heads + h * G + g;
    if (w == 0 && lg == 0) {
      lds.len[16 * m + li] = set.seq.first + t + 1;
      lds.rid[16 * m + li] = rows.first + 16 * m + li < rows.count ? rid : -1;
    }
#pragma unroll
    for (int j = 0; j < QL; ++j) {
      const int k = min(ROWS_WAVES * j + w, KS - 1);
      query[m][j] = ld16(a.q + (size_t)rid * D + (F::CODED ? 16 * lg + 64 * (k / 2) + 8 * (k % 2) : 8 * lg + 32 * k));
    }
  }

  // A scale below zero turns the query rows' signs: the largest product is the largest exponent.
  const uint32_t turn = a.scale_hi < 0.f ? 0x80008000u : 0u;
  const float scale_hi = fabsf(a.scale_hi), scale_lo = fabsf(a.scale_lo);
  f32x4 acc[RT][DL];
  float mx[RT], sum[RT];
#pragma unroll
  for (int m = 0; m < RT; ++m) {
    mx[m] = -FLT_MAX;
    sum[m] = 0.f;
#pragma unroll
    for (int d = 0; d < DL; ++d) acc[m][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  if (w == 0 && lane == 0) lds.risen = 0;
  __builtin_amdgcn_sched_barrier(0);
  bool more = tiles.find();
  loads_done();
  if (more) {
    load_keys();
    load_values();
  }
#pragma unroll
  for (int m = 0; m < RT; ++m) {
#pragma unroll
    for (int j = 0; j < QL; ++j) {
      const int k = ROWS_WAVES * j + w;
      const uint4& u = query[m][j];
      if (KS % ROWS_WAVES == 0 || k < KS)
        lds.q[m][k][lane] = make_uint4(u.x ^ turn, u.y ^ turn, u.z ^ turn, u.w ^ turn);
    }
  }
  lds_barrier();

  for (int count = 1; more; ++count) {
    const int now = tiles.p0;
    const bool whole = rows.all_see(a, now, F::TILE);
    f32x4 s[RT];
#pragma unroll
    for (int m = 0; m < RT; ++m) s[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    // query operands are read from LDS AHEAD steps before their products (the compiler would read each just before)
    constexpr int AHEAD = KS < 3 || D == 256 || RT == 4 ? 1 : 2;
    uint4 qk[AHEAD + 1][RT];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
#pragma unroll
      for (int m = 0; m < RT; ++m) qk[k][m] = lds.q[m][k][lane];
    }
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      if (k + AHEAD < KS) {
#pragma unroll
        for (int m = 0; m < RT; ++m) qk[(k + AHEAD) % (AHEAD + 1)][m] = lds.q[m][k + AHEAD][lane];
      }
      __builtin_amdgcn_sched_barrier(0);
      const uint4 key = operand<CODE>(kf[k / HALVES], k % HALVES);
#pragma unroll
      for (int m = 0; m < RT; ++m) s[m] = mfma(key, qk[k % (AHEAD + 1)][m], s[m]);
      __builtin_amdgcn_sched_barrier(0);
    }
    const f32x4 ks_now = ks, vs = vs_next;
    __builtin_amdgcn_sched_barrier(0);
    more = tiles.find();
    load_keys();
    __builtin_amdgcn_sched_barrier(0);

    const int mine = now + 16 * w + 4 * lg;  // the position of the lane's first product
    float v[RT][4], largest[RT];
    bool rises = false;
#pragma unroll
    for (int m = 0; m < RT; ++m) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[m][i] = F::CODED ? s[m][i] * ks_now[i] : s[m][i];
      if (!whole) hide(v[m], row_reach(m).template bits<4>(mine), scale_hi);
      largest[m] = fmaxf(fmaxf(v[m][0], v[m][1]), fmaxf(v[m][2], v[m][3])) * scale_hi;
      rises |= largest[m] > mx[m] + 8.f;
    }
    // Maxima move in the first tile and rarely behind it: only then are they taken over lanes and waves (64 rows of D = 64
    // over 200,000 positions 117 -> 110 us).  Through a window always: runs are short, and prompts were slower (87 -> 89).
    bool risen = SEEN == WINDOW || count == 1;
    if (!risen) {
      if (__any(rises) && lane == 0) lds.risen = count;
      lds_barrier();
      risen = __builtin_amdgcn_readfirstlane(lds.risen) == count;
    }
    if (risen) {
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        const float top = rows_max(largest[m]);
        if (lg == 0) reinterpret_cast<float*>(&lds.tops[16 * m + li])[w] = top;
      }
      lds_barrier();
      f32x4 tops[RT];
#pragma unroll
      for (int m = 0; m < RT; ++m) tops[m] = lds.tops[16 * m + li];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        const float top = fmaxf(fmaxf(tops[m][0], tops[m][1]), fmaxf(tops[m][2], tops[m][3]));
        if (__any(top > mx[m] + 8.f)) {
          const float high = top > mx[m] + 8.f ? top : mx[m];  // a row's own: no row feels another's
          const float f = exp2_of(mx[m] - high);
          mx[m] = high;
          sum[m] *= f;
#pragma unroll
          for (int d = 0; d < DL; ++d) acc[m][d] *= f;
        }
      }
    }
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      f32x4 p;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        p[i] = exp2_of(__builtin_fmaf(v[m][i], scale_lo, __builtin_fmaf(v[m][i], scale_hi, -mx[m])));
      sum[m] += (p[0] + p[1]) + (p[2] + p[3]);
      if constexpr (F::CODED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] *= vs[i];
        if (!whole) {  // a scale that the row does not see may be anything
          const uint32_t seen = row_reach(m).template bits<4>(mine);
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = __uint_as_float(__float_as_uint(p[i]) & bit_mask(seen, i));
        }
      }
      uint2 hi, low;
      split_hi_lo4(p, hi, low);
      uint2* to = reinterpret_cast<uint2*>(&lds.p[0][m][w][lg >> 1][li]) + (lg & 1);
      constexpr int PART = RT * 4 * 2 * 16 * 2;  // of uint2
      to[0] = hi;
      to[PART] = low;
      if (a.out_type == HCR_F32) to[2 * PART] = split_rest4(p, hi, low);
    }

    // A value that is no number and that only some of the rows see leaves the product, and its dimension of the rows
    // that see it becomes NaN (as in hcr_attn_device.h)
    if constexpr (CODE != HCR_INT8) {
      if (!whole) {
        const Reach any{rows.start_min, rows.len_max, a.window.first}, all{rows.start_max, rows.len_min, a.window.first};
        const f32x4 none = {0.f, 0.f, 0.f, 0.f};
        const auto spoil = [&](int d, int p, const uint4& at) {  // at: ones where 8 values from p on were dropped
#pragma unroll
          for (int m = 0; m < RT; ++m) {
            const f32x4 met = mfma(at, ones8(row_reach(m).template bits<8>(p)), none);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][d][i] = met[i] > 0.f ? NAN : acc[m][d][i];
          }
          __builtin_amdgcn_sched_barrier(0);
        };
        if constexpr (CODE == HCR_BF16) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int p = now + 32 * u + 8 * lg;
            const uint32_t seen = any.bits<8>(p), common = all.bits<8>(p);
            uint4 of[DL];
#pragma unroll
            for (int d = 0; d < DL; ++d) of[d] = vf[d][u] = masked8(vf[d][u], seen);
            if (any_odd(of)) {
#pragma unroll
              for (int d = 0; d < DL; ++d) spoil(d, p, drop_odd_but(vf[d][u], common));
            }
          }
        } else {
          uint32_t hit = 0;
#pragma unroll
          for (int d = 0; d < DL; ++d)
            hit |= odd_codes(vf[d][0].x) | odd_codes(vf[d][0].y) | odd_codes(vf[d][0].z) | odd_codes(vf[d][0].w);
          if (__any(hit != 0)) {
            const int p = now + 16 * lg;
            const uint32_t common = all.bits<16>(p);
#pragma unroll
            for (int d = 0; d < DL; ++d) {
              const uint4 low = drop_odd_codes(vf[d][0].x, vf[d][0].y, common & 0xFFu);
              const uint4 high = drop_odd_codes(vf[d][0].z, vf[d][0].w, common >> 8);
              spoil(d, p, low);
              spoil(d, p + 8, high);
            }
          }
        }
      }
    }

    // the values' operands; codes are widened ahead of the barrier, and the next ones' loads go out at once
    uint4 value[2][DL];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int d = 0; d < DL; ++d) value[u][d] = F::CODED ? operand<CODE>(vf[d][0], u) : vf[d][VL == 2 ? u : 0];
    }
    constexpr bool EARLY = F::CODED && D != 256;
    if constexpr (EARLY) {
      __builtin_amdgcn_sched_barrier(0);
      load_values();
      __builtin_amdgcn_sched_barrier(0);
    }
    lds_barrier();
    // the 8 positions of the lane's values in operand u: of codes 8 (u) of wave lg's 16, of BF16 32 u + 8 lg and on
    const auto part = [&](int i, int u, int m) {
      return F::CODED ? lds.p[i][m][lg][u][li] : lds.p[i][m][2 * u + (lg >> 1)][lg & 1][li];
    };
    // the parts of a row tile are read two steps ahead of their products; the third ones for float outputs alone
    const auto products = [&](auto first, auto steps) {
      uint4 ps[3];
      const auto read = [&](int g) { ps[g % 3] = part(first + g / (2 * RT), g / RT & 1, g % RT); };
      read(0);
      read(1);
#pragma unroll
      for (int g = 0; g < steps; ++g) {
        if (g + 2 < steps) read(g + 2);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = 0; d < DL; ++d) acc[g % RT][d] = mfma(value[g / RT & 1][d], ps[g % 3], acc[g % RT][d]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    products(std::integral_constant<int, 0>{}, std::integral_constant<int, 4 * RT>{});
    if (a.out_type == HCR_F32) products(std::integral_constant<int, 2>{}, std::integral_constant<int, 2 * RT>{});
    if constexpr (!EARLY) {
      __builtin_amdgcn_sched_barrier(0);
      load_values();
      __builtin_amdgcn_sched_barrier(0);
    }
  }

#pragma unroll
  for (int m = 0; m < RT; ++m) {
    sum[m] = rows_sum(sum[m]);
    if (lg == 0) reinterpret_cast<float*>(&lds.sums[16 * m + li])[w] = sum[m];
  }
  lds_barrier();
#pragma unroll
  for (int m = 0; m < RT; ++m) {
    const f32x4 sums = lds.sums[16 * m + li];
    const float total = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    const int rid = lds.rid[16 * m + li];
    if (rid < 0) continue;
#pragma unroll
    for (int d = 0; d < DL; ++d)
      out.values(D, rid, 16 * m + li, 16 * (DL * w + d) + 4 * lg, acc[m][d], total);
    if (w == 0 && lg == 0) out.state(D, 16 * m + li, mx[m], total);
  }
}

template <int D, int RT, int SEEN, int CODE, bool PAIRED>
__global__ __launch_bounds__(64 * ROWS_WAVES, rows_held(D, RT)) void attn_rows_part(AttnArgs a) {
  __shared__ RowsLds<D, RT> lds;
  arguments_near(a);
  part_of<ROWS_SHIFT, SEEN, PAIRED>(a, [&](const Set& set, int h, int rb, int lo, int hi, int entry, const Out& out) {
    rows_run<D, RT, SEEN, CODE>(a, set, h, rb, lo, hi, entry, out, lds);
  });
}

}  // namespace hcr
