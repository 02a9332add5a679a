// Attention of a decode window over the paged cache, gfx950 (MI355X):
//   out[n] = sum_p softmax_p(scale q[n] . k[p]) v[p],   p <= the token's position
// for every page of a sequence, or for the pages listed per token and kv head.
//
// A unit is one kv head of one sequence: its rows are the T x G (tokens x heads of the group) query rows, which
// all read the same keys and values.  A wave takes tiles of 32 positions and holds 16, 32 or 64 of the rows:
//   S^T = K Q^T : A = 16 keys (two row tiles per 32 positions), B = 16 query rows; S^T arrives with one query row
//                 per lane column, so a row's maximum and sum run over a lane's 8 values and the 4 lane rows.
//   O^T += V^T P^T : the K index of this product is a position.  Row r of key tile t is position
//                 8 (r / 4) + 4 t + r % 4, so the 8 probabilities that a lane holds after S^T are 8 consecutive
//                 positions, its B operand as they are; the value pages keep 8 positions of a dimension in 16
//                 bytes, its A operand as loaded.  Nothing goes through LDS inside the loop.
// Probabilities are powers of two against a running maximum that moves only when a tile passes it by 2^8 (sums
// and products are FP32, so the offset costs no precision), split into BF16 parts: two (2^-17) for BF16 outputs,
// three (the whole FP32 value) for float ones, where two would be the largest error of all (1.1e-6 of the result's
// norm instead of 1.5e-7; the third costs matrix products that the loop has time for).
//
// The length is split over work-groups and their waves; waves join in LDS, splits in a second launch, each by
// (m, l, O) -> (max, sum of l 2^(m - max), sum of O 2^(m - max)), in a fixed order.

#include <float.h>
#include <hip/hip_runtime.h>

#include "hcr_device.h"
#include "hcr_paged_layout.h"

namespace hcr {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;

__device__ __forceinline__ bf16x8 as_bf16x8(const uint4& u) { return __builtin_bit_cast(bf16x8, u); }
__device__ __forceinline__ uint4 ld16(const void* p) { return *static_cast<const uint4*>(p); }
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// The larger of each value over the 4 lane rows (lanes l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float rows_max(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float rows_sum(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// What the high and low BF16 parts of 8 values leave of them, as BF16.
__device__ __forceinline__ uint4 split_rest(const float (&v)[8], const uint4& hi, const uint4& lo) {
  const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
  uint32_t r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f32x2 x = {v[2 * e], v[2 * e + 1]};
    x -= f32x2{__uint_as_float(h[e] << 16), __uint_as_float(h[e] & 0xFFFF0000u)};  // exact, twice
    x -= f32x2{__uint_as_float(l[e] << 16), __uint_as_float(l[e] & 0xFFFF0000u)};
    r[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ void store4(void* out, int type, size_t at, const f32x4& v) {
  if (type == HCR_F32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(out) + at) = v;
  } else {
    const f32x2 a = {v[0], v[1]}, b = {v[2], v[3]};
    uint2 u;
    u.x = __builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2));
    u.y = __builtin_bit_cast(uint32_t, __builtin_convertvector(b, bf16x2));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = u;
  }
}

template <int D, int MT, bool SEL>
__global__ __launch_bounds__(64 * ATTN_WAVES) void attn_part(AttnArgs a) {
  constexpr int KS = D / 32, DT = D / 16, W = ATTN_WAVES;
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // work-group -> (split, sequence[, token], kv head, row block); the row blocks of one unit run on one XCD (its
  // L2 then serves all but the first), the first splits, which every sequence has, come first
  const int RB = a.plan.row_blocks;
  const int turn = blockIdx.x / XCDS;
  const int rb = turn % RB;
  int u = turn / RB * XCDS + blockIdx.x % XCDS;
  const int windows = SEL ? a.b.max_tokens : 1;
  if (u >= a.plan.splits * a.b.n_seqs * windows * a.c.kv_heads) return;
  const int h = u % a.c.kv_heads;
  u /= a.c.kv_heads;
  const int token = SEL ? u % windows : 0;
  u /= windows;
  const int b = u % a.b.n_seqs;
  const int split = u / a.b.n_seqs;

  const Seq seq = seq_of(a.b, a.b.q_start[b], a.b.q_start[b + 1], a.b.ctx_len[b]);
  const int G = a.group;
  const int rows = SEL ? (token < seq.tokens ? G : 0) : seq.tokens * G;
  const int r0 = rb * 16 * MT;
  if (r0 >= rows) return;
  const int r_last = min(r0 + 16 * MT, rows) - 1;
  // positions a row sees: [0, len)
  const int len_max = seq.first + (SEL ? token : r_last / G) + 1;
  const int len_min = seq.first + (SEL ? token : r0 / G) + 1;
  const int psh = a.c.shift - TILE_SHIFT;
  const int tiles = SEL ? a.n_sel << psh : ceil_div(max(len_max, 0), TILE);
  const int lo = split * a.plan.chunk, hi = min(lo + a.plan.chunk, tiles);
  if (lo >= hi && a.plan.splits > 1) return;  // not joined

  // the lane's query row of each 16-row tile, its operand and its length
  uint4 qf[MT][KS];
  int len[MT];
  size_t rid[MT];
  bool live[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = r0 + 16 * m + li;
    live[m] = r < rows;
    const int rr = min(r, rows - 1);
    const int t = SEL ? token : rr / G, g = SEL ? rr : rr % G;
    len[m] = seq.first + t + 1;
    rid[m] = (size_t)(seq.row + t) * a.heads + h * G + g;
    const uint16_t* qp = a.q + rid[m] * D + 8 * lg;
#pragma unroll
    for (int k = 0; k < KS; ++k) qf[m][k] = ld16(qp + 32 * k);
  }

  f32x4 acc[MT][DT];
  float mx[MT], sum[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    mx[m] = -FLT_MAX;
    sum[m] = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[m][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const int page = 1 << a.c.shift;
  const int key_row = 8 * (li >> 2) + (li & 3);  // position of key tile 0's row li
  for (int pb = lo >> psh; pb << psh < hi; pb += 64) {
    // lane l: page pb + l of the list, as the page's number (-1: none) and its index in the sequence
    const int idx = pb + lane;
    int index = -1, number = -1;
    if (SEL) {
      if (idx < a.n_sel) index = a.sel[((size_t)(seq.row + token) * a.c.kv_heads + h) * a.n_sel + idx];
      if (index >= 0 && index <= (len_max - 1) >> a.c.shift && len_max > 0)
        number = page_or_none(a.b.table[(size_t)b * a.b.table_stride + index], a.c.n_pages);
    } else {
      index = idx;
      if (idx << psh < tiles) number = page_or_none(a.b.table[(size_t)b * a.b.table_stride + idx], a.c.n_pages);
    }
    const int end = min(hi, (pb + 64) << psh);
    int tile = max(lo, pb << psh);
    tile += (wave - (tile - lo)) & (W - 1);  // this wave's: lo + wave, + W, ...
    for (; tile < end; tile += W) {
      const int at = (tile >> psh) - pb;
      const int pn = __builtin_amdgcn_readlane(number, at);
      if (pn < 0) continue;
      const int off = (tile << TILE_SHIFT) & (page - 1);
      const int p0 = (__builtin_amdgcn_readlane(index, at) << a.c.shift) + off;
      if (p0 >= len_max) continue;
      const size_t base = head_base(a.c, pn, h);
      const uint16_t* kp = a.c.k + base + ((size_t)(lg << a.c.shift) + off + key_row) * 8;
      const uint16_t* vp = a.c.v + base + ((size_t)((off >> 3) + lg) * D + li) * 8;
      uint4 kf[2][KS], vf[DT];
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        kf[0][k] = ld16(kp + ((size_t)(4 * k) << a.c.shift) * 8);
        kf[1][k] = ld16(kp + ((size_t)(4 * k) << a.c.shift) * 8 + 4 * 8);
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) vf[d] = ld16(vp + 16 * 8 * d);

      const bool whole = p0 + TILE <= len_min;
      if (!whole) {
        // values behind the last visible position may be anything: zeros in their place (their
        // probabilities are zero, but zero times NaN is not)
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          uint32_t w[4] = {vf[d].x, vf[d].y, vf[d].z, vf[d].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int p = p0 + 8 * lg + 2 * e;
            w[e] = p + 1 < len_max ? w[e] : p < len_max ? w[e] & 0xFFFFu : 0u;
          }
          vf[d] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }

#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float s[8], y[8];  // products, and as exponents of two
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < KS; ++k)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(kf[t][k]), as_bf16x8(qf[m][k]), c, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[4 * t + i] = c[i];
            y[4 * t + i] = c[i] * a.scale_hi;
          }
        }
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = p0 + 8 * lg + i < len[m] ? y[i] : -INFINITY;
        }
        float top = fmaxf(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), fmaxf(fmaxf(y[4], y[5]), fmaxf(y[6], y[7])));
        top = rows_max(top);
        if (__any(top > mx[m] + 8.f)) {
          const float now = fmaxf(mx[m], top);
          const float f = exp2_of(mx[m] - now);
          mx[m] = now;
          sum[m] *= f;
#pragma unroll
          for (int d = 0; d < DT; ++d) acc[m][d] *= f;
        }
        // exponents with the scale in two parts: one rounding, of the difference from the maximum
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          p[i] = exp2_of(__builtin_fmaf(s[i], a.scale_hi, __builtin_fmaf(s[i], a.scale_lo, -mx[m])));
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = p0 + 8 * lg + i < len[m] ? p[i] : 0.f;
        }
        sum[m] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
        uint4 ph, pl;
        split_hi_lo(p, ph, pl);
#pragma unroll
        for (int d = 0; d < DT; ++d)
          acc[m][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(vf[d]), as_bf16x8(ph), acc[m][d], 0, 0, 0);
#pragma unroll
        for (int d = 0; d < DT; ++d)
          acc[m][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(vf[d]), as_bf16x8(pl), acc[m][d], 0, 0, 0);
        if (a.out_type == HCR_F32) {
          const uint4 pr = split_rest(p, ph, pl);
#pragma unroll
          for (int d = 0; d < DT; ++d)
            acc[m][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(vf[d]), as_bf16x8(pr), acc[m][d], 0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) sum[m] = rows_sum(sum[m]);

  // the waves joined by halves: the upper half writes, the lower half adds
  __shared__ f32x4 lds_acc[W / 2][MT * DT][64];
  __shared__ float lds_ml[W / 2][MT][2][64];
#pragma unroll
  for (int half = W / 2; half >= 1; half /= 2) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        lds_ml[wave - half][m][0][lane] = mx[m];
        lds_ml[wave - half][m][1][lane] = sum[m];
#pragma unroll
        for (int d = 0; d < DT; ++d) lds_acc[wave - half][m * DT + d][lane] = acc[m][d];
      }
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float m2 = lds_ml[wave][m][0][lane], l2 = lds_ml[wave][m][1][lane];
        const float now = fmaxf(mx[m], m2);
        const float f1 = exp2_of(mx[m] - now), f2 = exp2_of(m2 - now);
        mx[m] = now;
        sum[m] = sum[m] * f1 + l2 * f2;
#pragma unroll
        for (int d = 0; d < DT; ++d) acc[m][d] = acc[m][d] * f1 + lds_acc[wave][m * DT + d][lane] * f2;
      }
    }
    __syncthreads();
  }
  if (wave != 0) return;

  const size_t all = (size_t)a.b.n_tokens * a.heads;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (!live[m]) continue;
    if (a.plan.splits == 1) {
      const float f = sum[m] > 0.f ? 1.f / sum[m] : 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) store4(a.out, a.out_type, rid[m] * D + 16 * d + 4 * lg, acc[m][d] * f);
    } else {
      const size_t at = rid[m] * a.plan.splits + split;
#pragma unroll
      for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4*>(a.part + at * D + 16 * d + 4 * lg) = acc[m][d];
      if (lg == 0) *reinterpret_cast<f32x2*>(a.part + all * a.plan.splits * D + at * 2) = f32x2{mx[m], sum[m]};
    }
  }
}

// One row's splits joined: D / 4 lanes hold a row of 4 values each, the groups of lanes take the splits in turn
// and join in LDS, in a fixed order.
template <int D, bool SEL>
__global__ __launch_bounds__(256) void attn_join(AttnArgs a) {
  constexpr int LANES = D / 4, GROUPS = 256 / LANES;
  const int l = threadIdx.x % LANES, grp = threadIdx.x / LANES;
  const int hq = blockIdx.x % a.heads, bt = blockIdx.x / a.heads;
  const int t = bt % a.b.max_tokens, b = bt / a.b.max_tokens;
  const Seq seq = seq_of(a.b, a.b.q_start[b], a.b.q_start[b + 1], a.b.ctx_len[b]);
  if (t >= seq.tokens) return;
  const size_t rid = (size_t)(seq.row + t) * a.heads + hq;
  const size_t all = (size_t)a.b.n_tokens * a.heads;
  const int len = max(seq.first + t + 1, 0);
  const int n = SEL ? a.plan.splits : min(a.plan.splits, ceil_div(ceil_div(len, TILE), a.plan.chunk));
  const float* ml = a.part + all * a.plan.splits * D + rid * a.plan.splits * 2;
  const float* pa = a.part + rid * a.plan.splits * D + 4 * l;
  float mx = -FLT_MAX, sum = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = grp; s < n; s += GROUPS) {
    const f32x2 v = ld2(ml + 2 * s);
    const f32x4 o = ld4(pa + (size_t)s * D);
    const float now = fmaxf(mx, v[0]);
    const float f1 = exp2_of(mx - now), f2 = exp2_of(v[0] - now);
    mx = now;
    sum = sum * f1 + v[1] * f2;
    acc = acc * f1 + o * f2;
  }
  __shared__ f32x4 lds_acc[256];
  __shared__ f32x2 lds_ml[GROUPS];
  lds_acc[threadIdx.x] = acc;
  if (l == 0) lds_ml[grp] = f32x2{mx, sum};
  __syncthreads();
  if (grp != 0) return;
  float top = -FLT_MAX;
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) top = fmaxf(top, lds_ml[g][0]);
  sum = 0.f;
  acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    const float f = exp2_of(lds_ml[g][0] - top);
    sum += lds_ml[g][1] * f;
    acc += lds_acc[g * LANES + l] * f;
  }
  const float f = sum > 0.f ? 1.f / sum : 0.f;
  store4(a.out, a.out_type, rid * D + 4 * l, acc * f);
}

namespace {

template <int D, int MT, bool SEL>
void run_part(const AttnArgs& a, int grid, hipStream_t st) {
  hipLaunchKernelGGL((attn_part<D, MT, SEL>), dim3(grid), dim3(64 * ATTN_WAVES), 0, st, a);
}
template <int D, bool SEL>
void run_part_rows(const AttnArgs& a, int grid, hipStream_t st) {
  if (a.plan.q_tiles == 1) return run_part<D, 1, SEL>(a, grid, st);
  if (D == 256 || a.plan.q_tiles == 2) return run_part<D, 2, SEL>(a, grid, st);
  if constexpr (D != 256) return run_part<D, 4, SEL>(a, grid, st);
}
template <bool SEL>
void run_attn(const AttnArgs& a, int grid, int join_grid, hipStream_t st) {
  const bool join = a.plan.splits > 1;
  switch (a.c.head_dim) {
    case 64:
      run_part_rows<64, SEL>(a, grid, st);
      if (join) hipLaunchKernelGGL((attn_join<64, SEL>), dim3(join_grid), dim3(256), 0, st, a);
      break;
    case 128:
      run_part_rows<128, SEL>(a, grid, st);
      if (join) hipLaunchKernelGGL((attn_join<128, SEL>), dim3(join_grid), dim3(256), 0, st, a);
      break;
    default:
      run_part_rows<256, SEL>(a, grid, st);
      if (join) hipLaunchKernelGGL((attn_join<256, SEL>), dim3(join_grid), dim3(256), 0, st, a);
  }
}

}  // namespace

int launch_attn(const AttnArgs& a, void* stream) {
  const AttnPlan& p = a.plan;
  const int units = p.splits * a.b.n_seqs * (a.sel ? a.b.max_tokens : 1) * a.c.kv_heads;
  const int grid = ceil_div(units, XCDS) * XCDS * p.row_blocks;
  const int join_grid = a.b.n_seqs * a.b.max_tokens * a.heads;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (a.sel)
    run_attn<true>(a, grid, join_grid, st);
  else
    run_attn<false>(a, grid, join_grid, st);
  return hipGetLastError() == hipSuccess ? HCR_OK : HCR_EHIP;
}

}  // namespace hcr
