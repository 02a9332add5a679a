// Append of a decode window to the paged cache, gfx950 (MI355X): per head, y = x w / sqrt(mean(x^2) + eps), the
// first rope_dim values rotated by the angles of the token's position, rounded once to BF16; q to its rows, k and
// v into the pages, and the mean key of each page that the window completes.
//
// One launch.  A lane holds 4 consecutive dimensions, D / 4 lanes a head: the sum of squares is a butterfly inside
// a row of 16 lanes and one or two row swaps; the partner of a rotated value (j, j + r/2) sits in another lane at
// the same place, that of (2j, 2j + 1) in the same lane.  The first work-groups take (sequence, page, kv head, k or
// v): the page's new tokens are staged in LDS, 64 slots at a time, and written in the page's order, so that a
// prompt's pages go out as whole lines (a lane writes 8 dimensions of a slot, or 8 slots of a dimension).  The
// others take query heads.  Nothing bounds it but the bytes of the rows, and for a few tokens the launch itself.

#include <hip/hip_runtime.h>

#include "hcr_device.h"
#include "hcr_paged_layout.h"

namespace hcr {

constexpr int APPEND_THREADS = 256;
constexpr int SLOTS = 64;  // slots of a page staged at a time

// 4 consecutive values of a row
template <bool F32>
__device__ __forceinline__ f32x4 load4(const void* p, size_t at) {
  if constexpr (F32) {
    return ld4(static_cast<const float*>(p) + at);
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
    return f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                 __uint_as_float(u.y & 0xFFFF0000u)};
  }
}
__device__ __forceinline__ uint2 round4(const f32x4& v) {
  const f32x2 a = {v[0], v[1]}, b = {v[2], v[3]};
  return make_uint2(__builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2)),
                    __builtin_bit_cast(uint32_t, __builtin_convertvector(b, bf16x2)));
}

// The sum over the LANES (16, 32 or 64) lanes of a head, in every one of them.
template <int LANES>
__device__ __forceinline__ float head_sum(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  if constexpr (LANES >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (LANES == 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// Norm and rotation of a head's values 4 l .. 4 l + 3 at position pos (every lane of the wave takes part).
template <int D>
__device__ __forceinline__ f32x4 norm_rotate(f32x4 x, const float* w, const AppendArgs& a, int l, int pos) {
  constexpr int LANES = D / 4;
  if (w) {
    const float ss = head_sum<LANES>((x[0] * x[0] + x[1] * x[1]) + (x[2] * x[2] + x[3] * x[3]));
    const float rs = 1.f / sqrtf(ss * (1.f / D) + a.eps);
    x = x * rs * ld4(w + 4 * l);
  }
  if (a.rope_dim) {
    const float* row = a.rope + (size_t)pos * a.rope_dim;
    const int half = a.rope_dim >> 1;
    const bool in = 4 * l < a.rope_dim;
    if (a.rope_style == HCR_ROPE_PAIRS) {
      if (in) {
        const f32x2 c = ld2(row + 2 * l), s = ld2(row + half + 2 * l);
        x = f32x4{x[0] * c[0] - x[1] * s[0], x[1] * c[0] + x[0] * s[0], x[2] * c[1] - x[3] * s[1],
                  x[3] * c[1] + x[2] * s[1]};
      }
    } else {
      const bool low = 4 * l < half;
      const int from = (threadIdx.x & 63) + (in ? (low ? half >> 2 : -(half >> 2)) : 0);
      f32x4 y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = __shfl(x[e], from);
      if (in) {
        const int j = low ? 4 * l : 4 * l - half;
        const f32x4 c = ld4(row + j), s = ld4(row + half + j);
        x = low ? x * c - y * s : x * c + y * s;
      }
    }
  }
  return x;
}

// The new tokens of one page of one kv head: staged, written in the page's order, the mean key where complete.
template <int D, bool F32>
__device__ void append_page(const AppendArgs& a, const Seq& seq, int b, int pg, int h, bool key) {
  constexpr int LANES = D / 4, PER = APPEND_THREADS / LANES;  // tokens of a pass
  constexpr int ROW = D + 8;                                  // 16 bytes more: slots start in other banks
  constexpr int C = D / 8;                                    // 16-byte chunks of a slot
  __shared__ uint16_t tile[SLOTS * ROW];
  const int page = 1 << a.c.shift, tid = threadIdx.x;
  const int ctx = seq.first + seq.tokens;
  const int start = pg << a.c.shift;
  const int lo = max(max(seq.first, 0), start) - start, hi = min(ctx - start, page);  // new slots
  if (lo >= hi) return;
  const int number = page_or_none(a.b.table[(size_t)b * a.b.table_stride + pg], a.c.n_pages);
  if (number < 0) return;
  uint16_t* out = (key ? a.c.k : a.c.v) + head_base(a.c, number, h);
  const hcr_rows rows = key ? a.k : a.v;
  const bool mean = key && a.c.means && hi == page;
  const int l = tid % LANES, sub = tid / LANES;
  const int mc = tid % C, mg = tid / C;  // for the mean: chunk, and slots mg, mg + groups, ...
  constexpr int MG = APPEND_THREADS / C;
  float total[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};

  for (int base = mean ? 0 : lo / SLOTS * SLOTS; base < hi; base += SLOTS) {
    const int s0 = max(lo, base), s1 = min(hi, base + SLOTS);  // new slots of this part (s0 >= s1: none)
    for (int s = s0; s < s1; s += PER) {
      const int slot = min(s + sub, s1 - 1);  // past the end: the last one again, for the wave's sums
      const int pos = start + slot;
      const size_t at = (size_t)(seq.row + pos - seq.first) * rows.token_stride + (size_t)h * rows.head_stride + 4 * l;
      f32x4 x = load4<F32>(rows.data, at);
      if (key) x = norm_rotate<D>(x, a.k_norm, a, l, pos);
      if (s + sub < s1) *reinterpret_cast<uint2*>(&tile[(slot - base) * ROW + 4 * l]) = round4(x);
    }
    __syncthreads();
    if (key) {
      const int n = max(s1 - s0, 0);
      for (int i = tid; i < n * C; i += APPEND_THREADS) {
        const int c = i / n, slot = s0 + i % n;
        *reinterpret_cast<uint4*>(out + k_at(a.c.shift, slot, 8 * c)) =
            *reinterpret_cast<const uint4*>(&tile[(slot - base) * ROW + 8 * c]);
      }
      if (mean) {
        for (int slot = base + mg; slot < min(base + SLOTS, page); slot += MG) {
          const uint4 u = slot >= lo ? *reinterpret_cast<const uint4*>(&tile[(slot - base) * ROW + 8 * mc])
                                     : *reinterpret_cast<const uint4*>(out + k_at(a.c.shift, slot, 8 * mc));
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            total[2 * e] += __uint_as_float(w[e] << 16);
            total[2 * e + 1] += __uint_as_float(w[e] & 0xFFFF0000u);
          }
        }
      }
    } else if (s0 < s1) {
      const int o0 = s0 >> 3, n = ((s1 - 1) >> 3) - o0 + 1;  // octets of slots
      for (int i = tid; i < n * D; i += APPEND_THREADS) {
        const int o = o0 + i / D, d = i % D;
        uint16_t* to = out + v_at(D, 8 * o, d);
        if (8 * o >= s0 && 8 * o + 8 <= s1) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = tile[(8 * o + 2 * e - base) * ROW + d] | (uint32_t)tile[(8 * o + 2 * e + 1 - base) * ROW + d] << 16;
          *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          for (int s = max(8 * o, s0); s < min(8 * o + 8, s1); ++s) to[s & 7] = tile[(s - base) * ROW + d];
        }
      }
    }
    __syncthreads();
  }

  if (mean) {
    float* part = reinterpret_cast<float*>(tile);  // [MG][D]
    static_assert(MG * D * 4 <= (int)sizeof(tile), "the mean's partial sums fit the tile");
#pragma unroll
    for (int e = 0; e < 8; ++e) part[mg * D + 8 * mc + e] = total[e];
    __syncthreads();
    if (tid < D) {
      float m = 0.f;
#pragma unroll
      for (int g = 0; g < MG; ++g) m += part[g * D + tid];
      const f32x2 v = {m / page, 0.f};
      a.c.means[((size_t)number * a.c.kv_heads + h) * D + tid] =
          (uint16_t)__builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    }
  }
}

template <int D, bool F32>
__global__ __launch_bounds__(APPEND_THREADS) void append(AppendArgs a, int kv_groups, int pages, int passes,
                                                         int tokens_each) {
  constexpr int LANES = D / 4, PER = APPEND_THREADS / LANES;
  int g = blockIdx.x;
  if (g < kv_groups) {
    const bool key = g & 1;
    g >>= 1;
    const int h = g % a.c.kv_heads;
    g /= a.c.kv_heads;
    const int b = g / pages;
    const Seq seq = seq_of(a.b, a.b.q_start[b], a.b.q_start[b + 1], a.b.ctx_len[b]);
    const int pg = (max(seq.first, 0) >> a.c.shift) + g % pages;
    if (seq.tokens > 0) append_page<D, F32>(a, seq, b, pg, h, key);
    return;
  }
  g -= kv_groups;
  const int pass = g % passes;
  g /= passes;
  const int parts = ceil_div(a.b.max_tokens, tokens_each);
  const int b = g / parts;
  const Seq seq = seq_of(a.b, a.b.q_start[b], a.b.q_start[b + 1], a.b.ctx_len[b]);
  const int l = threadIdx.x % LANES, head = pass * PER + threadIdx.x / LANES;
  const int hh = min(head, a.heads - 1);
  const int t0 = g % parts * tokens_each, t1 = min(t0 + tokens_each, seq.tokens);
  for (int t = t0; t < t1; ++t) {
    const int pos = seq.first + t;
    f32x4 x = load4<F32>(a.q.data, (size_t)(seq.row + t) * a.q.token_stride + (size_t)hh * a.q.head_stride + 4 * l);
    x = norm_rotate<D>(x, a.q_norm, a, l, max(pos, 0));
    if (pos < 0) x = f32x4{0.f, 0.f, 0.f, 0.f};
    if (head < a.heads)
      *reinterpret_cast<uint2*>(a.q_out + ((size_t)(seq.row + t) * a.heads + head) * D + 4 * l) = round4(x);
  }
}

template <int D>
void run_append(const AppendArgs& a, hipStream_t st) {
  constexpr int PER = APPEND_THREADS / (D / 4);
  const int pages = ((a.b.max_tokens - 1) >> a.c.shift) + 2;
  const int kv_groups = a.b.n_seqs * pages * a.c.kv_heads * 2;
  const int passes = ceil_div(a.heads, PER);
  const int each = a.b.max_tokens >= 64 ? 8 : 1;  // tokens of a work-group, one where there are few
  const int grid = kv_groups + a.b.n_seqs * ceil_div(a.b.max_tokens, each) * passes;
  if (a.type == HCR_F32)
    hipLaunchKernelGGL((append<D, true>), dim3(grid), dim3(APPEND_THREADS), 0, st, a, kv_groups, pages, passes, each);
  else
    hipLaunchKernelGGL((append<D, false>), dim3(grid), dim3(APPEND_THREADS), 0, st, a, kv_groups, pages, passes, each);
}

int launch_append(const AppendArgs& a, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (a.c.head_dim == 64)
    run_append<64>(a, st);
  else if (a.c.head_dim == 128)
    run_append<128>(a, st);
  else
    run_append<256>(a, st);
  return hipGetLastError() == hipSuccess ? HCR_OK : HCR_EHIP;
}

}  // namespace hcr
