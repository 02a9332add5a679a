// Append of a decode window to the paged cache, gfx950 (MI355X): per head, y = x w / sqrt(mean(x^2) + eps), the
// first rope_dim values rotated by the angles of the token's position, rounded once to BF16; q to its rows, k and
// v into the pages, and the mean key of each page that the window completes.
//
// One launch.  A lane holds 8 consecutive dimensions (16 bytes of BF16), D / 8 lanes a head: the sum of squares is a
// butterfly over them; the partner of a rotated value (j, j + r/2) sits in another lane at the same place, that of
// (2j, 2j + 1) in the same lane.  The first work-groups take (sequence, page, kv head, k or v): the page's new tokens
// are staged in LDS, 64 slots at a time, and written in the page's order, so that a prompt's pages go out as whole
// lines (a lane writes 8 dimensions of a slot, or 8 slots of a dimension).  The others take query heads.  Loads of
// several tokens go out together.  Nothing bounds it but the bytes of the rows, and for a few tokens the launch
// itself.  Measured on MI355X: 4,352 tokens of 32 + 16 heads of 128, BF16, 26.1 us, 4.2 TB/s (in graphs of calls, inputs
// rotated, 27.4 against 28.5 with loads that stay in the caches, 28.3 against 40.7 with 4 dimensions a lane and one
// token's load at a time); one token of 48 + 16 heads of 256 3.8 us.

#include <hip/hip_runtime.h>

#include "hcr_paged_device.h"

namespace hcr {

constexpr int SLOTS = 64;  // slots of a page staged at a time

struct Values {
  float v[8];
};
// 8 consecutive values of a row, as loaded and as FP32
template <bool F32>
struct Raw {
  uint4 u[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw<F32> load8(const void* p, size_t at) {
  Raw<F32> r;
  if constexpr (F32) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
    r.u[0] = ldw16(q);
    r.u[1] = ldw16(q + 1);
  } else {
    r.u[0] = ldw16(static_cast<const uint16_t*>(p) + at);
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ Values values(const Raw<F32>& r) {
  Values x;
  if constexpr (F32) {
    const uint32_t w[8] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w, r.u[1].x, r.u[1].y, r.u[1].z, r.u[1].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) x.v[e] = __uint_as_float(w[e]);
  } else {
    const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x.v[2 * e] = __uint_as_float(w[e] << 16);
      x.v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
  return x;
}
__device__ __forceinline__ uint4 round8(const Values& x) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const f32x2 a = {x.v[2 * e], x.v[2 * e + 1]};
    w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ Values load_f8(const float* p) {
  const f32x4 a = ld4(p), b = ld4(p + 4);
  return Values{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}

// The sum over the LANES (8, 16 or 32) lanes of a head, in every one of them.
template <int LANES>
__device__ __forceinline__ float head_sum(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  if constexpr (LANES >= 16) v += dpp<0x140>(v);
  if constexpr (LANES == 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// Norm and rotation of a head's values 8 l .. 8 l + 7 at position pos (every lane of the wave takes part).
template <int D>
__device__ __forceinline__ Values norm_rotate(Values x, const float* w, const AppendArgs& a, int l, int pos) {
  constexpr int LANES = D / 8;
  if (w) {
    const Values g = load_f8(w + 8 * l);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += x.v[e] * x.v[e];
    const float rs = 1.f / sqrtf(head_sum<LANES>(ss) * (1.f / D) + a.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) x.v[e] = x.v[e] * rs * g.v[e];
  }
  if (a.rope_dim) {
    const float* row = a.rope + (size_t)pos * a.rope_dim;
    const int half = a.rope_dim >> 1;
    const bool in = 8 * l < a.rope_dim;
    if (a.rope_style == HCR_ROPE_PAIRS) {
      if (in) {
        const f32x4 c = ld4(row + 4 * l), s = ld4(row + half + 4 * l);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = x.v[2 * e], q = x.v[2 * e + 1];
          x.v[2 * e] = p * c[e] - q * s[e];
          x.v[2 * e + 1] = q * c[e] + p * s[e];
        }
      }
    } else {
      const bool low = 8 * l < half;
      const int from = (threadIdx.x & 63) + (in ? (low ? half >> 3 : -(half >> 3)) : 0);
      Values y;
#pragma unroll
      for (int e = 0; e < 8; ++e) y.v[e] = __shfl(x.v[e], from);
      if (in) {
        const int j = low ? 8 * l : 8 * l - half;
        const Values c = load_f8(row + j), s = load_f8(row + half + j);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x.v[e] = low ? x.v[e] * c.v[e] - y.v[e] * s.v[e] : x.v[e] * c.v[e] + y.v[e] * s.v[e];
      }
    }
  }
  return x;
}

// The new tokens of one page of one kv head: staged, written in the page's order, the mean key where complete.
template <int D, bool F32>
__device__ void append_page(const AppendArgs& a, const Seq& seq, int b, int pg, int h, bool key) {
  constexpr int LANES = D / 8, PER = APPEND_THREADS / LANES;  // tokens of a pass
  constexpr int PASSES = SLOTS / PER;
  constexpr int ROW = D + 8;  // 16 bytes more: slots start in other banks
  constexpr int C = D / 8;    // 16-byte chunks of a slot
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
    if (s0 < s1) {
      Raw<F32> raw[PASSES];
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {  // past the end the last slot again: its line is there, nothing is branched
        const int slot = min(s0 + p * PER + sub, s1 - 1);
        raw[p] = load8<F32>(rows.data, (size_t)(seq.row + start + slot - seq.first) * rows.token_stride +
                                           (size_t)h * rows.head_stride + 8 * l);
      }
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        if (s0 + p * PER >= s1) break;
        const int slot = min(s0 + p * PER + sub, s1 - 1);
        Values x = values<F32>(raw[p]);
        if (key) x = norm_rotate<D>(x, a.k_norm, a, l, start + slot);
        if (s0 + p * PER + sub < s1) *reinterpret_cast<uint4*>(&tile[(slot - base) * ROW + 8 * l]) = round8(x);
      }
    }
    __syncthreads();
    if (key) {
      for (int i = tid; i < SLOTS * C; i += APPEND_THREADS) {
        const int c = i / SLOTS, slot = base + i % SLOTS;
        if (slot >= s0 && slot < s1)
          *reinterpret_cast<uint4*>(out + k_at(a.c.shift, slot, 8 * c)) =
              *reinterpret_cast<const uint4*>(&tile[(slot - base) * ROW + 8 * c]);
      }
      if (mean) {
        for (int slot = base + mg; slot < min(base + SLOTS, page); slot += MG) {
          const uint4 u = slot >= lo ? *reinterpret_cast<const uint4*>(&tile[(slot - base) * ROW + 8 * mc])
                                     : *reinterpret_cast<const uint4*>(out + k_at(a.c.shift, slot, 8 * mc));
          Raw<false> r;
          r.u[0] = u;
          const Values x = values<false>(r);
#pragma unroll
          for (int e = 0; e < 8; ++e) total[e] += x.v[e];
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

// EACH tokens of a work-group of query heads, their loads together.
template <int D, bool F32, int EACH>
__global__ __launch_bounds__(APPEND_THREADS) void append(AppendArgs a, int kv_groups, int pages, int passes) {
  constexpr int LANES = D / 8, PER = APPEND_THREADS / LANES;
  int g = blockIdx.x;
  if (g < kv_groups) {
    const bool key = g & 1;
    g >>= 1;
    const int h = g % a.c.kv_heads;
    g /= a.c.kv_heads;
    const int b = g / pages;
    const Seq seq = wave_seq(a.b, b);
    const int pg = (max(seq.first, 0) >> a.c.shift) + g % pages;
    if (seq.tokens > 0) append_page<D, F32>(a, seq, b, pg, h, key);
    return;
  }
  g -= kv_groups;
  const int pass = g % passes;
  g /= passes;
  const int parts = ceil_div(a.b.max_tokens, EACH);
  const int b = g / parts;
  const Seq seq = wave_seq(a.b, b);
  const int l = threadIdx.x % LANES, head = pass * PER + threadIdx.x / LANES;
  const int hh = min(head, a.heads - 1);
  const int t0 = g % parts * EACH;
  if (t0 >= seq.tokens) return;
  Raw<F32> raw[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int t = min(t0 + i, seq.tokens - 1);
    raw[i] = load8<F32>(a.q.data, (size_t)(seq.row + t) * a.q.token_stride + (size_t)hh * a.q.head_stride + 8 * l);
  }
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int t = t0 + i;
    if (t >= seq.tokens) break;
    const int pos = seq.first + t;
    // a token of a padded sequence has no position: zeros, and no row of the table is read (one token a work-group's
    // pass, so nothing diverges)
    const Values x = pos < 0 ? Values{} : norm_rotate<D>(values<F32>(raw[i]), a.q_norm, a, l, pos);
    if (head < a.heads)
      *reinterpret_cast<uint4*>(a.q_out + ((size_t)(seq.row + t) * a.heads + head) * D + 8 * l) = round8(x);
  }
}

template <int D, bool F32, int EACH>
void run(const AppendArgs& a, hipStream_t st) {
  const AppendGrid g = append_grid(a.c, a.b, a.heads);
  hipLaunchKernelGGL((append<D, F32, EACH>), dim3(g.groups), dim3(APPEND_THREADS), 0, st, a, (int)g.kv_groups, g.pages,
                     g.passes);
}
template <int D>
void run_append(const AppendArgs& a, hipStream_t st) {
  const bool many = append_each(a.b) > 1;
  if (a.type == HCR_F32)
    many ? run<D, true, APPEND_EACH>(a, st) : run<D, true, 1>(a, st);
  else
    many ? run<D, false, APPEND_EACH>(a, st) : run<D, false, 1>(a, st);
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
