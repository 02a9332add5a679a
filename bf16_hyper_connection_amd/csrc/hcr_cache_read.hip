// Reading the paged cache back as rows, gfx950 (MI355X): keys and values of either kind of pages, a code times its scale
// in FP32, rounded once.
//
// A work-group takes READ_SLOTS positions of a sequence (aligned, so that they lie in one page and in whole chunks) of
// one kv head, keys or values.  Keys: 16 bytes of a page are some dimensions of one position, a lane's part of a row as
// they are.  Values: 16 bytes are some positions of one dimension; they are turned in LDS, four bytes (codes) or two
// values (BF16) at a time.

#include "hcr_append_device.h"

namespace hcr {

template <int D, int CODE, bool F32>
__global__ __launch_bounds__(READ_THREADS) void cache_read(ReadArgs a, int parts) {
  constexpr bool CODED = CODE != HCR_BF16;
  constexpr int BYTES = CODED ? 1 : 2, EACH = 16 / BYTES;  // of a value; values in 16 bytes
  constexpr int ROW = D * BYTES + 16;                      // a row in LDS, 16 bytes more: rows start in other banks
  constexpr int LANES = D / 8;                             // of a row, 8 values each
  __shared__ __align__(16) uint8_t tile[READ_SLOTS * ROW];
  int g = blockIdx.x;
  const bool key = g & 1;
  g >>= 1;
  const int h = g % a.c.kv_heads;
  g /= a.c.kv_heads;
  const int b = g / parts;
  if (!(key ? a.k_out : a.v_out)) return;
  const Seq seq = wave_seq(a.b, b);
  if (seq.tokens <= 0) return;
  const int tid = threadIdx.x;
  // positions [lo, hi) of this part (one that begins before position 0 lies there whole)
  const int start = read_start(seq.first) + g % parts * READ_SLOTS;
  const int lo = max(start, seq.first), hi = min(start + READ_SLOTS, seq.first + seq.tokens);
  if (lo >= hi) return;
  const int pg = start >> a.c.shift, slot = start & ((1 << a.c.shift) - 1);
  const int number =
      start < 0 ? -1 : page_or_none(a.b.table[(size_t)b * a.b.table_stride + pg], a.c.n_pages);
  const uint8_t* in = nullptr;
  const float* scales = nullptr;
  if (number >= 0) {
    in = reinterpret_cast<const uint8_t*>(key ? a.c.k : a.c.v) + head_base(a.c, number, h) * BYTES;
    if (CODED) scales = (key ? a.code.k_scales : a.code.v_scales) + scale_base(a.c, number, h) + slot;
    if (!key) {
      // 32 bits of a row's dimensions (4 codes, 2 BF16) from as many 16-byte chunks
      constexpr int N = 4 / BYTES;
      for (int i = tid; i < READ_SLOTS / EACH * (D / N); i += READ_THREADS) {
        const int o = i / (D / N), d = N * (i % (D / N));
        const uint8_t* from = in + ((size_t)(slot / EACH + o) * D + d) * 16;
        uint32_t w[N][4];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const uint4 u = ldw16(from + 16 * e);
          w[e][0] = u.x;
          w[e][1] = u.y;
          w[e][2] = u.z;
          w[e][3] = u.w;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t t[N];
          if constexpr (CODED) {
            const uint32_t r[4] = {w[0][k], w[1][k], w[2][k], w[3][k]};
            transpose4(r, t);
          } else {
            t[0] = __builtin_amdgcn_perm(w[1][k], w[0][k], 0x05040100u);
            t[1] = __builtin_amdgcn_perm(w[1][k], w[0][k], 0x07060302u);
          }
#pragma unroll
          for (int s = 0; s < N; ++s)
            *reinterpret_cast<uint32_t*>(&tile[(EACH * o + N * k + s) * ROW + d * BYTES]) = t[s];
        }
      }
      __syncthreads();
    }
  }
  for (int i = tid; i < READ_SLOTS * LANES; i += READ_THREADS) {
    // keys: neighbouring lanes take 8 positions of a chunk, then the next chunks; values: a row's dimensions
    int s, l;
    if (key) {
      s = i % 8 + i / (8 * LANES) * 8;
      l = i / 8 % LANES;
    } else {
      s = i / LANES;
      l = i % LANES;
    }
    const int p = start + s;
    if (p < lo || p >= hi) continue;
    Values x{};
    if (number >= 0) {
      if constexpr (CODED) {
        const uint2 u = key ? *reinterpret_cast<const uint2*>(in + k_code_at(a.c.shift, slot + s, 8 * l))
                            : *reinterpret_cast<const uint2*>(&tile[s * ROW + 8 * l]);
        const float scale = scales[s];
        x = code_values<CODE>(u);
#pragma unroll
        for (int e = 0; e < 8; ++e) x.v[e] *= scale;
      } else {
        Raw<false> r;
        r.u[0] = key ? *reinterpret_cast<const uint4*>(in + 2 * (size_t)k_at(a.c.shift, slot + s, 8 * l))
                     : *reinterpret_cast<const uint4*>(&tile[s * ROW + 16 * l]);
        x = values<false>(r);
      }
    }
    const size_t at = ((size_t)(seq.row + p - seq.first) * a.c.kv_heads + h) * D + 8 * l;
    void* out = key ? a.k_out : a.v_out;
    if constexpr (F32) {
      float* to = static_cast<float*>(out) + at;
      *reinterpret_cast<f32x4*>(to) = f32x4{x.v[0], x.v[1], x.v[2], x.v[3]};
      *reinterpret_cast<f32x4*>(to + 4) = f32x4{x.v[4], x.v[5], x.v[6], x.v[7]};
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = round8(x);
    }
  }
}

template <int D, int CODE>
void run_read(const ReadArgs& a, hipStream_t st) {
  const int parts = read_parts(a.b);
  const dim3 grid(a.b.n_seqs * parts * a.c.kv_heads * 2);
  if (a.out_type == HCR_F32)
    hipLaunchKernelGGL((cache_read<D, CODE, true>), grid, dim3(READ_THREADS), 0, st, a, parts);
  else
    hipLaunchKernelGGL((cache_read<D, CODE, false>), grid, dim3(READ_THREADS), 0, st, a, parts);
}
template <int CODE>
void run_read_of(const ReadArgs& a, hipStream_t st) {
  if (a.c.head_dim == 64)
    run_read<64, CODE>(a, st);
  else if (a.c.head_dim == 128)
    run_read<128, CODE>(a, st);
  else
    run_read<256, CODE>(a, st);
}

int launch_read(const ReadArgs& a, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (a.code.code == HCR_INT8)
    run_read_of<HCR_INT8>(a, st);
  else if (a.code.code == HCR_E4M3)
    run_read_of<HCR_E4M3>(a, st);
  else
    run_read_of<HCR_BF16>(a, st);
  return hipGetLastError() == hipSuccess ? HCR_OK : HCR_EHIP;
}

}  // namespace hcr
