// Reading the paged cache back as rows, gfx950 (MI355X): keys and values of either kind of pages, a code times its scale
// in FP32, rounded once.
//
// A work-group takes READ_SLOTS positions of a sequence (aligned, so that each 32 of them lie in one page and in whole
// chunks) of one kv head, keys and values, all of their loads on their way together.  Keys: 16 bytes of a page are some
// dimensions of one position, a lane's part of a row as they are.  Values: 16 bytes are some positions of one dimension;
// they are turned in registers, four bytes (codes) or two values (BF16) at a time, and go through LDS.
//
// Bound by the bytes.  Measured on MI355X: 51,200 positions of 8 sequences, 8 kv heads of 128, int8 to BF16 (318 MB) 72
// us, 4.4 TB/s, where a 4 GiB device copy moves 4.7 (to floats 123 us, 4.3 TB/s; BF16 pages 88 us, 4.8 TB/s).  On the way there: 32 positions a work-group 85 us; 64 positions, 16
// bytes of a lane's own row at a time 83; neighbouring lanes' 16 bytes beside each other and stores past the caches 71.
#include "hcr_append_device.h"

namespace hcr {

// Rows are stored once and read later: past the caches.
template <typename T>
__device__ __forceinline__ void put16(void* p, const T& v) {
  static_assert(sizeof(T) == 16, "16 bytes");
  __builtin_nontemporal_store(v, static_cast<T*>(p));
}

// N values of a page, as loaded: a lane's share of a row.
template <int CODE, int N>
struct Share {
  static constexpr int WORDS = N * (CODE == HCR_BF16 ? 2 : 1) / 4;
  alignas(4 * WORDS) uint32_t w[WORDS];
  __device__ __forceinline__ void load(const void* p) {
    if constexpr (WORDS == 4) {
      const uint4 u = ldw16(p);
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else if constexpr (WORDS == 2) {
      const uint2 u = ldw8(p);
      w[0] = u.x, w[1] = u.y;
    } else {
      w[0] = ldw4(p);
    }
  }
  __device__ __forceinline__ void values(float (&x)[N]) const {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      if constexpr (CODE == HCR_BF16) {
        x[e] = __uint_as_float(w[e / 2] << 16);
        x[e + 1] = __uint_as_float(w[e / 2] & 0xFFFF0000u);
      } else if constexpr (CODE == HCR_INT8) {
        x[e] = code(w[e / 4], e % 4);
        x[e + 1] = code(w[e / 4], e % 4 + 1);
      } else {
        const f32x2 v = e % 4 ? __builtin_amdgcn_cvt_pk_f32_fp8(w[e / 4], true)
                              : __builtin_amdgcn_cvt_pk_f32_fp8(w[e / 4], false);
        x[e] = v[0];
        x[e + 1] = v[1];
      }
    }
  }
};
// Times a scale in FP32, stored; `none`: zeros.
template <bool F32, int CODE, int N>
__device__ __forceinline__ void store_share(const Share<CODE, N>& u, float scale, bool none, void* out, size_t at) {
  float x[N] = {};
  if (!none) {
    u.values(x);
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = CODE == HCR_BF16 ? x[e] : x[e] * scale;
  }
  if constexpr (F32) {
#pragma unroll
    for (int e = 0; e < N; e += 4)
      put16(static_cast<float*>(out) + at + e, f32x4{x[e], x[e + 1], x[e + 2], x[e + 3]});
  } else {
    const uint4 r = round8(Values{{x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]}});
    put16(static_cast<uint16_t*>(out) + at, u32x4_t{r.x, r.y, r.z, r.w});
  }
}

template <int D, int CODE, bool F32>
__global__ __launch_bounds__(READ_THREADS) void cache_read(ReadArgs a, int parts) {
  constexpr bool CODED = CODE != HCR_BF16;
  constexpr int BYTES = CODED ? 1 : 2, EACH = 16 / BYTES;  // of a value; values in 16 bytes
  constexpr int ROW = D * BYTES + 16;                      // a row in LDS, 16 bytes more: rows start in other banks
  // values of a lane's share: 16 bytes of its row, so that a wave stores whole lines (int8 to floats, D = 256: 116 us against
  // 133 with 32 bytes); of BF16 8 for floats too (128 against 136), whose loads would else be of 8 bytes
  constexpr int OUT = F32 && CODED ? 4 : 8;
  constexpr int LANES = D / OUT;                           // of a row
  constexpr int ITEMS = READ_SLOTS * LANES / READ_THREADS;  // shares of a thread
  constexpr int N = 4 / BYTES;                             // dimensions of a thread's values
  constexpr int VITEMS = (READ_SLOTS / EACH * (D / N) + READ_THREADS - 1) / READ_THREADS;
  static_assert(ITEMS * READ_THREADS == READ_SLOTS * LANES && READ_SLOTS == 64, "a part has whole passes");
  __shared__ __align__(16) uint8_t tile[READ_SLOTS * ROW];
  int g = blockIdx.x;
  const int h = g % a.c.kv_heads;
  g /= a.c.kv_heads;
  const Seq seq = wave_seq(a.b, g / parts);
  if (seq.tokens <= 0) return;
  const int tid = threadIdx.x;
  // positions [lo, hi) of this part
  const int start = read_start(seq.first) + g % parts * READ_SLOTS;
  const int lo = max(start, seq.first), hi = min(start + READ_SLOTS, seq.first + seq.tokens);
  if (lo >= hi) return;
  // each 32 positions' page (-1: none, or no position asked for) and slot
  const int* table = a.b.table + (size_t)(g / parts) * a.b.table_stride;
  int number[2], slot[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int p = start + 32 * k;
    const bool in = p + 32 > 0 && p + 32 > lo && p < hi && p >= 0;
    number[k] = in ? table[p >> a.c.shift] : -1;
    slot[k] = p & ((1 << a.c.shift) - 1);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) number[k] = page_or_none(number[k], a.c.n_pages);
  const uint8_t* kp[2];
  const uint8_t* vp[2];
  size_t scales[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const size_t base = number[k] < 0 ? 0 : head_base(a.c, number[k], h) * BYTES;  // (page 0 is there: not stored)
    kp[k] = reinterpret_cast<const uint8_t*>(a.c.k) + base;
    vp[k] = reinterpret_cast<const uint8_t*>(a.c.v) + base;
    scales[k] = (number[k] < 0 ? 0 : scale_base(a.c, number[k], h)) + slot[k];
  }

  uint4 w[VITEMS][N];
  if (a.v_out) {
#pragma unroll
    for (int t = 0; t < VITEMS; ++t) {
      const int i = min(tid + t * READ_THREADS, READ_SLOTS / EACH * (D / N) - 1);
      const int o = i / (D / N), d = N * (i % (D / N)), k = o * EACH / 32;
      if (start + EACH * o >= hi || start + EACH * (o + 1) <= lo) continue;  // no position asked for
      const uint8_t* from = (k ? vp[1] : vp[0]) + ((size_t)((k ? slot[1] : slot[0]) / EACH + o % (32 / EACH)) * D + d) * 16;
#pragma unroll
      for (int e = 0; e < N; ++e) w[t][e] = ldw16(from + 16 * e);
    }
  }
  if (a.k_out) {
    Share<CODE, OUT> u[ITEMS];
    float scale[ITEMS];
#pragma unroll
    for (int t = 0; t < ITEMS; ++t) {  // neighbouring lanes: a row's values; 64 / LANES rows a wave
      const int i = tid + t * READ_THREADS, s = i / LANES, c = i % LANES, k = s / 32;
      if (start + s < lo || start + s >= hi) continue;
      const int at = (k ? slot[1] : slot[0]) + s % 32;
      u[t].load((k ? kp[1] : kp[0]) + (CODED ? k_code_at(a.c.shift, at, OUT * c) : 2 * k_at(a.c.shift, at, OUT * c)));
      if constexpr (CODED) scale[t] = a.code.k_scales[(k ? scales[1] : scales[0]) + s % 32];
    }
#pragma unroll
    for (int t = 0; t < ITEMS; ++t) {
      const int i = tid + t * READ_THREADS, s = i / LANES, c = i % LANES, k = s / 32;
      const int p = start + s;
      if (p >= lo && p < hi)
        store_share<F32>(u[t], CODED ? scale[t] : 1.f, (k ? number[1] : number[0]) < 0, a.k_out,
                    ((size_t)(seq.row + p - seq.first) * a.c.kv_heads + h) * D + OUT * c);
    }
  }
  if (!a.v_out) return;
#pragma unroll
  for (int t = 0; t < VITEMS; ++t) {
    const int i = tid + t * READ_THREADS, o = i / (D / N), d = N * (i % (D / N));
    if (i >= READ_SLOTS / EACH * (D / N)) break;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t r[N], turned[N];
#pragma unroll
      for (int e = 0; e < N; ++e) r[e] = k == 0 ? w[t][e].x : k == 1 ? w[t][e].y : k == 2 ? w[t][e].z : w[t][e].w;
      if constexpr (CODED) {
        transpose4(r, turned);
      } else {
        turned[0] = __builtin_amdgcn_perm(r[1], r[0], 0x05040100u);
        turned[1] = __builtin_amdgcn_perm(r[1], r[0], 0x07060302u);
      }
#pragma unroll
      for (int s = 0; s < N; ++s)
        *reinterpret_cast<uint32_t*>(&tile[(EACH * o + N * k + s) * ROW + d * BYTES]) = turned[s];
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < ITEMS; ++t) {
    const int i = tid + t * READ_THREADS, s = i / LANES, c = i % LANES, k = s / 32;
    const int p = start + s;
    if (p < lo || p >= hi) continue;
    const float scale = CODED ? a.code.v_scales[(k ? scales[1] : scales[0]) + s % 32] : 1.f;
    store_share<F32>(*reinterpret_cast<const Share<CODE, OUT>*>(&tile[s * ROW + OUT * BYTES * c]), scale,
                (k ? number[1] : number[0]) < 0, a.v_out,
                ((size_t)(seq.row + p - seq.first) * a.c.kv_heads + h) * D + OUT * c);
  }
}

template <int D, int CODE>
void run_read(const ReadArgs& a, hipStream_t st) {
  const int parts = read_parts(a.b);
  const dim3 grid(a.b.n_seqs * parts * a.c.kv_heads);
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
