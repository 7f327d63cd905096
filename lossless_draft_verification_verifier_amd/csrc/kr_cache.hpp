// kr_cache.hpp -- the paged key/value cache: writing tokens, reading them back.
//
// A page holds `page` tokens of every kv head, [n_pages][Hkv][page][D]: the
// tokens of one head in one page are one block of memory, which is what an
// attention over that head streams.  E4M3 caches hold each (token, head) row
// as 8-bit codes and one power of two, the smallest 2^e with
// max |x| <= 448 * 2^e, as the byte e + 127.  A power of two costs none of
// the codes' relative precision (they are floating), makes x * 2^-e exact, so
// the one rounding is the code's own, and makes code * 2^e exact in bf16 for
// e >= -124: a reader loses nothing by widening to bf16.  (At e = -126 and -125
// the lowest codes end below 2^-133, the least step of bf16.)
//
// Both kernels are bound by HBM: a row is read once and written once, D / 8 lanes
// per row with 16-byte accesses on the wide side.  32768 tokens of 8 heads of 128,
// bf16 to E4M3 and back: 57 us to write (3.5 TB/s: a row waits for its length, then its
// page, then its source, which is loaded for a row with a page only; four rows per lane
// group saved 4 us but cost a single token 1.4) and 37 us to read (5.5 TB/s).
#pragma once

#include "svd_device.hpp"

namespace svd {

constexpr int kCacheBlock = 256;

// Where a cache's arrays are and how a sequence's positions map to them.
struct CacheView {
  uint8_t *k, *v;              // rows of D codes (1 byte) or bf16 (2 bytes)
  uint8_t *k_scale, *v_scale;  // [n_pages][Hkv][page], E4M3 only
  const int32_t *table;        // [B][max_pages]
  int64_t n_pages;
  int max_pages, page_shift, Hkv;
};

// Row (page, head, place) of position pos of sequence b, or -1 when the
// position has no page.
__device__ __forceinline__ int64_t cache_row(const CacheView &c, int64_t b, int64_t pos, int h) {
  const int64_t col = pos >> c.page_shift;
  if (pos < 0 || col >= c.max_pages) return -1;
  const int64_t pg = c.table[b * c.max_pages + col];
  if (pg < 0 || pg >= c.n_pages) return -1;
  return ((pg * c.Hkv + h) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {  // one instruction
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// The scale byte of a row whose largest finite magnitude is a: 448 = 1.75 * 2^8,
// so with a = m * 2^k, 1 <= m < 2, it is k - 8 for m <= 1.75 and k - 7 above.
__device__ __forceinline__ int e4m3_scale(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int k = (int)(bits >> 23) - 127;
  int e = (bits & 0x7fffffu) <= 0x600000u ? k - 8 : k - 7;
  e = a > 0.0f ? e : 0;
  return max(e, -126) + 127;
}
__device__ __forceinline__ float pow2_of_scale(int byte) {  // 2^(byte - 127)
  return byte == 255 ? __uint_as_float(0x7fc00000u)
                     : __uint_as_float(byte ? (uint32_t)byte << 23 : 0x00400000u);
}

// 8 elements of a source row
template <typename E, bool kVec>
__device__ __forceinline__ void load8(const typename E::elem *p, float *x) {
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < 8; i += E::kPerVec) {
      const vec16 w = *reinterpret_cast<const vec16 *>(p + i);
      E::unpack(w, x + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = E::at(p, i);
  }
}

// k and v rows of B x T tokens into the cache.  L = D / 8 lanes per (token,
// head, k or v) row; blocks_per_b workgroups per sequence.
template <typename E, bool kVec, bool kE4M3, int D>
__global__ __launch_bounds__(kCacheBlock) void kr_cache_write(
    const typename E::elem *__restrict__ k, const typename E::elem *__restrict__ v,
    int64_t k_stride, int64_t v_stride, const int32_t *__restrict__ ctx_len,
    const int32_t *__restrict__ n_new, const int32_t *__restrict__ dst, int64_t T,
    int64_t blocks_per_b, CacheView c) {
  constexpr int L = D / 8, kRows = kCacheBlock / L;
  const int64_t b = blockIdx.x / blocks_per_b;
  const int64_t row = (blockIdx.x % blocks_per_b) * kRows + threadIdx.x / L;
  const int lane = threadIdx.x % L;
  const int64_t rows = T * c.Hkv * 2;
  if (row >= rows) return;
  // v rows behind the k rows of a token
  const int hv = (int)(row % (2 * c.Hkv));
  const int64_t t = row / (2 * c.Hkv);
  const bool is_v = hv >= c.Hkv;
  const int h = is_v ? hv - c.Hkv : hv;
  const int n = n_new ? n_new[b] : (int)T;
  if (t >= n) return;
  int64_t at = t;
  if (dst) {
    at = dst[b * T + t];
    if (at < 0) return;
  }
  const int64_t ctx = ctx_len[b];
  if (ctx < 0) return;
  const int64_t to = cache_row(c, b, ctx + at, h);
  if (to < 0) return;
  const typename E::elem *src = (is_v ? v + (b * T + t) * v_stride : k + (b * T + t) * k_stride) +
                                (int64_t)h * D + lane * 8;
  float x[8];
  load8<E, kVec>(src, x);
  uint8_t *out = is_v ? c.v : c.k;
  if constexpr (!kE4M3) {
    vec16 w;
    w.x = pack_bf16(x[0], x[1]);
    w.y = pack_bf16(x[2], x[3]);
    w.z = pack_bf16(x[4], x[5]);
    w.w = pack_bf16(x[6], x[7]);
    *reinterpret_cast<vec16 *>(out + (to * D + lane * 8) * 2) = w;
  } else {
    const float inf = __builtin_huge_valf();
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // an infinity has no code: it is held as NaN
      const float m = fabsf(x[i]);
      const bool finite = m < inf;
      a = finite ? fmaxf(a, m) : a;
      x[i] = finite ? x[i] : __uint_as_float(0x7fc00000u);
    }
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor(a, off, 64));
    const int byte = e4m3_scale(a);
    const float r = __uint_as_float((uint32_t)(254 - byte) << 23);  // 2^(127 - byte), exact
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= r;
    if (byte == 247) {  // 256 * 2^120 is no number: the largest ones are held as 240 * 2^120
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = fabsf(x[i]) > 240.0f ? copysignf(240.0f, x[i]) : x[i];
    }
    uint32_t lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
    uint2 w;
    w.x = lo;
    w.y = hi;
    *reinterpret_cast<uint2 *>(out + to * D + lane * 8) = w;
    if (lane == 0) (is_v ? c.v_scale : c.k_scale)[to] = (uint8_t)byte;
  }
}

// Positions start[b] .. start[b] + count[b] - 1 of every sequence, widened to
// E.  A position without a page gives NaN.
template <typename E, bool kE4M3, int D>
__global__ __launch_bounds__(kCacheBlock) void kr_cache_read(
    CacheView c, const int32_t *__restrict__ start, const int32_t *__restrict__ count, int64_t N,
    int64_t blocks_per_b, typename E::elem *__restrict__ k, typename E::elem *__restrict__ v) {
  constexpr int L = D / 8, kRows = kCacheBlock / L;
  const int64_t b = blockIdx.x / blocks_per_b;
  const int64_t row = (blockIdx.x % blocks_per_b) * kRows + threadIdx.x / L;
  const int lane = threadIdx.x % L;
  if (row >= N * c.Hkv * 2) return;
  const int hv = (int)(row % (2 * c.Hkv));
  const int64_t t = row / (2 * c.Hkv);
  const bool is_v = hv >= c.Hkv;
  const int h = is_v ? hv - c.Hkv : hv;
  if (t >= (count ? count[b] : (int)N)) return;
  const int64_t s = start ? start[b] : 0;
  const int64_t from = s < 0 ? -1 : cache_row(c, b, s + t, h);
  float x[8];
  if (from < 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(0x7fc00000u);
  } else if constexpr (kE4M3) {
    const uint2 w = *reinterpret_cast<const uint2 *>((is_v ? c.v : c.k) + from * D + lane * 8);
    const float r = pow2_of_scale((is_v ? c.v_scale : c.k_scale)[from]);
    x[0] = __builtin_amdgcn_cvt_f32_fp8(w.x, 0) * r;
    x[1] = __builtin_amdgcn_cvt_f32_fp8(w.x, 1) * r;
    x[2] = __builtin_amdgcn_cvt_f32_fp8(w.x, 2) * r;
    x[3] = __builtin_amdgcn_cvt_f32_fp8(w.x, 3) * r;
    x[4] = __builtin_amdgcn_cvt_f32_fp8(w.y, 0) * r;
    x[5] = __builtin_amdgcn_cvt_f32_fp8(w.y, 1) * r;
    x[6] = __builtin_amdgcn_cvt_f32_fp8(w.y, 2) * r;
    x[7] = __builtin_amdgcn_cvt_f32_fp8(w.y, 3) * r;
  } else {
    const vec16 w =
        *reinterpret_cast<const vec16 *>((is_v ? c.v : c.k) + (from * D + lane * 8) * 2);
    BF16::unpack(w, x);
  }
  typename E::elem *out = (is_v ? v : k) + ((b * N + t) * c.Hkv + h) * D + lane * 8;
  if constexpr (sizeof(typename E::elem) == 2) {
    vec16 w;
    w.x = pack_bf16(x[0], x[1]);
    w.y = pack_bf16(x[2], x[3]);
    w.z = pack_bf16(x[4], x[5]);
    w.w = pack_bf16(x[6], x[7]);
    *reinterpret_cast<vec16 *>(out) = w;
  } else {
    vec16 w;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      w.x = __float_as_uint(x[i]);
      w.y = __float_as_uint(x[i + 1]);
      w.z = __float_as_uint(x[i + 2]);
      w.w = __float_as_uint(x[i + 3]);
      *reinterpret_cast<vec16 *>(out + i) = w;
    }
  }
}

}  // namespace svd
