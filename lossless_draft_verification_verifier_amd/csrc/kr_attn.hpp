// kr_attn.hpp -- attention of a draft tree over the paged cache.
//
// Row r = t * group + i of kv head h is query head h * group + i of node t; all
// rows of a (prefix, kv head) read the same keys and values.  A wave holds
// 16 * NT rows and walks tiles of 32 cached tokens with the running maximum m
// and sum l of the softmax:
//   S^T = K Q^T         v_mfma_f32_16x16x32_bf16, tokens x rows
//   p = exp2(S c - m c), c = scale * log2(e)
//   O^T += V^T P^T      the same instruction, head dimension x rows
// In the transposed products a lane keeps one row (lane % 16) throughout: the
// maximum over tokens is in-lane plus two shuffles, the rescaling of O is a
// per-lane factor, and the p that the first product leaves in a lane are the
// operand the second one wants there, so p never crosses lanes.  The order of
// the reduction index is free as long as both operands share it; it is chosen
// so that every load of K and V is 16 bytes of one token's row, and V is
// transposed in registers (one byte permute per two elements).
// E4M3 rows are widened to bf16 with their power of two by the conversion
// instruction, which is exact, so both cache types run the same products.
// p is rounded to bf16 once, as the operand of the second product; m, l and O
// stay in 32 bits and l sums the unrounded p.
//
// The tiles of a prefix (its context, then its tree) are split evenly over S
// workgroups when there are few (prefix, head) pairs, and over the 4 waves of
// a workgroup; kr_attn_join merges the S parts.
#pragma once

#include "kr_cache.hpp"
#include "kr_tree.hpp"
#include "svd_device.hpp"

namespace svd {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kAttnBlock = 256;
constexpr int kAttnWaves = kAttnBlock / 64;
constexpr int kAttnTile = 32;       // cached tokens per step of a wave
constexpr int kAttnMaxSplits = 64;

struct AttnArgs {
  const uint16_t *q;        // [B][T][Hq][D] bf16, q_stride elements between tokens
  int64_t q_stride;
  const int32_t *ctx_len, *n_nodes;
  const uint32_t *anc;      // [B][T][W] or null: a chain
  int64_t room;             // positions of a sequence's pages
  int T, group, S, m_tiles, units;  // units = B * Hkv * S
  float c;                  // scale * log2(e)
  uint16_t *out;            // [B][T][Hq][D]
  float *lse;               // [B][T][Hq] or null
  float *part_o;            // [S][B][T][Hq][D] when S > 1
  float *part_ms;           // [S][B][T][Hq][2]
  int64_t rows_all;         // B * T * Hq
};

__device__ __forceinline__ f32x4 mfma_bf16(const vec16 &a, const vec16 &b, const f32x4 &c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// two E4M3 codes of word w, times the power of two s, as bf16
template <bool kHigh>
__device__ __forceinline__ uint32_t widen2(uint32_t w, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, kHigh));
}

__device__ __forceinline__ bool nonfinite2(uint32_t w) {  // a bf16 pair that holds NaN or inf
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const vec16 x = *reinterpret_cast<const vec16 *>(p + 4 * i);
      w[i] = x.x;
      w[i + 1] = x.y;
      w[i + 2] = x.z;
      w[i + 3] = x.w;
    }
  } else if constexpr (N == 2) {
    const u32x2 x = *reinterpret_cast<const u32x2 *>(p);
    w[0] = x.x;
    w[1] = x.y;
  } else {
    static_assert(N == 1, "");
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
}

// The state of a wave: NT groups of 16 rows.
template <int D, int NT>
struct AttnState {
  static constexpr int DT = D / 16;
  f32x4 o[NT][DT];
  float m[NT], l[NT];
  float base[NT];  // m * c as rounded: the exponent that l and o are held over
};

// One tile of 32 tokens.  row_k[2]: the cache rows of tokens lane % 16 and
// 16 + lane % 16; row_v[8]: of tokens 4 g + i and 16 + 4 g + i, g = lane / 16.
// A row of -1 is a token that is not there (v is taken as zero).  allow[n]: bits of
// the tile's tokens that row 16 n + lane % 16 attends to.
template <int D, bool kE4M3, int NT, bool kTree>
__device__ __forceinline__ void attn_tile(const CacheView &cv, const vec16 (&qf)[NT][D / 32],
                                          const int64_t (&row_k)[2], const int64_t (&row_v)[8],
                                          const uint32_t (&allow)[NT], bool all, bool poison,
                                          float c, AttnState<D, NT> &st) {
  constexpr int DT = D / 16, ST = D / 32;
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  // keys
  vec16 kf[2][ST];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int64_t row = row_k[s] < 0 ? 0 : row_k[s];
    if constexpr (kE4M3) {
      const float sc = pow2_of_scale(cv.k_scale[row]);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const vec16 w = *reinterpret_cast<const vec16 *>(cv.k + row * D + 64 * i + 16 * g);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a = h ? w.z : w.x, b = h ? w.w : w.y;
          kf[s][2 * i + h].x = widen2<false>(a, sc);
          kf[s][2 * i + h].y = widen2<true>(a, sc);
          kf[s][2 * i + h].z = widen2<false>(b, sc);
          kf[s][2 * i + h].w = widen2<true>(b, sc);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < ST; ++i)
        kf[s][i] = *reinterpret_cast<const vec16 *>(cv.k + (row * D + 32 * i + 8 * g) * 2);
    }
  }
  // values, as pairs of neighbouring head dimensions of one token
  uint32_t vr[8][DT / 2];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t row = row_v[j] < 0 ? 0 : row_v[j];
    if constexpr (kE4M3) {
      const float sc = pow2_of_scale(cv.v_scale[row]);
      uint32_t w[DT / 4];
      load_words<DT / 4>(cv.v + row * D + DT * n, w);
#pragma unroll
      for (int i = 0; i < DT / 4; ++i) {
        vr[j][2 * i] = widen2<false>(w[i], sc);
        vr[j][2 * i + 1] = widen2<true>(w[i], sc);
      }
    } else {
      load_words<DT / 2>(cv.v + (row * D + DT * n) * 2, vr[j]);
    }
    if (row_v[j] < 0) {
#pragma unroll
      for (int i = 0; i < DT / 2; ++i) vr[j][i] = 0;
    }
  }
  // a masked p is 0, and 0 * NaN is NaN: values that are not finite leave the
  // product and join the rows that attend to them one by one
  bool odd = false;
  if constexpr (kTree) {
    bool any = false;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < DT / 2; ++i) any |= nonfinite2(vr[j][i]);
    odd = __any(any);
    if (odd) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < DT / 2; ++i) {
          if ((vr[j][i] & 0x7f80u) == 0x7f80u) vr[j][i] &= 0xffff0000u;
          if ((vr[j][i] & 0x7f800000u) == 0x7f800000u) vr[j][i] &= 0x0000ffffu;
        }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    f32x4 s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < ST; ++i) s[u] = mfma_bf16(kf[u][i], qf[t][i], s[u]);
    }
    if (poison) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) s[u][r] = __uint_as_float(0x7fc00000u);
    }
    if (!all) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (!((allow[t] >> (16 * u + 4 * g + r)) & 1u)) s[u][r] = kNegInf;
    }
    float mx = st.m[t];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) mx = fmaxf(mx, s[u][r]);
    mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
    mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
    if (__any(mx != st.m[t])) {
      const float next = mx * c;
      const float f = mx == st.m[t] ? 1.0f : fast_exp2(st.base[t] - next);
      st.l[t] *= f;
#pragma unroll
      for (int i = 0; i < DT; ++i) st.o[t][i] *= f;
      st.m[t] = mx;
      st.base[t] = next;
    }
    const float base = mx == kNegInf ? 0.0f : st.base[t];
    float p[8];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        p[4 * u + r] = fast_exp2(__builtin_fmaf(s[u][r], c, -base));
        st.l[t] += p[4 * u + r];
      }
    vec16 pf;
#pragma unroll
    for (int j = 0; j < 4; ++j) pf[j] = pack_bf16(p[2 * j], p[2 * j + 1]);
#pragma unroll
    for (int i = 0; i < DT; ++i) {
      vec16 vf;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        vf[j] = __builtin_amdgcn_perm(vr[2 * j + 1][i / 2], vr[2 * j][i / 2],
                                      (i & 1) ? 0x07060302u : 0x05040100u);
      st.o[t][i] = mfma_bf16(vf, pf, st.o[t][i]);
    }
    if constexpr (kTree) {
      if (odd) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          for (int from = 0; from < 4; ++from) {
            const int tok = 16 * (j >> 2) + 4 * from + (j & 3);
            const float pt = __shfl(p[j], 16 * from + n, 64);
            const uint32_t hi = __shfl((uint32_t)((uint64_t)row_v[j] >> 32), 16 * from, 64);
            const uint32_t lo = __shfl((uint32_t)row_v[j], 16 * from, 64);
            const int64_t row = (int64_t)(((uint64_t)hi << 32) | lo);
            if (row < 0 || !((allow[t] >> tok) & 1u)) continue;
            const float sc = kE4M3 ? pow2_of_scale(cv.v_scale[row]) : 1.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int i = 0; i < DT; ++i) {
                const int64_t at = row * D + DT * (4 * g + r) + i;
                float x;
                if constexpr (kE4M3)
                  x = __builtin_amdgcn_cvt_f32_fp8((uint32_t)cv.v[at], 0) * sc;
                else
                  x = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(cv.v)[at] << 16);
                if (!(fabsf(x) < __builtin_huge_valf())) st.o[t][i][r] += pt * x;
              }
          }
      }
    }
  }
}

// What a part (exponent m, sum l) is scaled by under the common exponent mm.  A
// part without scores has l = 0; one whose scores were all NaN has no maximum
// either, and its NaN sum has to stay.
__device__ __forceinline__ float part_factor(float m, float l, float mm) {
  return m == kNegInf ? (l == 0.0f ? 0.0f : 1.0f) : fast_exp2(m - mm);
}

// Whether a prefix's lengths are out of range.
__device__ __forceinline__ bool attn_bad(int ctx, int nodes, int T, int64_t room) {
  return ctx < 0 || nodes < 0 || nodes > T || (int64_t)ctx + nodes > room;
}

template <int D, bool kE4M3, int NT>
__global__ __launch_bounds__(kAttnBlock) void kr_tree_attention(CacheView cv, AttnArgs a) {
  constexpr int DT = D / 16, ST = D / 32, M = 16 * NT;
  __shared__ float lds_ms[kAttnWaves][M][2];
  __shared__ float lds_o[kAttnWaves][M][D + 4];  // + 4: rows start in different banks
  // units on neighbouring blocks run on different XCDs; the row tiles of one
  // unit, which read the same keys and values, stay on one
  const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
  const int unit = (idx / a.m_tiles) * 8 + xcd, mt = idx % a.m_tiles;
  if (unit >= a.units) return;
  const int s = unit % a.S, bh = unit / a.S;
  const int h = bh % cv.Hkv;
  const int64_t b = bh / cv.Hkv;
  const int Hq = cv.Hkv * a.group;
  const int ctx = a.ctx_len[b];
  const int nodes = a.n_nodes ? a.n_nodes[b] : a.T;
  // lengths out of range: every row of the prefix is NaN
  const bool bad = attn_bad(ctx, nodes, a.T, a.room);
  const int rows = (bad ? a.T : nodes) * a.group;
  if (mt * M >= rows) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = lane & 15, g = lane >> 4;

  vec16 qf[NT][ST];
  int node[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = mt * M + 16 * t + n;
    node[t] = min(r, rows - 1) / a.group;
    const uint16_t *q = a.q + (b * a.T + node[t]) * a.q_stride +
                        (int64_t)(h * a.group + min(r, rows - 1) % a.group) * D;
#pragma unroll
    for (int i = 0; i < ST; ++i)
      qf[t][i] = *reinterpret_cast<const vec16 *>(
          q + (kE4M3 ? 64 * (i / 2) + 16 * g + 8 * (i & 1) : 32 * i + 8 * g));
  }
  AttnState<D, NT> st;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    st.m[t] = kNegInf;
    st.base[t] = kNegInf;
    st.l[t] = 0.0f;
#pragma unroll
    for (int i = 0; i < DT; ++i) st.o[t][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  if (!bad) {
    const int ctx_tiles = (ctx + kAttnTile - 1) / kAttnTile;
    const int tree_tiles = (nodes + kAttnTile - 1) / kAttnTile;
    const int all_tiles = ctx_tiles + tree_tiles;
    const int per = (all_tiles + a.S - 1) / a.S;
    const int lo = s * per, hi = min(lo + per, all_tiles);
    const int W = (a.T + 31) / 32;
    for (int tile = lo + wave; tile < hi; tile += kAttnWaves) {
      const bool tree = tile >= ctx_tiles;
      const int64_t p0 = tree ? (int64_t)ctx + (int64_t)(tile - ctx_tiles) * kAttnTile
                              : (int64_t)tile * kAttnTile;
      const int left = (int)min((int64_t)kAttnTile, (tree ? (int64_t)ctx + nodes : ctx) - p0);
      int64_t row_k[2], row_v[8];
      bool poison = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = 16 * i + n;
        row_k[i] = k < left ? cache_row(cv, b, p0 + k, h) : -1;
        poison |= k < left && row_k[i] < 0;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = 16 * (i >> 2) + 4 * g + (i & 3);
        row_v[i] = k < left ? cache_row(cv, b, p0 + k, h) : -1;
      }
      poison = __any(poison);
      const uint32_t there = left == 32 ? 0xffffffffu : (1u << left) - 1u;
      uint32_t allow[NT];
      if (tree) {
        const int w = tile - ctx_tiles;
#pragma unroll
        for (int t = 0; t < NT; ++t)
          allow[t] = there & (a.anc ? a.anc[(b * a.T + node[t]) * W + w]
                                    : range_bits(0, node[t], w));
        attn_tile<D, kE4M3, NT, true>(cv, qf, row_k, row_v, allow, false, poison, a.c, st);
      } else {
#pragma unroll
        for (int t = 0; t < NT; ++t) allow[t] = there;
        attn_tile<D, kE4M3, NT, false>(cv, qf, row_k, row_v, allow, left == 32, poison, a.c, st);
      }
    }
  }
  // join the waves: O over the largest maximum, l summed over the lanes of a row
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    st.l[t] += __shfl_xor(st.l[t], 16, 64);
    st.l[t] += __shfl_xor(st.l[t], 32, 64);
    if (g == 0) {
      lds_ms[wave][16 * t + n][0] = st.base[t];
      lds_ms[wave][16 * t + n][1] = st.l[t];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < DT; i += 4)
        *reinterpret_cast<f32x4 *>(&lds_o[wave][16 * t + n][DT * (4 * g + r) + i]) =
            f32x4{st.o[t][i][r], st.o[t][i + 1][r], st.o[t][i + 2][r], st.o[t][i + 3][r]};
  }
  __syncthreads();
  constexpr int V = D / 4;  // 16-byte pieces of a row
  for (int i = tid; i < M * V; i += kAttnBlock) {
    const int r = i / V, d = (i % V) * 4;
    if (mt * M + r >= rows) continue;
    float m = kNegInf, l = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) m = fmaxf(m, lds_ms[w][r][0]);
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      const float f = part_factor(lds_ms[w][r][0], lds_ms[w][r][1], m);
      l += lds_ms[w][r][1] * f;
      o += *reinterpret_cast<const f32x4 *>(&lds_o[w][r][d]) * f;
    }
    if (bad) l = __uint_as_float(0x7fc00000u);
    const int R = mt * M + r;
    const int64_t row = (b * a.T + R / a.group) * Hq + h * a.group + R % a.group;
    if (a.S > 1) {
      const int64_t pr = (int64_t)s * a.rows_all + row;
      *reinterpret_cast<f32x4 *>(a.part_o + pr * D + d) = o;
      if (d == 0) {
        a.part_ms[2 * pr] = m;
        a.part_ms[2 * pr + 1] = l;
      }
    } else {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      uint2 w;
      w.x = pack_bf16(o[0] * inv, o[1] * inv);
      w.y = pack_bf16(o[2] * inv, o[3] * inv);
      *reinterpret_cast<uint2 *>(a.out + row * D + d) = w;
      if (d == 0 && a.lse)
        a.lse[row] = l == 0.0f ? kNegInf : (m + __log2f(l)) * 0.6931471805599453f;
    }
  }
}

// The S parts of every row: D / 4 lanes per row.
template <int D>
__global__ __launch_bounds__(kAttnBlock) void kr_attn_join(AttnArgs a, int Hq) {
  constexpr int L = D / 4;
  const int64_t row = (int64_t)blockIdx.x * (kAttnBlock / L) + threadIdx.x / L;
  if (row >= a.rows_all) return;
  const int d = (threadIdx.x % L) * 4;
  const int64_t bt = row / Hq;
  const int64_t b = bt / a.T;
  const int nodes = a.n_nodes ? a.n_nodes[b] : a.T;
  // a prefix out of range wrote NaN parts for every row
  if (bt % a.T >= nodes && !attn_bad(a.ctx_len[b], nodes, a.T, a.room)) return;
  float m = kNegInf;
  for (int s = 0; s < a.S; ++s) m = fmaxf(m, a.part_ms[2 * (s * a.rows_all + row)]);
  float l = 0.0f;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < a.S; ++s) {
    const int64_t pr = s * a.rows_all + row;
    const float ms = a.part_ms[2 * pr], ls = a.part_ms[2 * pr + 1];
    const float f = part_factor(ms, ls, m);
    l += ls * f;
    o += *reinterpret_cast<const f32x4 *>(a.part_o + pr * D + d) * f;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint2 w;
  w.x = pack_bf16(o[0] * inv, o[1] * inv);
  w.y = pack_bf16(o[2] * inv, o[3] * inv);
  *reinterpret_cast<uint2 *>(a.out + row * D + d) = w;
  if (d == 0 && a.lse)
    a.lse[row] = l == 0.0f ? kNegInf : (m + __log2f(l)) * 0.6931471805599453f;
}

}  // namespace svd
