// kr_shared.hpp -- attention of a group's rows over the tokens that its sequences share.
//
// The rows of all nodes of all sequences of a group, query heads of a kv head included,
// see the same shared tokens, all of them: no masks, whole tiles, and every key and value
// is used for hundreds of rows.  So this is a matrix product with a softmax in its middle:
//   S^T = K Q^T     v_mfma_f32_32x32x16_bf16, 32 tokens x 32 rows
//   p = exp2(S c - m c)
//   O^T += V^T P^T  the same instruction, 32 head elements x 32 rows
// A lane keeps one row of 32 and half of the tokens of a product's block; p leaves the
// first product in the order in which the second one takes it.  A wave has 32 rows, eight
// waves a workgroup, two a SIMD, one workgroup per CU.  With 16 rows of a wave the reads of
// K and V from LDS are what bounds it (141 us for 256 sequences of 9 nodes, 32 query and 8 kv
// heads, over 2048 shared E4M3 tokens), with 64 rows and one wave per SIMD the issue of one
// wave's instructions (125 us); 32 rows and two waves take 92 us (97 on another card), 840
// TFLOP/s, where a large library product reaches 1328.  Capped scores bind the vector units:
// 210 GFLOP (32 trees of 17 to 33 nodes over 16000 bf16 tokens of four groups) in 344 us (358),
// 610 TFLOP/s.
//
// p is rounded to bf16 once, as the operand of the second product, by at most 2^-8 of itself;
// m, l and O stay in 32 bits and l sums the unrounded p.  That is a choice, the same as in
// kr_attn.hpp: outputs of random values are off by 0.0021 (the trees) to 0.0022 (the batch) of
// their norm, where their own rounding to bf16 alone makes 0.0017.  With the rest of p as a
// second operand they are off by 0.0017 and 0.0018 (the batch's own part still rounds its p),
// and whole calls take 309 instead of 285 us for the batch and 493 instead of 420 for the trees.
//
// Inside a wave the steps are laid side by side: a block of 32 tokens is exponentiated
// while the next block's scores are computed, and its values meet their p a block later,
// while the maxima of the next one are taken.
//
// Few rows of a group (64 at most) would leave six of the eight waves idle; then four waves share
// 64 rows, two and two with half of the tokens each.
//
// K and V tiles lie in LDS as they are in memory, bf16 rows (widened on the way from E4M3,
// exactly); V^T comes from a transposing read, four tokens of one head element per lane.
// 16-byte blocks of K at an index xor'ed with the token, 32-byte ones of V, so that neither
// read meets a bank twice.
//
// The work of all groups is one line of steps (row tile, kv head, 64 tokens), cut into 256
// equal pieces whatever the lengths are; a piece leaves a part (m, l, O) in fp32 for every
// unit that it meets, one or two mostly, and the rows' own kernel joins them.
#pragma once

#include "kr_share.hpp"

namespace svd {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kSharedTile = 64;      // tokens

// NW waves of 32 rows, WT of them with the same rows and other tokens.
template <int D, int NW, int WT>
struct SharedShape {
  static constexpr int kBlock = 64 * NW;
  static constexpr int M = NW / WT * 32;                 // rows of a workgroup
  static constexpr int SUB = 2 / WT;                     // blocks of 32 tokens per wave and tile
  static constexpr int NB = SUB == 2 ? 3 : 4;            // tiles in LDS
  static constexpr int kTile = kSharedTile * D * 2;      // bytes of K, or of V
  static constexpr int kJoin = WT > 1 ? WT * M * (D + 4) * 4 : 0;
  static constexpr int kLds = 2 * NB * kTile > kJoin ? 2 * NB * kTile : kJoin;
};

__device__ __forceinline__ f32x16 mfma32(const vec16 &a, const vec16 &b, const f32x16 &c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// The other half's value of the same row.
__device__ __forceinline__ float half_max(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

// How scores become base-2 logarithms: scaled; capped; or scaled or capped, as the call says,
// and less what the distance takes.
enum SharedScores { kPlain = 0, kCapped = 1, kSloped = 2 };

// The order in which a stretch of code issues: N times two products, `valu` vector
// instructions beside them, and the LDS reads of the products three turns later.
template <int N, int kReads, int kValu>
__device__ __forceinline__ void beside_products() {
  __builtin_amdgcn_sched_group_barrier(0x100, 3 * kReads, 0);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, kValu, 0);
    if (i + 3 < N) __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
  }
}

template <int D, bool kE4M3, int NW, int WT, int kScores>
__global__ __launch_bounds__(64 * NW, NW / 4) void kr_shared_attention(CacheView cv, AttnArgs a,
                                                                       int64_t G, float *part_o,
                                                                       float *part_ms) {
  using Shape = SharedShape<D, NW, WT>;
  constexpr int kBlock = Shape::kBlock;
  constexpr bool kShape = kScores != kPlain;
  constexpr int M = Shape::M, SUB = Shape::SUB, NB = Shape::NB;
  constexpr int TK = kSharedTile, ST = D / 16, DT = D / 32;
  constexpr int RowB = D * 2;                         // bytes of a row in LDS
  constexpr int E = kE4M3 ? 16 : 8;                   // elements of a 16-byte load
  constexpr int PC = D / E;                           // loads of a token
  constexpr int L = TK * PC > kBlock ? TK * PC / kBlock : 1;  // loads of a thread, of K and of V
  constexpr int TL = kBlock / PC;                     // tokens of a round of loads
  static_assert(64 / PC <= 16, "a wave's tokens are in one page");
  __shared__ __align__(16) unsigned char lds[Shape::kLds];
  __shared__ float lds_ms[WT > 1 ? WT : 1][WT > 1 ? M : 1][2];
  unsigned char *const ldk = lds, *const ldv = lds + NB * Shape::kTile;

  const int tid = threadIdx.x, lane = tid & 63, n = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wq = wave / WT, wt = wave % WT;
  // neighbouring pieces, which read the same keys and values, on one XCD
  const int64_t piece = (int64_t)(blockIdx.x & 7) * (kShareWorkgroups / 8) + (blockIdx.x >> 3);
  const int64_t total = a.cut->total, per = a.cut->per;
  const int64_t end = min((piece + 1) * per, total);
  const int Hq = cv.Hkv * a.group;

  // where a lane reads: keys of token n, values of four tokens and one element
  const int kx = D == 128 ? n & 15 : (n >> 1) & 7;
  const int k_at = n * RowB + ((half ^ (kx & 1)) << 4) + ((kx & ~1) << 4);
  const int vi = lane & 15, vt = 4 * half + (vi >> 2);  // place among 16 lanes, token
  const int vx = D == 128 ? vt & 7 : (vt >> 1) & 3;
  int v_at[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i)
    v_at[i] = vt * RowB + (((2 * i + ((lane >> 4) & 1)) ^ vx) << 5) + ((vi & 3) << 3);
  // where a thread writes, and what it loads: piece tid % PC of token tid / PC + round * TL
  const int s_tok = tid / PC % TK, s_pc = tid % PC;
  const bool loads = TK * PC >= kBlock || tid < TK * PC;
  const uint32_t in_page = (1u << cv.page_shift) - 1;
  constexpr uint32_t Row = kE4M3 ? D : 2 * D;  // bytes of a cached row
  const uint32_t page_rows = (uint32_t)cv.Hkv << cv.page_shift;

  for (int64_t pos = piece * per; pos < end;) {
    // the group of this step: the last one that begins at or before it and has steps
    int64_t gi = 0;
    for (int64_t g0 = 0; g0 < G; g0 += 64) {
      const int64_t i = g0 + lane;
      const bool there = i < G && a.groups[min(i, G - 1)].tokens > 0 &&
                         a.groups[min(i, G - 1)].step0 <= pos;
      const unsigned long long who = __ballot(there);
      if (who) gi = g0 + 63 - __builtin_clzll(who);
    }
    gi = __builtin_amdgcn_readfirstlane((int)gi);
    const ShareGroup g = a.groups[gi];
    const int64_t rel = pos - g.step0;
    const int unit = __builtin_amdgcn_readfirstlane((int)(rel / g.steps));
    const int t_lo = __builtin_amdgcn_readfirstlane((int)(rel % g.steps));
    const int t_hi = (int)min((int64_t)g.steps, t_lo + (end - pos));
    const int h = unit / g.tiles, r_lo = unit % g.tiles * M;
    const int rows = g.nodes * a.group;
    const int64_t slot = (int64_t)g.unit0 + unit + piece;
    const int32_t *const list = a.nodes + (int64_t)g.lo * a.T;
    const int32_t *const table = a.table + (int64_t)g.first * cv.max_pages;
    const uint32_t head_row = (uint32_t)h << cv.page_shift;
    pos += t_hi - t_lo;

    vec16 qf[ST];
    const int r = min(r_lo + wq * 32 + n, rows - 1);
    const int64_t token = list[r / a.group];
    const int head = h * a.group + r % a.group;
    const uint16_t *q = a.q + token * a.q_stride + (int64_t)head * D + 8 * half;
#pragma unroll
    for (int i = 0; i < ST; ++i) qf[i] = *reinterpret_cast<const vec16 *>(q + 16 * i);
    int at_row = 0;
    float slope = 0.0f;
    if constexpr (kScores == kSloped) {
      at_row = a.ctx_len[token / a.T] + (a.depth ? a.depth[token] : (int)(token % a.T));
      slope = a.slopes[head] * 1.4426950408889634f;
    }

    vec16 rk[L], rv[L];
    uint32_t sk[L], sv[L];
    int ok = 0, pages[L];
    // the table's entries for a tile go out a tile before its loads, which wait for them
    auto load_pages = [&](int tile) {
#pragma unroll
      for (int j = 0; j < L; ++j) {
        const uint32_t p = (uint32_t)min(tile, t_hi - 1) * TK + j * TL + s_tok;
        pages[j] = table[__builtin_amdgcn_readfirstlane(p >> cv.page_shift)];
      }
    };
    auto load_tile = [&](int tile) {  // behind the last tile: that one again
      ok = 0;
#pragma unroll
      for (int j = 0; j < L; ++j) {
        const uint32_t p = (uint32_t)min(tile, t_hi - 1) * TK + j * TL + s_tok;
        const int pg = pages[j];
        const bool good = (uint32_t)pg < (uint32_t)cv.n_pages;
        ok |= good << j;
        const uint32_t at = head_row + (p & in_page);
        const uint64_t row = (uint64_t)(good ? pg : 0) * page_rows;
        rk[j] = *reinterpret_cast<const vec16 *>(cv.k + row * Row + (at * Row + s_pc * 16));
        rv[j] = *reinterpret_cast<const vec16 *>(cv.v + row * Row + (at * Row + s_pc * 16));
        if constexpr (kE4M3) {
          sk[j] = cv.k_scale[row + at];
          sv[j] = cv.v_scale[row + at];
        }
      }
      load_pages(tile + 1);
    };
    auto store_tile = [&](int buf) {
      if (!loads) return;
#pragma unroll
      for (int j = 0; j < L; ++j) {
        const int tok = j * TL + s_tok;
        const int kt = D == 128 ? tok & 15 : (tok >> 1) & 7, vt_ = D == 128 ? tok & 7 : (tok >> 1) & 3;
        unsigned char *const pk = ldk + buf * Shape::kTile + tok * RowB;
        unsigned char *const pv = ldv + buf * Shape::kTile + tok * RowB;
        // a token without a page: NaN keys, so that every row is NaN
        const bool good = (ok >> j) & 1;
#pragma unroll
        for (int i = 0; i < (kE4M3 ? 2 : 1); ++i) {
          vec16 k, v;
          if constexpr (kE4M3) {
            const float fk = scale_factor(sk[j]), fv = scale_factor(sv[j]);
            const uint32_t x = i ? rk[j].z : rk[j].x, y = i ? rk[j].w : rk[j].y;
            const uint32_t z = i ? rv[j].z : rv[j].x, w = i ? rv[j].w : rv[j].y;
            k = vec16{widen2<false>(x, fk), widen2<true>(x, fk), widen2<false>(y, fk),
                      widen2<true>(y, fk)};
            v = vec16{widen2<false>(z, fv), widen2<true>(z, fv), widen2<false>(w, fv),
                      widen2<true>(w, fv)};
          } else {
            k = rk[j];
            v = rv[j];
          }
          if (!good) {
            k = vec16{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
            v = vec16{0, 0, 0, 0};
          }
          const int blk = s_pc * (E / 8) + i;
          *reinterpret_cast<vec16 *>(pk + ((blk ^ kt) << 4)) = k;
          *reinterpret_cast<vec16 *>(pv + (((blk >> 1) ^ vt_) << 5) + ((blk & 1) << 4)) = v;
        }
      }
    };

    f32x16 o[DT], sc;
    float base = kNegInf, l = 0.0f;
    vec16 pf[2];
#pragma unroll
    for (int i = 0; i < DT; ++i) o[i] = f32x16{};
    // the scores of a block of 32 tokens; a block's values with its p
    auto scores = [&](int buf, int sub) {
      const unsigned char *const p = ldk + buf * Shape::kTile + sub * 32 * RowB;
      f32x16 s = {};
#pragma unroll
      for (int i = 0; i < ST; ++i) {
        const vec16 kf = *reinterpret_cast<const vec16 *>(p + (k_at ^ (i << 5)));
        s = mfma32(kf, qf[i], s);
      }
      sc = s;
    };
    auto values = [&](int buf, int sub) {
      const unsigned char *const p = ldv + buf * Shape::kTile + sub * 32 * RowB;
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int i = 0; i < DT; ++i) {
          typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
          const unsigned char *const q = p + w * 16 * RowB + v_at[i];
          const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)q);
          const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(q + 8 * RowB));
          const u32x2 x2 = __builtin_bit_cast(u32x2, x), y2 = __builtin_bit_cast(u32x2, y);
          const vec16 vf = {x2.x, x2.y, y2.x, y2.y};
          o[i] = mfma32(vf, pf[w], o[i]);
        }
    };
    const float cs = kShape ? 1.0f : a.c;
    auto shape = [&](int tile, int sub) {
      const int p0 = tile * TK + sub * 32 + 4 * half;
      if (kScores == kCapped || a.cap_in > 0.0f) {
#pragma unroll
        for (int r = 0; r < 16; ++r) sc[r] = capped(sc[r], a.cap_in, a.cap_out);
      } else {
        sc *= a.c;
      }
      if constexpr (kScores == kSloped) {
        const float from = (float)(p0 - at_row);
#pragma unroll
        for (int r = 0; r < 16; ++r)
          sc[r] = __builtin_fmaf(slope, from + (float)(8 * (r / 4) + r % 4), sc[r]);
      }
    };
    // A block of 32 tokens: the values of the block before (from vb) beside this one's maxima,
    // the next one's scores (from kb) beside this one's exponentials.  The exponent moves
    // when a score passes it by 2^8, so most blocks rescale nothing.
    auto block = [&](auto with_values, int tile, int sub, int vb, int vsub, int kb, int ksub) {
      if constexpr (with_values.value) values(vb, vsub);
      if constexpr (kShape) shape(tile, sub);
      float mx = sc[0];
#pragma unroll
      for (int r = 1; r < 16; ++r) mx = fmaxf(mx, sc[r]);
      const float next = half_max(mx) * cs;
      const bool up = next > base + 8.0f;
      // vector instructions beside two products: those of the shape and the maxima
      constexpr int kOps = kScores == kPlain ? 4 : kScores == kCapped ? 24 : 12;
      if constexpr (with_values.value) beside_products<DT, 4, kOps>();
      if (__any(up)) {
        const float f = up ? fast_exp2(base - next) : 1.0f;
        l *= f;
#pragma unroll
        for (int i = 0; i < DT; ++i) o[i] *= f;
        base = up ? next : base;
      }
      f32x16 p = sc;
      scores(kb, ksub);
      const float less = base == kNegInf ? 0.0f : base;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        p[r] = fast_exp2(__builtin_fmaf(p[r], cs, -less));
        l += p[r];
      }
#pragma unroll
      for (int w = 0; w < 2; ++w)
        pf[w] = vec16{pack_bf16(p[8 * w], p[8 * w + 1]),
                      pack_bf16(p[8 * w + 2], p[8 * w + 3]),
                      pack_bf16(p[8 * w + 4], p[8 * w + 5]),
                      pack_bf16(p[8 * w + 6], p[8 * w + 7])};
      beside_products<ST / 2, 2, 128 / ST>();
    };

    __syncthreads();  // the piece before is done with LDS
    load_pages(t_lo);
    load_tile(t_lo);
    store_tile(0);
    load_tile(t_lo + 1);
    __syncthreads();
    scores(0, SUB == 2 ? 0 : wt);
    // Behind the last tile there are scores of whatever LDS holds, which nothing uses.
    int buf = 0, last = 0;  // where this tile is, and the one before
    auto tile_of = [&](auto with_values, int tile) {
      const int next = buf + 1 == NB ? 0 : buf + 1;
      store_tile(next);
      load_tile(tile + 2);
      if constexpr (SUB == 2) {
        block(with_values, tile, 0, last, 1, buf, 1);
        __syncthreads();  // the next tile is there, and the last one's values are done with
        block(std::true_type{}, tile, 1, buf, 0, next, 0);
      } else {
        __syncthreads();
        block(with_values, tile, wt, last, wt, next, wt);
      }
      last = buf;
      buf = next;
    };
    tile_of(std::false_type{}, t_lo);
    for (int tile = t_lo + 1; tile < t_hi; ++tile) tile_of(std::true_type{}, tile);
    values(last, SUB == 2 ? 1 : wt);

    l += __shfl_xor(l, 32, 64);
    if constexpr (WT == 1) {
      const int R = wq * 32 + n;
      const int64_t at = slot * M + R;
      if (r_lo + R < rows) {
        if (half == 0) {
          part_ms[2 * at] = base;
          part_ms[2 * at + 1] = l;
        }
        float *const to = part_o + at * D + 4 * half;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4 *>(to + 32 * i + 8 * q) =
                f32x4{o[i][4 * q], o[i][4 * q + 1], o[i][4 * q + 2], o[i][4 * q + 3]};
      }
    } else {
      // the waves that split the tokens join over the largest exponent
      __syncthreads();
      float (*lo)[M][D + 4] = reinterpret_cast<float (*)[M][D + 4]>(lds);
      const int R = wq * 32 + n;
      if (half == 0) {
        lds_ms[wt][R][0] = base;
        lds_ms[wt][R][1] = l;
      }
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<f32x4 *>(&lo[wt][R][32 * i + 8 * q + 4 * half]) =
              f32x4{o[i][4 * q], o[i][4 * q + 1], o[i][4 * q + 2], o[i][4 * q + 3]};
      __syncthreads();
      for (int i = tid; i < M * (D / 4); i += kBlock) {
        const int R = i / (D / 4), d = i % (D / 4) * 4;
        if (r_lo + R >= rows) break;
        float mm = kNegInf, ll = 0.0f;
#pragma unroll
        for (int w = 0; w < WT; ++w) mm = fmaxf(mm, lds_ms[w][R][0]);
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < WT; ++w) {
          const float f = part_factor(lds_ms[w][R][0], lds_ms[w][R][1], mm);
          ll += lds_ms[w][R][1] * f;
          x += *reinterpret_cast<const f32x4 *>(&lo[w][R][d]) * f;
        }
        const int64_t at = slot * M + R;
        *reinterpret_cast<f32x4 *>(part_o + at * D + d) = x;
        if (d == 0) {
          part_ms[2 * at] = mm;
          part_ms[2 * at + 1] = ll;
        }
      }
    }
  }
}

}  // namespace svd
