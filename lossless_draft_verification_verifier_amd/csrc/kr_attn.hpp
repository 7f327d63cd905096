// kr_attn.hpp -- attention of a draft tree over the paged cache.
//
// Row r = t * group + i of kv head h is query head h * group + i of node t; all
// rows of a (prefix, kv head) read the same keys and values.  With the running
// maximum m and sum l of the softmax, per 32 cached tokens:
//   S^T = K Q^T         v_mfma_f32_16x16x32_bf16, tokens x rows
//   p = exp2(S c - m c), c = scale * log2(e)
//   O^T += V^T P^T      the same instruction, head dimension x rows
// In the transposed products a lane keeps one row (lane % 16) throughout: the
// maximum over tokens is in-lane plus two shuffles, the rescaling of O is a
// per-lane factor, and the p that the first product leaves in a lane are the
// operand the second one wants there, so p never crosses lanes.
//
// A workgroup takes up to 16 * NT * WQ rows and walks tiles of TK tokens, written to
// LDS once for all rows: widened from E4M3 to bf16 with the row's power of two (by the
// conversion instruction; exact down to 2^-124), and V transposed.  WQ waves split the
// rows, and where these are few, WT waves split the tile's tokens and merge at the end.
// One barrier per tile.  LDS rows hold 16-byte blocks at an index xor'ed with the row,
// so that 16 lanes reading 16 rows touch all banks.  The 8-byte stores of V^T do not:
// lanes of different elements meet in a block, and of all LDS cycles 39 % (the 9-node
// batch below) and 31 % (the trees) are bank conflicts.
//   - Up to 64 rows (NT = 1) the cache's bytes are what counts: 4 waves of their own
//     keep the next PF tiles on their way in registers and write one to LDS while
//     the others compute the one before, two workgroups per CU.  Against one kind of wave
//     with the next tile in registers, 256 requests of 9 nodes over 1 to 4096 E4M3
//     tokens: 360 -> 293 us.
//   - With more rows (NT = 2) the products are: all 8 waves compute, 32 rows each, and
//     bring keys or values, the two waves of a SIMD at opposite ends of a step.
// p is rounded to bf16 once, as the operand of the second product, by at most 2^-8 of
// itself; m, l and O stay in 32 bits and l sums the unrounded p.  The rounding is a
// choice: with the rest of p as a second bf16 operand the outputs' error is their own
// rounding alone, root mean square 4.0e-4 instead of 5.3e-4 (9-node batch below, outputs
// of 0.24; 1.3e-5 instead of 1.9e-5 for the trees, of 0.008), but the second product
// and the packing double: 297 -> 325 us, 363 -> 456 for the trees, 56 -> 62 for 24
// requests of 33 nodes.  An output is rounded to bf16 in any case, and the errors of many
// tokens' p average out, so one operand is kept.
//
// Bounds, on one MI355X.  The 9-node batch above: 1.12 GB in 293 us, 3.8 TB/s; the
// tiles alone, nothing computed, take 246 us, a copy of as many bytes 230, and at the
// rate of a plain read (6.9 TB/s) they would take 163.  Trees of 65 to 129 nodes over
// 30000 bf16 tokens, 4 requests: 200 GFLOP in 363 us, 550 TFLOP/s; the matrix units are
// busy for a quarter of that and the vector units for a third.  Two things are left.
// Rows are dealt to workgroups by T, not by a prefix's own nodes: these prefixes have
// rows for 51 of the 80 waves they hold.  And inside a tile a wave's scores, maxima,
// exponentials and second product depend on each other, with two waves per SIMD all
// that the registers allow.
//
// The tiles of a prefix are split evenly over S workgroups when there are few
// (prefix, head) pairs; kr_attn_join merges the S parts.
#pragma once

#include <type_traits>

#include "kr_cache.hpp"
#include "kr_tree.hpp"
#include "svd_device.hpp"

namespace svd {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef vec16 u32x4;

constexpr int kAttnLoaders = 256;   // threads that bring tiles to LDS
constexpr int kAttnJoinBlock = 256;
constexpr int kAttnMaxSplits = 64;

// Sequences lo .. hi - 1 of a batch whose first `tokens` cached tokens are in the same pages,
// those of sequence `first`.  tokens is a multiple of kShareTokens.  Their rows are cut into
// tiles of m_rows; a unit is a tile of one kv head, head by head, `steps` tiles of tokens
// long, and the units of all groups, one behind the other, are one line of steps.
constexpr int kShareTokens = 128;
struct ShareGroup {
  int32_t lo, hi, first, tokens;
  int32_t nodes;            // nodes in use of its sequences, listed from lo * T on
  int32_t tiles, steps;     // row tiles; steps of a unit
  int32_t unit0;            // its first unit, and where that begins on the line
  int64_t step0;
};
// Workgroup w takes steps w * per .. of the line, and leaves a part for each unit that it meets:
// part unit + w, in m_rows rows.
struct ShareCut {
  int64_t total, per;
};
struct ShareSeq {           // one sequence
  int32_t eff;              // tokens that the shared parts cover
  int32_t group, start;     // its group, and its first node's number there
  int32_t pad;
};

struct AttnArgs {
  const uint16_t *q;        // [B][T][Hq][D] bf16, q_stride elements between tokens
  int64_t q_stride;
  const int32_t *ctx_len, *n_nodes, *table;
  const uint32_t *anc;      // [B][T][W] or null: a chain
  int64_t room;             // positions of a sequence's pages
  int T, group, S, m_tiles, m_rows, units;  // units = B * Hkv * S
  float c;                  // scale * log2(e)
  uint16_t *out;            // [B][T][Hq][D]
  float *lse;               // [B][T][Hq] or null
  float *part_o;            // [S][B][T][Hq][D] when S > 1
  float *part_ms;           // [S][B][T][Hq][2]
  int64_t rows_all;         // B * T * Hq
  // scores that are capped or fall off with distance (kShaped), and shared prefixes
  float cap_in, cap_out;    // 2 log2(e) scale / cap and cap * log2(e); 0: no cap
  const float *slopes;      // [Hq] or null
  const int32_t *depth;     // [B][T] or null: a chain
  const ShareSeq *seqs;     // [B], or null: nothing is shared
  const ShareGroup *groups;
  const ShareCut *cut;
  const int32_t *nodes;     // [B][T] b * T + t of the groups' nodes
  const float *share_o;     // [parts][share_rows][D]
  const float *share_ms;    // [parts][share_rows][2]
  int share_rows;
};
struct AttnCall {
  CacheView cache;
  AttnArgs args;
};

__device__ __forceinline__ f32x4 mfma_bf16(const vec16 &a, const vec16 &b, const f32x4 &c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ float scale_factor(uint32_t byte) {  // of a byte from 1 to 254
  return __uint_as_float(byte << 23);
}

// two E4M3 codes of word w, times the power of two s, as bf16
template <bool kHigh>
__device__ __forceinline__ uint32_t widen2(uint32_t w, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, kHigh));
}

// The maximum over the 4 lanes that hold a row (lane % 16): two exchanges of half
// the lanes, which stay in the vector unit.
__device__ __forceinline__ float row_max(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t v = __float_as_uint(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
  const auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// What a part (exponent m, sum l) is scaled by under the common exponent mm.  A
// part without scores has l = 0; one whose scores were all NaN has no maximum
// either, and its NaN sum has to stay.
__device__ __forceinline__ float part_factor(float m, float l, float mm) {
  return m == kNegInf ? (l == 0.0f ? 0.0f : 1.0f) : fast_exp2(m - mm);
}

// cap * tanh(scale * z / cap) as a base-2 logarithm: tanh(x) = 1 - y, y = 2 / (1 + exp(2 x)).  It
// is off by at most 2^-21 of the cap.  In units of 2^-23 of it: the argument, rounded twice,
// 0.45 (its relative error times the largest |2 x| exp(2 x) / (1 + exp(2 x))^2 * 2); exp2 and rcp, one
// unit in the last place each, 0.5 and 1; 1 + e 1; `out` and the last sum, rounded once each,
// 0.5 and 0.5.
__device__ __forceinline__ float capped(float z, float in, float out) {
  return __builtin_fmaf(-2.0f * out, __builtin_amdgcn_rcpf(1.0f + fast_exp2(z * in)), out);
}

// Whether a prefix's lengths are out of range.
__device__ __forceinline__ bool attn_bad(int ctx, int nodes, int T, int64_t room) {
  return ctx < 0 || nodes < 0 || nodes > T || (int64_t)ctx + nodes > room;
}

// one element of a cached row
template <bool kE4M3, int D>
__device__ __forceinline__ float cache_element(const uint8_t *p, const uint8_t *scale, int64_t row,
                                               int d) {
  if constexpr (kE4M3)
    return __builtin_amdgcn_cvt_f32_fp8((uint32_t)p[row * D + d], 0) * pow2_of_scale(scale[row]);
  else
    return BF16::at(reinterpret_cast<const uint16_t *>(p) + row * D, d);
}

// 4 elements of an output row: o over its sum, and the row's log-sum.
template <int D>
__device__ __forceinline__ void attn_row_out(const AttnArgs &a, int64_t row, int d, f32x4 o, float m,
                                             float l, bool first) {
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a row that attends to nothing is 0
  u32x2 w;
  w.x = pack_bf16(o[0] * inv, o[1] * inv);
  w.y = pack_bf16(o[2] * inv, o[3] * inv);
  *reinterpret_cast<u32x2 *>(a.out + row * D + d) = w;
  if (first && a.lse)
    a.lse[row] = l == 0.0f ? kNegInf : (m + __log2f(l)) * 0.6931471805599453f;
}

// The shared parts of row (node t of sequence b, query head i of kv head h): `at` rows into the
// first of `n` parts.
struct ShareRow {
  int64_t at;
  int n;
};
__device__ __forceinline__ ShareRow share_row(const AttnArgs &a, int64_t b, int t, int i, int h) {
  const ShareSeq q = a.seqs[b];
  if (q.eff == 0) return ShareRow{0, 0};
  const ShareGroup g = a.groups[q.group];
  const int64_t R = (int64_t)(q.start + t) * a.group + i;
  const int64_t unit = (int64_t)h * g.tiles + R / a.share_rows;
  const int64_t s0 = g.step0 + unit * g.steps, per = a.cut->per;
  const int64_t w0 = s0 / per, w1 = (s0 + g.steps - 1) / per;
  return ShareRow{(g.unit0 + unit + w0) * a.share_rows + R % a.share_rows, (int)(w1 - w0) + 1};
}
// 4 elements of a row's own part (exponent m, sum l) joined by those of its shared parts, kAhead
// of them on their way at a time: one or two behind a long loop; where few rows made many parts,
// one per piece of the line that their unit meets, 256 at most (8 for a single token behind 1024
// shared ones, of 8 kv heads: 9.2 us with one on its way, 5.7 with eight).
template <int D, int kAhead>
__device__ __forceinline__ void share_join(const AttnArgs &a, const ShareRow &r, int d, f32x4 &o,
                                           float &m, float &l) {
  float mm = m;
#pragma unroll kAhead
  for (int s = 0; s < r.n; ++s)
    mm = fmaxf(mm, a.share_ms[2 * (r.at + (int64_t)s * a.share_rows)]);
  const float f = part_factor(m, l, mm);
  l *= f;
  o *= f;
#pragma unroll kAhead
  for (int s = 0; s < r.n; ++s) {
    const int64_t at = r.at + (int64_t)s * a.share_rows;
    const float ms = a.share_ms[2 * at], ls = a.share_ms[2 * at + 1];
    const float g = part_factor(ms, ls, mm);
    l += ls * g;
    o += *reinterpret_cast<const f32x4 *>(a.share_o + at * D + d) * g;
  }
  m = mm;
}

// 32 bits of node t's ancestors from bit i0 on; bits below 0 are context, which
// every row attends to.  words null: a chain.
__device__ __forceinline__ uint32_t allow_window(const uint32_t *words, int W, int t, int i0) {
  if (!words) {
    const int last = t - i0;  // tokens up to the node itself
    return last < 0 ? 0u : last >= 31 ? 0xffffffffu : (2u << last) - 1u;
  }
  if (i0 <= -32) return 0xffffffffu;
  if (i0 < 0) return (words[0] << -i0) | ((1u << -i0) - 1u);
  const int w = i0 >> 5, k = i0 & 31;
  const uint32_t lo = w < W ? words[w] : 0u;
  if (k == 0) return lo;
  const uint32_t hi = w + 1 < W ? words[w + 1] : 0u;
  return (lo >> k) | (hi << (32 - k));
}

template <int D, bool kE4M3, int NT, int WQ, int WT>
struct AttnShape {
  static constexpr int TK = 8192 / D;                 // tokens per tile: 32 KB of K and V
  static constexpr int M = 16 * NT * WQ;              // most rows per workgroup
  static constexpr int NC = WQ * WT;                  // computing waves
  static constexpr bool kRoles = NT == 1;             // loading waves of their own
  static constexpr int kBlock = 64 * NC + (kRoles ? kAttnLoaders : 0);
  static constexpr int PF = !kRoles ? 1 : kE4M3 ? 3 : 2;  // tiles on their way at a time
  static constexpr int kMinWaves = NT == 1 ? 4 : 2;   // per SIMD
  static constexpr int kTileBytes = 2 * TK * D * 2;
  static constexpr int kJoinBytes = WT * M * (D + 4) * 4;
  static constexpr int kLdsBytes = 2 * kTileBytes > kJoinBytes ? 2 * kTileBytes : kJoinBytes;
};

// How scores become base-2 logarithms: scaled; or capped, sloped or both, as the call says.
// Either way the tokens are those behind what a group shares, all of them without groups.
// Through the shaped form plain scores behind 2048 shared tokens take 184 us instead of 177;
// that one itself takes 345 for the batch above, capped and sloped, for 293 plain: the cap is
// an exponential and a reciprocal per score, at a quarter of the rate.
enum AttnForm { kTree = 0, kShaped = 1 };

template <int D, bool kE4M3, int NT, int WQ, int WT, int kForm>
__global__ __launch_bounds__((AttnShape<D, kE4M3, NT, WQ, WT>::kBlock),
                             (AttnShape<D, kE4M3, NT, WQ, WT>::kMinWaves))
void kr_tree_attention(AttnCall call) {
  const CacheView &cv = call.cache;
  const AttnArgs &a = call.args;
  constexpr bool kShape = kForm == kShaped;
  using Shape = AttnShape<D, kE4M3, NT, WQ, WT>;
  constexpr int TK = Shape::TK, M = Shape::M, PF = Shape::PF;
  constexpr bool kRoles = Shape::kRoles;
  constexpr int DT = D / 16, ST = D / 32;
  constexpr int KB = D / 8;               // 16-byte blocks of a key row in LDS
  constexpr int VB = TK / 8;              // 16-byte blocks of a row of V^T in LDS
  constexpr int TW = TK / WT;             // tokens of a wave
  constexpr int G = TW >= 64 ? 64 : 32;   // tokens per softmax step
  constexpr int KE = kE4M3 ? 16 : 8;      // key elements per 16-byte load
  constexpr int KL = TK * D / KE / kAttnLoaders;      // key loads per thread
  // values: one piece of 4 tokens x 8 elements per thread
  static_assert(KL >= 1 && TK * D == 32 * kAttnLoaders && TW % 32 == 0, "");
  static_assert(kRoles || Shape::kBlock == 2 * kAttnLoaders, "half of the waves bring keys, half values");
  __shared__ __align__(16) unsigned char lds[Shape::kLdsBytes];
  __shared__ float lds_ms[WT][M][2];
  __shared__ int lds_odd;                 // some value of a tile with nodes is not finite

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
  const int r_lo = mt * a.m_rows, r_hi = min(r_lo + a.m_rows, rows);  // this workgroup's rows
  if (r_lo >= r_hi) return;
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int W = (a.T + 31) / 32;
  const float nan = __uint_as_float(0x7fc00000u);
  const int total = bad ? 0 : ctx + nodes;
  // a sequence's room goes up to 2^31 - page: sums past its length are 64 bits
  const int all_tiles = (int)(((int64_t)total + TK - 1) / TK);
  const int first = a.seqs && !bad ? a.seqs[b].eff / TK : 0;
  const int per = (all_tiles - first + a.S - 1) / a.S;
  const int t_lo = first + s * per, t_hi = min(t_lo + per, all_tiles);

  __shared__ ShareRow lds_share[M];
  if (threadIdx.x == 0) lds_odd = 0;
  if (first && a.S == 1)
    for (int r = r_lo + (int)threadIdx.x; r < r_hi; r += Shape::kBlock)
      lds_share[r - r_lo] = share_row(a, b, r / a.group, r % a.group, h);
  __syncthreads();

  // the threads that bring a tile to LDS: the loading waves do keys and values,
  // without them waves 0 to 3 do values and waves 4 to 7 keys
  const int tid = kRoles ? (int)threadIdx.x - 64 * Shape::NC : (int)threadIdx.x & (kAttnLoaders - 1);
  const bool do_k = kRoles || wave >= kAttnLoaders / 64, do_v = kRoles || !do_k;
  // the table's entry for 16-token block `lane` of a tile.  It is looked at when the
  // tile is loaded, not here: that would wait for it
  const int32_t *table = a.table + b * cv.max_pages;
  const int blocks = (int)(((int64_t)total + 15) / 16);
  auto load_pages = [&](int tile) -> int {
    const int blk = tile * (TK / 16) + lane % (TK / 16);
    return table[min(blk, blocks - 1) >> (cv.page_shift - 4)];
  };
  const uint32_t in_page = (1u << cv.page_shift) - 1;
  constexpr uint32_t RB = kE4M3 ? D : 2 * D;  // bytes of a row
  const uint32_t page_rows = (uint32_t)cv.Hkv << cv.page_shift, head_row = (uint32_t)h << cv.page_shift;

  constexpr int VO = kRoles ? KL : 0;  // where values are held: with the keys, or in their place
  struct Staged {  // a thread's share of a tile on its way to LDS
    vec16 reg[VO + KL];
    uint32_t scale[VO ? KL + 1 : KL];
    int kok, vok;
  };
  // this thread's share of a tile: keys by 16 bytes, values by 4 tokens x 8 elements
  // pages: the table's entries for it, replaced by those of tile + PF.  Loads return
  // in order, so the entries go out before the tile's data: waiting for them must
  // not wait for that
  auto load_tile = [&](Staged &st, int tile, int &pages) {
    const int64_t p0 = (int64_t)tile * TK;
    // a token without a page reads page 0: no branch comes between the loads.  A
    // page's rows take less than 2^31 bytes, so a row's place in it is 32 bits
    st.kok = st.vok = 0;
    const uint32_t q0 = (uint32_t)p0;
    const int left = tile < t_hi ? (int)min((int64_t)TK, total - p0) : 0;
    int pk[KL];
#pragma unroll
    for (int j = 0; j < KL; ++j)
      pk[j] = __shfl(pages, (tid / (D / KE) + j * (kAttnLoaders / (D / KE))) / 16, 64);
    const int pv = __shfl(pages, tid / (D / 8) / 4, 64);  // 4 tokens, one page
    pages = load_pages(tile + PF);
    __builtin_amdgcn_sched_barrier(0);
    if (do_k) {
#pragma unroll
    for (int j = 0; j < KL; ++j) {
      const int tok = tid / (D / KE) + j * (kAttnLoaders / (D / KE)), ch = tid % (D / KE);
      const int pg = pk[j];
      const bool ok = tok < left && (uint32_t)pg < (uint32_t)cv.n_pages;
      const uint32_t at = head_row + ((q0 + tok) & in_page), p_ = ok ? pg : 0;
      st.kok |= ok << j;
      st.reg[j] = *reinterpret_cast<const vec16 *>(cv.k + (uint64_t)p_ * (page_rows * RB) +
                                                    (at * RB + ch * 16));
      if constexpr (kE4M3) st.scale[j] = *(cv.k_scale + (uint64_t)p_ * page_rows + at);
    }
    }
    if (do_v) {
      const int q = tid / (D / 8), ch = tid % (D / 8);
      const int pg = pv;
      const bool ok = 4 * q < left && (uint32_t)pg < (uint32_t)cv.n_pages;
      const uint32_t at = head_row + ((q0 + 4 * q) & in_page), p_ = ok ? pg : 0;
      st.vok = ok;
      const uint8_t *v = cv.v + (uint64_t)p_ * (page_rows * RB) + (at * RB + ch * (RB / D * 8));
      if constexpr (kE4M3) {
        st.scale[VO] = *reinterpret_cast<const uint32_t *>(cv.v_scale + (uint64_t)p_ * page_rows + at);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const u32x2 x = *reinterpret_cast<const u32x2 *>(v + 2 * i * RB);
          const u32x2 y = *reinterpret_cast<const u32x2 *>(v + (2 * i + 1) * RB);
          st.reg[VO + i] = vec16{x.x, x.y, y.x, y.y};
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) st.reg[VO + i] = *reinterpret_cast<const vec16 *>(v + i * RB);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // registers to LDS.  A token without a valid page gets NaN keys, so that every row
  // that attends to it is NaN; values behind the end are zero.
  auto store_tile = [&](const Staged &st, int tile) {
    const bool last = (int64_t)tile * TK + TK > ctx;  // holds nodes or the end
    vec16 *const lk = reinterpret_cast<vec16 *>(lds + ((tile - t_lo) & 1) * Shape::kTileBytes);
    unsigned char *const lv = lds + ((tile - t_lo) & 1) * Shape::kTileBytes + TK * D * 2;
    const int left = min((int64_t)TK, total - (int64_t)tile * TK);
    const bool gaps = __any(st.kok != (1 << KL) - 1);
    if (do_k) {
#pragma unroll
    for (int j = 0; j < KL; ++j) {
      const int tok = tid / (D / KE) + j * (kAttnLoaders / (D / KE)), ch = tid % (D / KE);
      vec16 w[KE / 8];
      if constexpr (kE4M3) {
        const float sc = scale_factor(st.scale[j]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t x = i ? st.reg[j].z : st.reg[j].x, y = i ? st.reg[j].w : st.reg[j].y;
          w[i] = vec16{widen2<false>(x, sc), widen2<true>(x, sc), widen2<false>(y, sc),
                       widen2<true>(y, sc)};
        }
      } else {
        w[0] = st.reg[j];
      }
      if (gaps && !((st.kok >> j) & 1)) {
#pragma unroll
        for (int i = 0; i < KE / 8; ++i)
          w[i] = vec16{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
      }
#pragma unroll
      for (int i = 0; i < KE / 8; ++i)
        lk[tok * KB + ((ch * (KE / 8) + i) ^ (tok & (KB - 1)))] = w[i];
    }
    }
    bool odd = false;
    if (do_v) {
      const int q = tid / (D / 8), ch = tid % (D / 8);
      uint32_t x[4][4];  // token, pair of neighbouring elements
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kE4M3) {
          const float sc = scale_factor((st.scale[VO] >> (8 * i)) & 255);
          const uint32_t u = st.reg[VO + i / 2][2 * (i & 1)], v = st.reg[VO + i / 2][2 * (i & 1) + 1];
          x[i][0] = widen2<false>(u, sc);
          x[i][1] = widen2<true>(u, sc);
          x[i][2] = widen2<false>(v, sc);
          x[i][3] = widen2<true>(v, sc);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[i][e] = st.reg[VO + i][e];
        }
      }
      if (last) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool there = 4 * q + i < left && st.vok;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (!there) x[i][e] = 0;
            // 0 * NaN is NaN: values that are not finite stay out of the product
            // and join the rows that attend to them at the end
            if ((x[i][e] & 0x7f80u) == 0x7f80u) {
              odd = true;
              x[i][e] &= 0xffff0000u;
            }
            if ((x[i][e] & 0x7f800000u) == 0x7f800000u) {
              odd = true;
              x[i][e] &= 0x0000ffffu;
            }
          }
        }
      }
      // tokens 4 g .. 4 g + 3 and 16 + 4 g .. of a group of 32 side by side: the
      // order in which the first product leaves p
      const int blk = (q / 8) * 4 + (q & 3), half = (q >> 2) & 1;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = ch * 8 + e;
        const uint32_t sel = (e & 1) ? 0x07060302u : 0x05040100u;
        const u32x2 w = {__builtin_amdgcn_perm(x[1][e / 2], x[0][e / 2], sel),
                         __builtin_amdgcn_perm(x[3][e / 2], x[2][e / 2], sel)};
        *reinterpret_cast<u32x2 *>(lv + d * (TK * 2) + ((blk ^ ((d / DT) & (VB - 1))) << 4) +
                                   half * 8) = w;
      }
    }
    if (odd) lds_odd = 1;
  };

  // the waves that compute: their rows, a loop over the tiles, the parts to LDS
  auto compute = [&](auto &&before, auto &&begin, auto &&end) {
  const int wq = wave % WQ, wt = wave / WQ;
  vec16 qf[NT][ST];
  int node[NT], pos[NT];  // a row's node, and its position where scores fall off with distance
  float slope[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = min(r_lo + (wq * NT + t) * 16 + n, r_hi - 1);
    node[t] = r / a.group;
    const uint16_t *q = a.q + (b * a.T + node[t]) * a.q_stride +
                        (int64_t)(h * a.group + r % a.group) * D;
    if constexpr (kShape) {
      pos[t] = 0;
      slope[t] = 0.0f;
      if (a.slopes) {
        pos[t] = ctx + (a.depth ? a.depth[b * a.T + node[t]] : node[t]);
        slope[t] = a.slopes[h * a.group + r % a.group] * 1.4426950408889634f;
      }
    }
#pragma unroll
    for (int i = 0; i < ST; ++i) qf[t][i] = *reinterpret_cast<const vec16 *>(q + 32 * i + 8 * g);
  }
  // rows of this wave that exist
  const bool active = r_lo + wq * NT * 16 < r_hi;
  f32x4 o[NT][DT];
  float base[NT], l[NT];  // base: the exponent that l and o are held over
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    base[t] = kNegInf;
    l[t] = 0.0f;
#pragma unroll
    for (int i = 0; i < DT; ++i) o[t][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  const float cs = kShape ? 1.0f : a.c;  // shaped scores are base-2 logarithms already
  const int steps = (t_hi - t_lo + PF - 1) / PF * PF;  // as the loading waves take
  if (t_lo < t_hi) before();
  for (int tile = t_lo; tile < t_lo + steps; ++tile) {
    const int64_t p0 = (int64_t)tile * TK;
    const bool last = p0 + TK > ctx;  // holds nodes or the end
    const vec16 *const lk =
        reinterpret_cast<const vec16 *>(lds + ((tile - t_lo) & 1) * Shape::kTileBytes);
    const unsigned char *const lv = lds + ((tile - t_lo) & 1) * Shape::kTileBytes + TK * D * 2;
    begin(tile);
    if (active && tile < t_hi) {
#pragma unroll
      for (int g0 = 0; g0 < TW; g0 += G) {
        const int k0 = wt * TW + g0;  // first token of the step within the tile
        f32x4 sc[NT][G / 16];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int u = 0; u < G / 16; ++u) sc[t][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < ST; ++i)
#pragma unroll
          for (int u = 0; u < G / 16; ++u) {
            const int tok = k0 + 16 * u + n;
            const vec16 kf = lk[tok * KB + ((4 * i + g) ^ (tok & (KB - 1)))];
#pragma unroll
            for (int t = 0; t < NT; ++t) sc[t][u] = mfma_bf16(kf, qf[t][i], sc[t][u]);
          }
        if constexpr (kShape) {
          // to base-2 logarithms: capped, then less what the distance takes
          if (a.cap_in > 0.0f) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int u = 0; u < G / 16; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r) sc[t][u][r] = capped(sc[t][u][r], a.cap_in, a.cap_out);
          } else {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int u = 0; u < G / 16; ++u) sc[t][u] *= a.c;
          }
          if (a.slopes) {
            const int at = (int)(p0 + k0) + 4 * g;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const float from = (float)(at - pos[t]);
#pragma unroll
              for (int u = 0; u < G / 16; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  float far = from + (float)(16 * u + r);
                  if (last && a.depth) {
                    const int i = at + 16 * u + r - ctx;
                    if (i >= 0 && i < nodes) far = (float)(ctx + a.depth[b * a.T + i] - pos[t]);
                  }
                  sc[t][u][r] = __builtin_fmaf(slope[t], far, sc[t][u][r]);
                }
            }
          }
        }
        if (last) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int w = 0; w < G / 32; ++w) {
              const int64_t p = p0 + k0 + 32 * w;
              const int64_t left = total - p;
              uint32_t ok = left <= 0 ? 0u : left >= 32 ? 0xffffffffu : (1u << left) - 1u;
              ok &= allow_window(a.anc ? a.anc + (b * a.T + node[t]) * W : nullptr, W, node[t],
                                 (int)(p - ctx));
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  if (!((ok >> (16 * u + 4 * g + r)) & 1u)) sc[t][2 * w + u][r] = kNegInf;
            }
        }
        // the exponent moves when a score passes it by 2^8: p, l and o lose nothing to
        // a factor of at most 256, and most steps rescale nothing
        float next[NT];
        bool moves = false;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float mx = kNegInf;
#pragma unroll
          for (int u = 0; u < G / 16; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) mx = fmaxf(mx, sc[t][u][r]);
          next[t] = row_max(mx) * cs;
          moves |= next[t] > base[t] + 8.0f;
        }
        if (__any(moves)) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const bool move = next[t] > base[t] + 8.0f;
            const float f = move ? fast_exp2(base[t] - next[t]) : 1.0f;
            l[t] *= f;
#pragma unroll
            for (int i = 0; i < DT; ++i) o[t][i] *= f;
            base[t] = move ? next[t] : base[t];
          }
        }
        vec16 pf[NT][G / 32];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float sub = base[t] == kNegInf ? 0.0f : base[t];
#pragma unroll
          for (int u = 0; u < G / 16; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              sc[t][u][r] = fast_exp2(__builtin_fmaf(sc[t][u][r], cs, -sub));
              l[t] += sc[t][u][r];
            }
#pragma unroll
          for (int w = 0; w < G / 32; ++w)
            pf[t][w] = vec16{pack_bf16(sc[t][2 * w][0], sc[t][2 * w][1]),
                             pack_bf16(sc[t][2 * w][2], sc[t][2 * w][3]),
                             pack_bf16(sc[t][2 * w + 1][0], sc[t][2 * w + 1][1]),
                             pack_bf16(sc[t][2 * w + 1][2], sc[t][2 * w + 1][3])};
        }
#pragma unroll
        for (int w = 0; w < G / 32; ++w) {
          const int blk = (k0 / 32 + w) * 4 + g;
#pragma unroll
          for (int i = 0; i < DT; ++i) {
            const int d = DT * n + i;
            const vec16 vf = *reinterpret_cast<const vec16 *>(
                lv + d * (TK * 2) + ((blk ^ (n & (VB - 1))) << 4));
#pragma unroll
            for (int t = 0; t < NT; ++t) o[t][i] = mfma_bf16(vf, pf[t][w], o[t][i]);
          }
        }
      }
    }
    end(tile);
  }
  if (kRoles && t_lo < t_hi) __syncthreads();
  float (*lo)[M][D + 4] = reinterpret_cast<float (*)[M][D + 4]>(lds);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    l[t] += __shfl_xor(l[t], 16, 64);
    l[t] += __shfl_xor(l[t], 32, 64);
    const int R = (wq * NT + t) * 16 + n;
    if (g == 0) {
      lds_ms[wt][R][0] = base[t];
      lds_ms[wt][R][1] = bad ? nan : l[t];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < DT; i += 4)
        *reinterpret_cast<f32x4 *>(&lo[wt][R][DT * (4 * g + r) + i]) =
            f32x4{o[t][i][r], o[t][i + 1][r], o[t][i + 2][r], o[t][i + 3][r]};
  }
  };
  Staged st[PF];
  int pages[PF];
  if constexpr (kRoles) {
    if (wave < Shape::NC) {
      compute([] {}, [](int) { __syncthreads(); }, [](int) {});
    } else if (t_lo < t_hi) {
#pragma unroll
      for (int k = 0; k < PF; ++k) pages[k] = load_pages(t_lo + k);
#pragma unroll
      for (int k = 0; k < PF; ++k) load_tile(st[k], t_lo + k, pages[k]);
      for (int tile0 = t_lo; tile0 < t_hi; tile0 += PF)
#pragma unroll
        for (int k = 0; k < PF; ++k) {
          const int tile = tile0 + k;
          // the steps are a multiple of PF, and behind the last tile the loads read page 0:
          // with a way out between them, or one around the loads, the waits of the next
          // tile would have to wait for all that is on its way
          if (tile < t_hi) store_tile(st[k], tile);
          load_tile(st[k], tile + PF, pages[k]);
          __syncthreads();  // this tile is there, and the one before it is done with
        }
      __syncthreads();  // the last tile is done with
    }
  } else {
    auto bring = [&](int tile) {  // tile to LDS, the one after it on its way
      if (tile < t_hi) store_tile(st[0], tile);
      load_tile(st[0], tile + 1, pages[0]);
    };
    // the two waves of a SIMD (w and w + 4) bring the next tile one before and one
    // after they compute: one's products then run beside the other's exponentials
    compute(
        [&] {
          pages[0] = load_pages(t_lo);
          load_tile(st[0], t_lo, pages[0]);
          bring(t_lo);
          __syncthreads();
        },
        [&](int tile) {
          if (do_k) bring(tile + 1);
        },
        [&](int tile) {
          if (do_v) bring(tile + 1);
          __syncthreads();
        });
  }

  __syncthreads();  // the parts of all waves are there

  // What follows reads its arguments again: held in registers all the way, they spill the
  // loop's own scalars (68 of them, 90 with shaped scores).
  // The call is the kernel's one parameter, so its arguments begin with it.
  static_assert(std::is_same_v<decltype(&kr_tree_attention<D, kE4M3, NT, WQ, WT, kForm>),
                               void (*)(AttnCall)>, "the arguments are one AttnCall");
  typedef __attribute__((address_space(4))) const char *kernarg;
  kernarg late = (kernarg)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(late));
  const AttnCall &again = *(const AttnCall *)late;
  const CacheView &cz = again.cache;
  const AttnArgs &az = again.args;

  // one row's 4 elements from d on, its exponent and its sum
  auto put = [&](int R, int d, f32x4 x, float mm, float ll) {
    const int64_t row = (b * az.T + R / az.group) * Hq + h * az.group + R % az.group;
    if (az.S > 1) {
      const int64_t pr = (int64_t)s * az.rows_all + row;
      *reinterpret_cast<f32x4 *>(az.part_o + pr * D + d) = x;
      if (d == 0) {
        az.part_ms[2 * pr] = mm;
        az.part_ms[2 * pr + 1] = ll;
      }
    } else {
      // shared parts are there already: the row ends here
      if (first) share_join<D, 1>(az, lds_share[R - r_lo], d, x, mm, ll);
      attn_row_out<D>(az, row, d, x, mm, ll, d == 0);
    }
  };
  // what the tokens of this part whose values are not finite add to 4 elements
  auto odd_values = [&](int R, int d, f32x4 x, float mm) {
    const int nd = R / az.group;
    const uint16_t *q = az.q + (b * az.T + nd) * az.q_stride +
                        (int64_t)(h * az.group + R % az.group) * D;
    // from the first tile whose values were looked at: it can begin with context, which
    // every row attends to
    const int64_t lo = (int64_t)max(t_lo, ctx / TK) * TK;
    const int64_t hi = min((int64_t)t_hi * TK, (int64_t)total);
    for (int64_t p = lo; p < hi; ++p) {
      const int i = (int)(p - ctx);
      if (i >= 0 && (az.anc ? !((az.anc[(b * az.T + nd) * W + (i >> 5)] >> (i & 31)) & 1u) : i > nd))
        continue;
      const int64_t row = cache_row(cz, b, p, h);
      if (row < 0) continue;
      float v[4];
      bool odd = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = cache_element<kE4M3, D>(cz.v, cz.v_scale, row, d + e);
        odd |= !(fabsf(v[e]) < __builtin_huge_valf());
      }
      if (!odd) continue;
      float z = 0.0f;
      for (int e = 0; e < D; ++e)
        z += cache_element<kE4M3, D>(cz.k, cz.k_scale, row, e) * BF16::at(q, e);
      const float sub = mm == kNegInf ? 0.0f : mm;
      float pt;
      if constexpr (kShape) {
        z = az.cap_in > 0.0f ? capped(z, az.cap_in, az.cap_out) : z * az.c;
        if (az.slopes) {
          const int64_t token = b * az.T + nd;
          const int to = ctx + (az.depth ? az.depth[token] : nd);
          const int from = i >= 0 && az.depth ? ctx + az.depth[b * az.T + i] : (int)p;
          z = __builtin_fmaf(az.slopes[h * az.group + R % az.group] * 1.4426950408889634f,
                             (float)(from - to), z);
        }
        pt = fast_exp2(z - sub);
      } else {
        pt = fast_exp2(__builtin_fmaf(z, az.c, -sub));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!(fabsf(v[e]) < __builtin_huge_valf())) x[e] += pt * v[e];
    }
    return x;
  };
  // the waves that split the tokens join over the largest exponent
  const float (*lo)[M][D + 4] = reinterpret_cast<const float (*)[M][D + 4]>(lds);
  constexpr int V = D / 4;  // 16-byte pieces of a row
  for (int i = threadIdx.x; i < M * V; i += Shape::kBlock) {
    const int r = i / V, d = (i % V) * 4;
    if (r_lo + r >= r_hi) break;
    float mm = kNegInf, ll = 0.0f;
#pragma unroll
    for (int w = 0; w < WT; ++w) mm = fmaxf(mm, lds_ms[w][r][0]);
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < WT; ++w) {
      const float f = part_factor(lds_ms[w][r][0], lds_ms[w][r][1], mm);
      ll += lds_ms[w][r][1] * f;
      x += *reinterpret_cast<const f32x4 *>(&lo[w][r][d]) * f;
    }
    if (lds_odd) x = odd_values(r_lo + r, d, x, mm);
    put(r_lo + r, d, x, mm, ll);
  }
}

// The S parts of every row: D / 4 lanes per row.
template <int D>
__global__ __launch_bounds__(kAttnJoinBlock) void kr_attn_join(AttnArgs a, int Hq) {
  constexpr int L = D / 4;
  const int64_t row = (int64_t)blockIdx.x * (kAttnJoinBlock / L) + threadIdx.x / L;
  if (row >= a.rows_all) return;
  const int d = (threadIdx.x % L) * 4;
  const int64_t bt = row / Hq;
  const int64_t b = bt / a.T;
  const int nodes = a.n_nodes ? a.n_nodes[b] : a.T;
  // a prefix out of range wrote NaN parts for every row
  if (bt % a.T >= nodes && !attn_bad(a.ctx_len[b], nodes, a.T, a.room)) return;
  float m = kNegInf;
#pragma unroll 8
  for (int s = 0; s < a.S; ++s) m = fmaxf(m, a.part_ms[2 * (s * a.rows_all + row)]);
  float l = 0.0f;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
  for (int s = 0; s < a.S; ++s) {
    const int64_t pr = s * a.rows_all + row;
    const float ms = a.part_ms[2 * pr], ls = a.part_ms[2 * pr + 1];
    const float f = part_factor(ms, ls, m);
    l += ls * f;
    o += *reinterpret_cast<const f32x4 *>(a.part_o + pr * D + d) * f;
  }
  if (a.seqs) {
    const int h = (int)(row % Hq);
    const ShareRow r = share_row(a, b, (int)(bt % a.T), h % a.group, h / a.group);
    if (r.n) share_join<D, 8>(a, r, d, o, m, l);
  }
  attn_row_out<D>(a, row, d, o, m, l, d == 0);
}

}  // namespace svd
