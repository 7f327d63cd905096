// kr_share.hpp -- which tokens the sequences of a group have in common: those of the pages
// that all of their block tables begin with.
//
// One workgroup per group compares the tables of its sequences with the first one's, page
// by page; a sequence without rows, or with lengths out of range, constrains nothing and
// shares nothing.  What is shared is rounded down to kShareTokens, whole tiles of either
// head size; the rest is each sequence's own, like everything where fewer than two
// sequences share.  So a wrong grouping costs time and changes no result.
//
// Latency bounds it: a table entry is one load behind lengths, offsets and the first
// sequence.  A single group of 4 sequences takes 6 us, of 256 with 64 pages in reach 14
// (with four sequences of a wave on their way at a time instead of sixteen 18, with one 32).
#pragma once

#include "kr_attn.hpp"
#include "kr_pages.hpp"

namespace svd {

constexpr int kShareBlock = 1024;
constexpr int kShareWorkgroups = 256;  // of the attention: one per CU
constexpr int kShareMinSteps = 2;      // a workgroup takes at least as many, where there are

struct ShareArgs {
  const int32_t *off;       // [G + 1]
  const int32_t *ctx_len, *n_nodes, *table;
  int64_t B, G, room;
  int T, max_pages, page_shift, group, heads, m_rows, tile;
  ShareSeq *seqs;           // [B]
  int32_t *nodes;           // [B][T]
  ShareGroup *groups;       // [G]
  ShareCut *cut;
};

__device__ __forceinline__ void share_cut(ShareCut *cut, int64_t total) {
  cut->total = total;
  cut->per = max((total + kShareWorkgroups - 1) / kShareWorkgroups, (int64_t)kShareMinSteps);
}

__global__ __launch_bounds__(kShareBlock) void kr_share(ShareArgs a) {
  __shared__ int lo_ok, n_act, first, ctx_min, pages;
  __shared__ int wave_sum[kShareBlock / 64];
  __shared__ unsigned long long who[kShareBlock / 64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t g = blockIdx.x;
  if (threadIdx.x == 0) {
    lo_ok = 1;
    n_act = 0;
    first = 0x7fffffff;
    ctx_min = 0x7fffffff;
  }
  __syncthreads();
  bool ok = true;
  for (int64_t i = threadIdx.x; i <= a.G; i += kShareBlock) {
    const int x = a.off[i];
    ok &= x >= 0 && x <= a.B && (i == 0 || a.off[i - 1] <= x);
  }
  if (!ok) lo_ok = 0;
  __syncthreads();
  const bool valid = lo_ok;
  // offsets out of order: nothing is shared
  const int lo = valid ? a.off[g] : 0, hi = valid ? a.off[g + 1] : 0;
  auto active = [&](int b) {
    const int ctx = a.ctx_len[b], nodes = a.n_nodes ? a.n_nodes[b] : a.T;
    return !attn_bad(ctx, nodes, a.T, a.room) && nodes > 0;
  };
  for (int b = lo + (int)threadIdx.x; b < hi; b += kShareBlock)
    if (active(b)) {
      atomicAdd(&n_act, 1);
      atomicMin(&first, b);
      atomicMin(&ctx_min, a.ctx_len[b]);
    }
  __syncthreads();
  const int f = first, cols = n_act >= 2 ? ctx_min >> a.page_shift : 0;
  if (threadIdx.x == 0) pages = cols;
  __syncthreads();
  if (cols > 0) {
    // a wave has every 16th sequence, all of a stretch and 256 columns at a time
    constexpr int kInFlight = 16;
    const int32_t *const one = a.table + (int64_t)f * a.max_pages;
    for (int b0 = lo; b0 < hi; b0 += kShareBlock) {
      // who is compared, of this stretch of sequences
      const int mine = b0 + (int)threadIdx.x;
      const unsigned long long act = __ballot(mine < hi && mine != f && active(mine));
      if (lane == 0) who[w] = act;
      __syncthreads();
      // every thread takes the bound between two barriers with no change of it
      for (int c0 = 0, c_end = pages; c0 < c_end; c0 += 256) {
        __syncthreads();
        int at[4], want[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          at[i] = min(c0 + 64 * i + lane, cols - 1);
          want[i] = one[at[i]];
        }
        int least = cols;
        for (int k = w; k < kShareBlock && b0 + k < hi; k += kInFlight * (kShareBlock / 64)) {
          int got[kInFlight][4];
#pragma unroll
          for (int s = 0; s < kInFlight; ++s) {
            const int b = k + s * (kShareBlock / 64);
            const bool on = b < kShareBlock && b0 + b < hi && (who[b >> 6] >> (b & 63) & 1);
            const int32_t *const row = on ? a.table + (int64_t)(b0 + b) * a.max_pages : one;
#pragma unroll
            for (int i = 0; i < 4; ++i) got[s][i] = row[at[i]];
          }
#pragma unroll
          for (int s = 0; s < kInFlight; ++s)
#pragma unroll
            for (int i = 3; i >= 0; --i)
              if (got[s][i] != want[i]) least = min(least, at[i]);
        }
        if (least < cols) atomicMin(&pages, least);
        __syncthreads();
        c_end = pages;
      }
      __syncthreads();
    }
  }
  __syncthreads();
  const int tokens = (int)(((int64_t)pages << a.page_shift) / kShareTokens * kShareTokens);
  // inclusive sums over the workgroup, and the total
  auto scan = [&](int up, int &total) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int x = __shfl_up(up, off, 64);
      if (lane >= off) up += x;
    }
    if (lane == 63) wave_sum[w] = up;
    __syncthreads();
    total = 0;
    for (int k = 0; k < kShareBlock / 64; ++k) {
      if (k == w) up += total;
      total += wave_sum[k];
    }
    __syncthreads();
    return up;
  };
  // the nodes in use, one after another: rows that no node has are no workgroup's
  int listed = 0;
  for (int b0 = lo; b0 < hi; b0 += kShareBlock) {
    const int b = b0 + (int)threadIdx.x;
    int n = 0, total;
    if (b < hi && tokens && active(b)) n = a.n_nodes ? a.n_nodes[b] : a.T;
    const int from = listed + scan(n, total) - n;
    listed += total;
    if (b < hi) a.seqs[b] = ShareSeq{n ? tokens : 0, (int32_t)g, from, 0};
    for (int i = 0; i < n; ++i)
      a.nodes[(int64_t)lo * a.T + from + i] = (int32_t)((int64_t)b * a.T + i);
  }
  // sequences of no group
  const int64_t in_lo = valid ? a.off[0] : 0, in_hi = valid ? a.off[a.G] : 0;
  for (int64_t b = g + (int64_t)threadIdx.x * a.G; b < a.B; b += (int64_t)kShareBlock * a.G)
    if (b < in_lo || b >= in_hi) a.seqs[b] = ShareSeq{0, 0, 0, 0};
  if (threadIdx.x != 0) return;
  ShareGroup s;
  s.lo = lo;
  s.hi = hi;
  s.first = f;
  s.tokens = listed ? tokens : 0;
  s.nodes = listed;
  s.tiles = (int)(((int64_t)listed * a.group + a.m_rows - 1) / a.m_rows);
  s.steps = s.tokens / a.tile;
  s.unit0 = 0;
  s.step0 = 0;
  a.groups[g] = s;
  if (a.G == 1) share_cut(a.cut, (int64_t)s.tiles * a.heads * s.steps);
}

// The groups' places on the line, where there are several.
__global__ __launch_bounds__(kShareBlock) void kr_share_cut(ShareArgs a) {
  __shared__ int64_t lds[kShareBlock / 64][2];
  int64_t units = 0, steps = 0;  // before this chunk of groups
  for (int64_t i0 = 0; i0 < a.G; i0 += kShareBlock) {
    const int64_t i = i0 + threadIdx.x;
    int64_t u = 0, s = 0;
    if (i < a.G) {
      const ShareGroup g = a.groups[i];
      u = g.tokens ? (int64_t)g.tiles * a.heads : 0;
      s = u * g.steps;
    }
    int64_t upu = u, ups = s, tu, ts;
    block_scan2<kShareBlock>(upu, ups, tu, ts, lds);
    if (i < a.G) {
      a.groups[i].unit0 = (int32_t)(units + upu - u);
      a.groups[i].step0 = steps + ups - s;
    }
    units += tu;
    steps += ts;
  }
  if (threadIdx.x == 0) share_cut(a.cut, steps);
}

}  // namespace svd
