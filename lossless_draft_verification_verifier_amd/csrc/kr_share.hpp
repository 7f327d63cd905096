// kr_share.hpp -- which tokens the sequences of a group have in common: those of the pages
// that all of their block tables begin with.
//
// One workgroup per group compares the tables of its sequences with the first one's, page
// by page; a sequence without rows, or with lengths out of range, constrains nothing and
// shares nothing.  What is shared is rounded down to kShareTokens, whole tiles of either
// head size; the rest is each sequence's own, like everything where fewer than two
// sequences share.  So a wrong grouping costs time and changes no result.
#pragma once

#include "kr_attn.hpp"

namespace svd {

constexpr int kShareBlock = 1024;

struct ShareArgs {
  const int32_t *off;       // [G + 1]
  const int32_t *ctx_len, *n_nodes, *table;
  int64_t B, G, room;
  int T, max_pages, page_shift, group, m_rows, m_tiles;
  int32_t *eff;             // [B]
  ShareGroup *groups;       // [G]
  ShareTile *tiles;         // [m_tiles]
};

__global__ __launch_bounds__(kShareBlock) void kr_share(ShareArgs a) {
  __shared__ int lo_ok, n_act, first, ctx_min, pages;
  __shared__ int wave_sum[kShareBlock / 64];
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
    // entries of all tables, a run of columns per sequence
    const int64_t n = (int64_t)(hi - lo) * cols;
    int least = cols;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < n; i += kShareBlock) {
      const int b = lo + (int)(i / cols), c = (int)(i % cols);
      const bool same = a.table[(int64_t)b * a.max_pages + c] == a.table[(int64_t)f * a.max_pages + c];
      if (!same && c < least && active(b)) least = c;
    }
    if (least < cols) atomicMin(&pages, least);
  }
  __syncthreads();
  const int tokens = (int)(((int64_t)pages << a.page_shift) / kShareTokens * kShareTokens);
  if (threadIdx.x == 0) a.groups[g] = ShareGroup{lo, hi, f, tokens};
  for (int b = lo + (int)threadIdx.x; b < hi; b += kShareBlock)
    a.eff[b] = tokens && active(b) ? tokens : 0;
  // sequences of no group
  const int64_t in_lo = valid ? a.off[0] : 0, in_hi = valid ? a.off[a.G] : 0;
  for (int64_t b = g + (int64_t)threadIdx.x * a.G; b < a.B; b += (int64_t)kShareBlock * a.G)
    if (b < in_lo || b >= in_hi) a.eff[b] = 0;
  if (g != 0) return;
  // the workgroups' rows: m_rows of a group each
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int before = 0;
  for (int64_t i0 = 0; i0 < a.G; i0 += kShareBlock) {
    const int64_t i = i0 + threadIdx.x;
    int n = 0;
    if (i < a.G && valid)
      n = (int)(((int64_t)(a.off[i + 1] - a.off[i]) * a.T * a.group + a.m_rows - 1) / a.m_rows);
    int up = n;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int x = __shfl_up(up, off, 64);
      if (lane >= off) up += x;
    }
    if (lane == 63) wave_sum[w] = up;
    __syncthreads();
    int total = 0;
    for (int k = 0; k < kShareBlock / 64; ++k) {
      if (k == w) up += total;
      total += wave_sum[k];
    }
    for (int k = 0; k < n; ++k) {
      const int at = before + up - n + k;
      if (at < a.m_tiles) a.tiles[at] = ShareTile{(int32_t)i, k * a.m_rows};
    }
    before += total;
    __syncthreads();
  }
  for (int i = before + (int)threadIdx.x; i < a.m_tiles; i += kShareBlock)
    a.tiles[i] = ShareTile{-1, 0};
}

}  // namespace svd
