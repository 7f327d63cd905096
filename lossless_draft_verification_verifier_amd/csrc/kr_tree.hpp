// kr_tree.hpp -- the prefix tree of a prefix's K drafts.
//
// Drafts with a common prefix are scored by one verifier row per distinct
// prefix (the flattened draft tree of SpecDiff-2 appendix B.8).  With lcp(k', k)
// the common length of two drafts, draft k owns the positions from
// s_k = max_{k' < k} lcp(k', k) to its end: a run of consecutive nodes from
// base_k on.  The positions before s_k belong to the first draft par_k with
// lcp(par_k, k) = s_k, and so on up the chain of par, so a node's path is a
// few runs of consecutive node numbers and its ancestor words are ranges of
// bits: no walk over single nodes.
//
// Bound by latency: a call reads K*G tokens per prefix and its steps depend on
// each other, so one workgroup does a whole prefix.  8 drafts of 16 tokens: 4.6 us;
// 64 prefixes with 16 drafts of 32: 15.6 us (20.8 with 512 threads and a search for
// every word's owner instead of a table).  There the ancestor words are the largest
// part: 513 nodes of 17 words on 32 lanes each, and every word walks the chain of par by
// itself, one dependent read of LDS after another; without the walk a call takes less
// than the 11 us that its host side does.
#pragma once

#include "svd_device.hpp"

namespace svd {

constexpr int kTreeBlock = 1024;
constexpr int kTreeMaxK = 64;
constexpr int kTreeLdsTokens = 4096;  // drafts of at most this many tokens are staged in LDS
constexpr int kTreeMaxNodes = 4096;

// bits [lo, hi] of a bitmap that fall into word w
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int w) {
  const int a = max(lo - 32 * w, 0), b = min(hi - 32 * w, 31);
  if (a > b) return 0;
  return (0xffffffffu << a) & (0xffffffffu >> (31 - b));
}

// One workgroup per prefix; see svd_draft_tree for the arrays.
__global__ __launch_bounds__(kTreeBlock) void kr_draft_tree(
    const int32_t *__restrict__ drafts, const int32_t *__restrict__ root, int K, int G, int T,
    int W, int32_t *__restrict__ tokens, int32_t *__restrict__ parent,
    int32_t *__restrict__ depth, uint32_t *__restrict__ anc, int32_t *__restrict__ n_nodes,
    int32_t *__restrict__ p_index) {
  __shared__ int32_t tok[kTreeLdsTokens];
  __shared__ int lcp[kTreeMaxK][kTreeMaxK];
  __shared__ uint8_t owner[kTreeMaxNodes];  // the draft that owns a node
  __shared__ int len[kTreeMaxK], first[kTreeMaxK], base[kTreeMaxK + 1], par[kTreeMaxK];
  const int64_t b = blockIdx.x;
  const int tid = threadIdx.x;
  const int32_t *src = drafts + b * K * G;
  const bool staged = K * G <= kTreeLdsTokens;
  if (tid < K) len[tid] = G;
  __syncthreads();
  // a draft ends at its first negative token
  for (int i = tid; i < K * G; i += kTreeBlock) {
    const int32_t x = src[i];
    if (staged) tok[i] = x;
    if (x < 0) atomicMin(&len[i / G], i % G);
  }
  __syncthreads();
  // common lengths: a group of `gs` lanes compares gs positions of a pair at a time
  const int32_t *x = staged ? tok : src;
  int gs = 1;
  while (gs < G && gs < 64) gs *= 2;
  const int lane = tid & 63, sub = tid & (gs - 1);
  const uint64_t gmask = gs == 64 ? ~0ull : ((1ull << gs) - 1) << (lane & ~(gs - 1));
  for (int pair = tid / gs; pair < K * K; pair += kTreeBlock / gs) {
    const int a = pair / K, k = pair % K;
    if (a >= k) continue;
    const int n = min(len[a], len[k]);
    int common = n;
    for (int j0 = 0; j0 < n; j0 += gs) {
      const int j = j0 + sub;
      const bool differ = j < n && x[a * G + j] != x[k * G + j];
      const uint64_t hit = __ballot(differ) & gmask;
      if (hit) {
        common = j0 + (__ffsll((unsigned long long)hit) - 1) - (lane & ~(gs - 1));
        break;
      }
    }
    if (sub == 0) lcp[a][k] = common;
  }
  __syncthreads();
  if (tid < 64) {  // one lane per draft: its first own position, its parent draft, its first node
    int s = 0, p = -1, own = 0;
    if (tid < K) {
      for (int a = 0; a < tid; ++a)
        if (lcp[a][tid] > s) {
          s = lcp[a][tid];
          p = a;
        }
      first[tid] = s;
      par[tid] = p;
      own = len[tid] - s;
    }
    int sum = own;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int y = __shfl_up(sum, off, 64);
      if (tid >= off) sum += y;
    }
    if (tid < K) base[tid] = 1 + sum - own;
    if (tid == 63) base[K] = 1 + sum;
  }
  __syncthreads();
  const bool fits = base[K] <= T;
  const int n = fits ? base[K] : 0;
  if (tid == 0) n_nodes[b] = fits ? n : -1;
  if (fits)
    for (int i = tid; i < K * G; i += kTreeBlock) {
      const int k = i / G, j = i % G;
      if (j >= first[k] && j < len[k]) owner[base[k] + j - first[k]] = (uint8_t)k;
    }
  __syncthreads();
  for (int t = tid; t < T; t += kTreeBlock) {
    int32_t xt = -1, pt = -1, dt = 0;
    if (t == 0 && n > 0) {
      xt = root ? root[b] : -1;
    } else if (t < n) {
      const int k = owner[t], j = t - base[k] + first[k];
      xt = x[k * G + j];
      dt = j + 1;
      pt = j == 0 ? 0 : j > first[k] ? t - 1 : base[par[k]] + j - 1 - first[par[k]];
    }
    tokens[b * T + t] = xt;
    parent[b * T + t] = pt;
    depth[b * T + t] = dt;
  }
  for (int i = tid; i < K * (G + 1); i += kTreeBlock) {
    int k = i / (G + 1);
    const int j = i % (G + 1) - 1;  // the drafted position whose node this is; -1: the root
    int node = 0;
    if (j >= 0) {
      if (j < len[k]) {
        while (j < first[k]) k = par[k];
        node = base[k] + j - first[k];
      } else {
        node = -1;
      }
    }
    p_index[b * K * (G + 1) + i] = n > 0 && node >= 0 ? (int32_t)(b * T + node) : -1;
  }
  // ancestor words: `ws` neighbouring threads share a node
  int ws = 1;
  while (ws < W && ws < 32) ws *= 2;
  const int w0 = tid & (ws - 1);
  for (int t = tid / ws; t < T; t += kTreeBlock / ws) {
    uint32_t *row = anc + (b * T + t) * W;
    for (int w = w0; w < W; w += ws) {
      uint32_t bits = 0;
      if (t < n) {
        bits = w == 0 ? 1u : 0u;
        if (t > 0) {
          int k = owner[t], hi = t - base[k] + first[k];
          while (true) {
            bits |= range_bits(base[k], base[k] + hi - first[k], w);
            hi = first[k] - 1;
            if (hi < 0) break;
            k = par[k];
          }
        }
      }
      row[w] = bits;
    }
  }
}

}  // namespace svd
