// svd_step.hpp -- entry points of the operators around a verification step
// (draft tree, paged cache, tree attention, logit adjustments): argument
// checks, plans and launches.  Part of svd_api.hip, after its helpers.
#pragma once

namespace {

// A launch holds fewer than 2^32 threads.
bool grid_ok(int64_t blocks, int64_t threads) {
  return blocks >= 1 && blocks <= (((int64_t)1 << 32) - 1) / threads;
}

bool tree_sizes_ok(int64_t B, int32_t T) {
  return B >= 1 && T >= 1 && T <= SVD_MAX_NODES && B < ((int64_t)1 << 30) / T;
}

// The cache's arrays and sizes; fills the view.
int cache_view(const svd_cache_t *c, CacheView &v) {
  if (!c || !c->k || !c->v || !c->block_table) return SVD_EINVAL;
  if (c->dtype != SVD_CACHE_BF16 && c->dtype != SVD_CACHE_E4M3) return SVD_EDTYPE;
  const bool e4m3 = c->dtype == SVD_CACHE_E4M3;
  if (e4m3 && (!c->k_scale || !c->v_scale)) return SVD_EINVAL;
  // the attention reads the scales of four tokens as one word
  if (e4m3 && (((uintptr_t)c->k_scale) % 4 != 0 || ((uintptr_t)c->v_scale) % 4 != 0))
    return SVD_EINVAL;
  if (c->head_dim != 64 && c->head_dim != 128) return SVD_EINVAL;
  if (c->page < 16 || c->page > 1024 || (c->page & (c->page - 1)) != 0) return SVD_EINVAL;
  if (c->n_pages < 1 || c->n_pages >= (int64_t)1 << 31 || c->max_pages < 1 || c->kv_heads < 1 ||
      c->kv_heads > 4096)
    return SVD_EINVAL;
  if ((int64_t)c->max_pages * c->page >= (int64_t)1 << 31) return SVD_EINVAL;
  if (((uintptr_t)c->k) % 16 != 0 || ((uintptr_t)c->v) % 16 != 0) return SVD_EINVAL;
  v.k = static_cast<uint8_t *>(c->k);
  v.v = static_cast<uint8_t *>(c->v);
  v.k_scale = static_cast<uint8_t *>(c->k_scale);
  v.v_scale = static_cast<uint8_t *>(c->v_scale);
  v.table = c->block_table;
  v.n_pages = c->n_pages;
  v.max_pages = c->max_pages;
  v.page_shift = __builtin_ctz((unsigned)c->page);
  v.Hkv = c->kv_heads;
  return SVD_OK;
}

template <typename E, bool kVec, bool kE4M3, int D>
int write_rows(const void *k, const void *v, int64_t ks, int64_t vs, const int32_t *ctx_len,
               const int32_t *n_new, const int32_t *dst, int64_t B, int64_t T, const CacheView &c,
               hipStream_t s) {
  using T_ = typename E::elem;
  constexpr int kRows = kCacheBlock / (D / 8);
  const int64_t per_b = (T * c.Hkv * 2 + kRows - 1) / kRows;
  if (B > ((int64_t)1 << 32) / per_b || !grid_ok(B * per_b, kCacheBlock)) return SVD_EINVAL;
  CallTimer tm;
  SVD_LAUNCH(tm, SVD_KERNEL_CACHE_WRITE, s, kr_cache_write<E, kVec, kE4M3, D>,
             dim3((unsigned)(B * per_b)), dim3(kCacheBlock), s, static_cast<const T_ *>(k),
             static_cast<const T_ *>(v), ks, vs, ctx_len, n_new, dst, T, per_b, c);
  return SVD_OK;
}

template <typename E, bool kVec>
int write_kind(bool e4m3, int D, const void *k, const void *v, int64_t ks, int64_t vs,
               const int32_t *ctx_len, const int32_t *n_new, const int32_t *dst, int64_t B,
               int64_t T, const CacheView &c, hipStream_t s) {
  if (e4m3)
    return D == 64 ? write_rows<E, kVec, true, 64>(k, v, ks, vs, ctx_len, n_new, dst, B, T, c, s)
                   : write_rows<E, kVec, true, 128>(k, v, ks, vs, ctx_len, n_new, dst, B, T, c, s);
  return D == 64 ? write_rows<E, kVec, false, 64>(k, v, ks, vs, ctx_len, n_new, dst, B, T, c, s)
                 : write_rows<E, kVec, false, 128>(k, v, ks, vs, ctx_len, n_new, dst, B, T, c, s);
}

template <typename E, bool kE4M3, int D>
int read_rows(const CacheView &c, const int32_t *start, const int32_t *count, int64_t B, int64_t N,
              void *k, void *v, hipStream_t s) {
  using T_ = typename E::elem;
  constexpr int kRows = kCacheBlock / (D / 8);
  const int64_t per_b = (N * c.Hkv * 2 + kRows - 1) / kRows;
  if (B > ((int64_t)1 << 32) / per_b || !grid_ok(B * per_b, kCacheBlock)) return SVD_EINVAL;
  CallTimer tm;
  SVD_LAUNCH(tm, SVD_KERNEL_CACHE_READ, s, kr_cache_read<E, kE4M3, D>, dim3((unsigned)(B * per_b)),
             dim3(kCacheBlock), s, c, start, count, N, per_b, static_cast<T_ *>(k),
             static_cast<T_ *>(v));
  return SVD_OK;
}

template <typename E>
int read_kind(bool e4m3, int D, const CacheView &c, const int32_t *start, const int32_t *count,
              int64_t B, int64_t N, void *k, void *v, hipStream_t s) {
  if (e4m3)
    return D == 64 ? read_rows<E, true, 64>(c, start, count, B, N, k, v, s)
                   : read_rows<E, true, 128>(c, start, count, B, N, k, v, s);
  return D == 64 ? read_rows<E, false, 64>(c, start, count, B, N, k, v, s)
                 : read_rows<E, false, 128>(c, start, count, B, N, k, v, s);
}

// Rows per workgroup and parts of an attention call: a function of the sizes alone.
struct AttnPlan {
  int nt, wq, wt, m_tiles, m_rows, S;
};

// Parts.  Up to 256 workgroups, one per CU, while that leaves a part no more than
// kAttnLongPart tiles; longer ones in two rounds (32-row waves, one workgroup per CU)
// or four (16-row waves, two per CU), which smooth prefixes of different
// lengths.  Measured over S = 1..64: eight requests with 16000 tokens, 95 us with 4 parts,
// 208 with 1 and 135 with 32; one with 4000 tokens and 129 nodes, 42 us with 10,
// 87 with 2 and 62 with 16; four with 30000 and 129 nodes, 381 us with 6, 555 with 2,
// 449 with 10; 24 with 500 to 5000 and 16 heads, 57 us with 3, 73 with 1, 70 with 8.
constexpr int64_t kAttnCus = 256;
constexpr int64_t kAttnLongPart = 64;
// Parts are cut for the room of the block table: it is what the host knows, and a captured
// call keeps its cut while lengths grow.  A sequence much shorter than its room has
// parts of one tile or none: eight requests of 9 nodes and 1000 tokens take 17 us with
// room for 1000 to 16000, 25 with room for 32000 or more (16 parts of a tile); 256 of them
// are not cut at all.
constexpr int64_t kAttnMinPart = 2;   // a part has room for at least this many tiles

AttnPlan attn_plan(int64_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t D, int64_t room) {
  AttnPlan p;
  const int64_t rows = (int64_t)T * (Hq / Hkv);
  p.nt = rows <= 64 ? 1 : 2;
  p.wq = rows <= 64 ? (int)((rows + 15) / 16) : rows <= 128 ? 4 : 8;
  p.wt = rows <= 32 || (p.nt == 2 && p.wq == 4) ? 2 : 1;
  const int m = 16 * p.nt * p.wq;
  p.m_tiles = (int)((rows + m - 1) / m);
  const int unit = 16 * p.nt;  // rows of a wave: the workgroups share them evenly
  const int64_t waves = (rows + unit - 1) / unit;
  p.m_rows = (int)((waves + p.m_tiles - 1) / p.m_tiles) * unit;
  const int64_t base = B * Hkv * p.m_tiles;
  const int64_t tk = 8192 / D, tiles = (room + tk - 1) / tk;  // as AttnShape::TK
  int64_t S = std::max<int64_t>(1, kAttnCus / base);
  if (tiles / S > kAttnLongPart || (p.nt == 1 && base > kAttnCus)) {
    const int64_t rounds = p.nt == 1 ? 4 : 2;
    S = std::max(S, (rounds * kAttnCus + base - 1) / base);
  }
  S = std::min<int64_t>({S, tiles / kAttnMinPart, kAttnMaxSplits});
  p.S = (int)std::max<int64_t>(1, S);
  return p;
}

bool attn_sizes_ok(int64_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t D, int64_t room) {
  if (!tree_sizes_ok(B, T) || Hkv < 1 || Hkv > 4096 || Hq < Hkv || Hq > 65536 || Hq % Hkv != 0)
    return false;
  if (D != 64 && D != 128) return false;
  if (room < 1 || room >= (int64_t)1 << 31) return false;
  const AttnPlan p = attn_plan(B, T, Hq, Hkv, D, room);
  const int64_t threads = 64 * p.wq * p.wt + (p.nt == 1 ? kAttnLoaders : 0);
  return B <= ((int64_t)1 << 32) / Hkv &&
         grid_ok(((B * Hkv * p.S + 7) / 8 * 8) * p.m_tiles, threads);
}

size_t attn_ms_offset(int64_t rows, int S, int D) {
  return align_up((size_t)rows * S * D * sizeof(float));
}

template <int D, bool kE4M3, int NT, int WQ, int WT>
int attn_launch(const CacheView &c, const AttnArgs &a, int Hq, hipStream_t s) {
  CallTimer tm;
  const int64_t grid = ((int64_t)a.units + 7) / 8 * 8 * a.m_tiles;
  SVD_LAUNCH(tm, SVD_KERNEL_TREE_ATTENTION, s, kr_tree_attention<D, kE4M3, NT, WQ, WT>,
             dim3((unsigned)grid), dim3(AttnShape<D, kE4M3, NT, WQ, WT>::kBlock), s, c, a);
  if (a.S > 1) {
    constexpr int rows = kAttnJoinBlock / (D / 4);
    SVD_LAUNCH(tm, SVD_KERNEL_ATTENTION_JOIN, s, kr_attn_join<D>,
               dim3((unsigned)((a.rows_all + rows - 1) / rows)), dim3(kAttnJoinBlock), s, a, Hq);
  }
  return SVD_OK;
}

template <int D, bool kE4M3>
int attn_rows(const AttnPlan &p, const CacheView &c, const AttnArgs &a, int Hq, hipStream_t s) {
  if (p.nt == 2 && p.wq == 8) return attn_launch<D, kE4M3, 2, 8, 1>(c, a, Hq, s);
  if (p.nt == 2) return attn_launch<D, kE4M3, 2, 4, 2>(c, a, Hq, s);
  if (p.wq == 4) return attn_launch<D, kE4M3, 1, 4, 1>(c, a, Hq, s);
  if (p.wq == 3) return attn_launch<D, kE4M3, 1, 3, 1>(c, a, Hq, s);
  if (p.wq == 2) return attn_launch<D, kE4M3, 1, 2, 2>(c, a, Hq, s);
  return attn_launch<D, kE4M3, 1, 1, 2>(c, a, Hq, s);
}

template <typename E, bool kVec, bool kBias, int PATH>
int adjust_launch(const void *logits, void *out, const AdjustArgs &a, int64_t blocks,
                  hipStream_t s) {
  using T_ = typename E::elem;
  CallTimer tm;
  SVD_LAUNCH(tm, SVD_KERNEL_ADJUST, s, kr_adjust<E, kVec, kBias, PATH>, dim3((unsigned)blocks),
             dim3(kAdjBlock), s, static_cast<const T_ *>(logits), static_cast<T_ *>(out), a);
  return SVD_OK;
}

template <typename E, bool kVec>
int adjust_kind(const void *logits, void *out, const AdjustArgs &a, int64_t blocks,
                hipStream_t s) {
  const bool small = a.T <= kAdjPathSmall;
  if (a.bias_off)
    return small ? adjust_launch<E, kVec, true, kAdjPathSmall>(logits, out, a, blocks, s)
                 : adjust_launch<E, kVec, true, kAdjPathMax>(logits, out, a, blocks, s);
  return small ? adjust_launch<E, kVec, false, kAdjPathSmall>(logits, out, a, blocks, s)
               : adjust_launch<E, kVec, false, kAdjPathMax>(logits, out, a, blocks, s);
}

}  // namespace

extern "C" {

int svd_draft_tree(const int32_t *drafts, const int32_t *root, int64_t B, int32_t K, int32_t gamma,
                   int32_t T, int32_t *tokens, int32_t *parent, int32_t *depth, uint32_t *anc,
                   int32_t *n_nodes, int32_t *p_index, void *hip_stream) {
  if (!drafts || !tokens || !parent || !depth || !anc || !n_nodes || !p_index) return SVD_EINVAL;
  if (K < 1 || K > SVD_MAX_K || gamma < 1 || gamma > SVD_MAX_GAMMA || !tree_sizes_ok(B, T) ||
      B >= ((int64_t)1 << 31) / ((int64_t)K * (gamma + 1)) || !grid_ok(B, kTreeBlock))
    return SVD_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  CallTimer tm;
  SVD_LAUNCH(tm, SVD_KERNEL_DRAFT_TREE, s, kr_draft_tree, dim3((unsigned)B), dim3(kTreeBlock), s,
             drafts, root, (int)K, (int)gamma, (int)T, (int)((T + 31) / 32), tokens, parent, depth,
             anc, n_nodes, p_index);
  return SVD_OK;
}

int svd_cache_write(const svd_cache_t *cache, const void *k, const void *v, svd_dtype_t dtype,
                    int64_t k_stride, int64_t v_stride, const int32_t *ctx_len,
                    const int32_t *n_new, const int32_t *dst, int64_t B, int64_t T,
                    void *hip_stream) {
  CacheView c;
  const int rc = cache_view(cache, c);
  if (rc != SVD_OK) return rc;
  if (!k || !v || !ctx_len) return SVD_EINVAL;
  if (dtype != SVD_F32 && dtype != SVD_BF16) return SVD_EDTYPE;
  if (B < 1 || T < 1 || T >= (int64_t)1 << 31 || B >= ((int64_t)1 << 31) / T) return SVD_EINVAL;
  const int D = cache->head_dim;
  const int64_t row = (int64_t)c.Hkv * D;
  if (k_stride < row || v_stride < row) return SVD_EINVAL;
  const int es = dtype == SVD_F32 ? 4 : 2;
  if (((uintptr_t)k) % es != 0 || ((uintptr_t)v) % es != 0) return SVD_EINVAL;
  const bool vec = ((uintptr_t)k) % 16 == 0 && ((uintptr_t)v) % 16 == 0 &&
                   k_stride * es % 16 == 0 && v_stride * es % 16 == 0;
  const bool e4m3 = cache->dtype == SVD_CACHE_E4M3;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if (dtype == SVD_BF16)
    return vec ? write_kind<BF16, true>(e4m3, D, k, v, k_stride, v_stride, ctx_len, n_new, dst, B,
                                        T, c, s)
               : write_kind<BF16, false>(e4m3, D, k, v, k_stride, v_stride, ctx_len, n_new, dst, B,
                                         T, c, s);
  return vec ? write_kind<F32, true>(e4m3, D, k, v, k_stride, v_stride, ctx_len, n_new, dst, B, T,
                                     c, s)
             : write_kind<F32, false>(e4m3, D, k, v, k_stride, v_stride, ctx_len, n_new, dst, B, T,
                                      c, s);
}

int svd_cache_read(const svd_cache_t *cache, const int32_t *start, const int32_t *count, int64_t B,
                   int64_t N, svd_dtype_t dtype, void *k, void *v, void *hip_stream) {
  CacheView c;
  const int rc = cache_view(cache, c);
  if (rc != SVD_OK) return rc;
  if (!k || !v) return SVD_EINVAL;
  if (dtype != SVD_F32 && dtype != SVD_BF16) return SVD_EDTYPE;
  if (B < 1 || N < 1 || N >= (int64_t)1 << 31 || B >= ((int64_t)1 << 31) / N) return SVD_EINVAL;
  if (((uintptr_t)k) % 16 != 0 || ((uintptr_t)v) % 16 != 0) return SVD_EINVAL;
  const bool e4m3 = cache->dtype == SVD_CACHE_E4M3;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if (dtype == SVD_BF16)
    return read_kind<BF16>(e4m3, cache->head_dim, c, start, count, B, N, k, v, s);
  return read_kind<F32>(e4m3, cache->head_dim, c, start, count, B, N, k, v, s);
}

size_t svd_tree_attention_workspace_bytes(int64_t B, int32_t T, int32_t q_heads, int32_t kv_heads,
                                          int32_t head_dim, int64_t max_len) {
  if (!attn_sizes_ok(B, T, q_heads, kv_heads, head_dim, max_len)) return 0;
  const AttnPlan p = attn_plan(B, T, q_heads, kv_heads, head_dim, max_len);
  if (p.S == 1) return kAlign;
  const int64_t rows = B * T * q_heads;
  return attn_ms_offset(rows, p.S, head_dim) + align_up((size_t)rows * p.S * 2 * sizeof(float));
}

int svd_tree_attention(const svd_cache_t *cache, const void *q, int64_t q_stride,
                       const int32_t *ctx_len, const int32_t *n_nodes, const uint32_t *anc,
                       float scale, int64_t B, int32_t T, int32_t q_heads, void *out, float *lse,
                       void *workspace, size_t workspace_bytes, void *hip_stream) {
  CacheView c;
  const int rc = cache_view(cache, c);
  if (rc != SVD_OK) return rc;
  if (!q || !ctx_len || !out || !workspace) return SVD_EINVAL;
  const int D = cache->head_dim;
  const int64_t room = (int64_t)c.max_pages << c.page_shift;
  if (!attn_sizes_ok(B, T, q_heads, c.Hkv, D, room)) return SVD_EINVAL;
  if (!(std::isfinite(scale) && scale > 0.0f)) return SVD_EINVAL;
  const float cs = (float)(1.4426950408889634 * (double)scale);
  if (!(std::isfinite(cs) && cs > 0.0f)) return SVD_EINVAL;
  if (q_stride < (int64_t)q_heads * D || q_stride % 8 != 0 || ((uintptr_t)q) % 16 != 0 ||
      ((uintptr_t)out) % 16 != 0 || ((uintptr_t)workspace) % kAlign != 0)
    return SVD_EINVAL;
  if (workspace_bytes < svd_tree_attention_workspace_bytes(B, T, q_heads, c.Hkv, D, room))
    return SVD_EWORKSPACE;
  // a row with values that are not finite reads its query again while pieces of its
  // output are written already
  const uintptr_t q0 = (uintptr_t)q, o0 = (uintptr_t)out;
  const uint64_t row = (uint64_t)q_heads * D * 2;
  if (q0 < o0 + (uint64_t)(B * T) * row &&
      o0 < q0 + (uint64_t)(B * T - 1) * ((uint64_t)q_stride * 2) + row)
    return SVD_EINVAL;
  const AttnPlan p = attn_plan(B, T, q_heads, c.Hkv, D, room);
  AttnArgs a;
  a.q = static_cast<const uint16_t *>(q);
  a.q_stride = q_stride;
  a.ctx_len = ctx_len;
  a.n_nodes = n_nodes;
  a.table = c.table;
  a.anc = anc;
  a.room = room;
  a.T = T;
  a.group = q_heads / c.Hkv;
  a.S = p.S;
  a.m_tiles = p.m_tiles;
  a.m_rows = p.m_rows;
  a.units = (int)(B * c.Hkv * p.S);
  a.c = cs;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.rows_all = B * T * q_heads;
  a.part_o = static_cast<float *>(workspace);
  a.part_ms = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                        attn_ms_offset(a.rows_all, p.S, D));
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if (cache->dtype == SVD_CACHE_E4M3)
    return D == 64 ? attn_rows<64, true>(p, c, a, q_heads, s)
                   : attn_rows<128, true>(p, c, a, q_heads, s);
  return D == 64 ? attn_rows<64, false>(p, c, a, q_heads, s)
                 : attn_rows<128, false>(p, c, a, q_heads, s);
}

int svd_adjust_logits(const void *logits, void *out, svd_dtype_t dtype, int64_t B, int32_t T,
                      int32_t V, const int32_t *n_rows, const int32_t *history,
                      int64_t hist_stride, const int32_t *hist_len, const int32_t *prompt_len,
                      const int32_t *tokens, const uint32_t *anc, const float *repetition,
                      const float *frequency, const float *presence, const int32_t *bias_off,
                      const int32_t *bias_tok, const float *bias_val, int64_t n_bias,
                      const uint32_t *allow, const int32_t *allow_index, int32_t n_masks,
                      void *hip_stream) {
  if (!logits || !out) return SVD_EINVAL;
  if (dtype != SVD_F32 && dtype != SVD_BF16) return SVD_EDTYPE;
  if (!tree_sizes_ok(B, T) || V < 1) return SVD_EINVAL;
  if (history && (!hist_len || hist_stride < 1 || hist_stride >= (int64_t)1 << 30))
    return SVD_EINVAL;
  if (anc && !tokens) return SVD_EINVAL;
  if (bias_off && (n_bias < 0 || (n_bias > 0 && (!bias_tok || !bias_val)))) return SVD_EINVAL;
  if (allow && (!allow_index || n_masks < 1)) return SVD_EINVAL;
  const size_t es = dtype == SVD_F32 ? 4 : 2;
  if (((uintptr_t)logits) % es != 0 || ((uintptr_t)out) % es != 0) return SVD_EINVAL;
  AdjustArgs a;
  a.n_rows = n_rows;
  a.history = history;
  a.hist_stride = hist_stride;
  a.hist_len = hist_len;
  a.prompt_len = prompt_len;
  a.tokens = tokens;
  a.anc = anc;
  a.repetition = repetition;
  a.frequency = frequency;
  a.presence = presence;
  a.bias_off = n_bias > 0 ? bias_off : nullptr;
  a.bias_tok = bias_tok;
  a.bias_val = bias_val;
  a.n_bias = n_bias;
  a.allow = allow;
  a.allow_index = allow_index;
  a.n_masks = n_masks;
  a.T = T;
  a.V = V;
  a.in_place = logits == out;
  // ranges as long as the workgroups still fill the GPU, then rows in chunks
  a.range = kAdjRange;
  while (a.range > kAdjRangeMin && B * T * (((int64_t)V + a.range - 1) / a.range) < 1024)
    a.range /= 2;
  const int64_t nr = ((int64_t)V + a.range - 1) / a.range;
  const int64_t want = std::max<int64_t>(1, 1024 / (B * nr));  // workgroups that fit at once
  a.row_step = (int)std::max<int64_t>(std::min(T, 4), (T + want - 1) / want);
  a.row_step = std::min(a.row_step, kAdjRowsMax);
  a.n_ranges = (int)nr;
  a.n_chunks = (T + a.row_step - 1) / a.row_step;
  const int64_t blocks = B * nr * a.n_chunks;
  if (!grid_ok(blocks, kAdjBlock)) return SVD_EINVAL;
  const bool vec = ((size_t)V * es) % 16 == 0 && ((uintptr_t)logits) % 16 == 0 &&
                   ((uintptr_t)out) % 16 == 0;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if (dtype == SVD_BF16)
    return vec ? adjust_kind<BF16, true>(logits, out, a, blocks, s)
               : adjust_kind<BF16, false>(logits, out, a, blocks, s);
  return vec ? adjust_kind<F32, true>(logits, out, a, blocks, s)
             : adjust_kind<F32, false>(logits, out, a, blocks, s);
}

}  // extern "C"
