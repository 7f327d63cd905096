// svd_serve.hpp -- entry points of a serving loop's other operators (block tables and
// slot maps, filtered and sampled logits, attention over shared prefixes): argument
// checks, plans and launches.  Part of svd_api.hip, after svd_step.hpp.
#pragma once

namespace {

// Whether two arrays of these sizes meet.
bool overlap(const void *a, uint64_t a_bytes, const void *b, uint64_t b_bytes) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + b_bytes && y < x + a_bytes;
}

bool page_ok(int32_t page) { return page >= 16 && page <= 1024 && (page & (page - 1)) == 0; }

bool pages_sizes_ok(int64_t B, int32_t max_pages, int32_t page, int64_t n_pages) {
  return page_ok(page) && max_pages >= 1 && (int64_t)max_pages * page < (int64_t)1 << 31 &&
         B >= 1 && B < ((int64_t)1 << 31) / max_pages && n_pages >= 1 &&
         n_pages < (int64_t)1 << 31;
}

template <typename E, bool kVec, bool kE4M3, int D>
int write_slot_rows(const void *k, const void *v, int64_t ks, int64_t vs, const int64_t *slots,
                    int64_t N, const CacheView &c, hipStream_t s) {
  using T_ = typename E::elem;
  constexpr int kRows = kCacheBlock / (D / 8);
  const int64_t blocks = (N * c.Hkv * 2 + kRows - 1) / kRows;
  if (!grid_ok(blocks, kCacheBlock)) return SVD_EINVAL;
  CallTimer tm;
  SVD_LAUNCH(tm, SVD_KERNEL_CACHE_WRITE, s, kr_cache_write_slots<E, kVec, kE4M3, D>,
             dim3((unsigned)blocks), dim3(kCacheBlock), s, static_cast<const T_ *>(k),
             static_cast<const T_ *>(v), ks, vs, slots, N, c);
  return SVD_OK;
}

template <typename E, bool kVec>
int write_slot_kind(bool e4m3, int D, const void *k, const void *v, int64_t ks, int64_t vs,
                    const int64_t *slots, int64_t N, const CacheView &c, hipStream_t s) {
  if (e4m3)
    return D == 64 ? write_slot_rows<E, kVec, true, 64>(k, v, ks, vs, slots, N, c, s)
                   : write_slot_rows<E, kVec, true, 128>(k, v, ks, vs, slots, N, c, s);
  return D == 64 ? write_slot_rows<E, kVec, false, 64>(k, v, ks, vs, slots, N, c, s)
                 : write_slot_rows<E, kVec, false, 128>(k, v, ks, vs, slots, N, c, s);
}

// The settings of a filter or sample call that both check alike.
int filter_args(FilterArgs &a, svd_dtype_t dtype, int64_t B, int32_t T, int32_t V,
                const void *logits, const int32_t *n_rows, const float *temperature,
                const int32_t *top_k, const float *top_p, const float *min_p) {
  if (!logits) return SVD_EINVAL;
  if (dtype != SVD_F32 && dtype != SVD_BF16) return SVD_EDTYPE;
  if (!tree_sizes_ok(B, T) || V < 1 || !grid_ok(B * T, kFilterBlock)) return SVD_EINVAL;
  if (((uintptr_t)logits) % (dtype == SVD_F32 ? 4 : 2) != 0) return SVD_EINVAL;
  a = FilterArgs{};
  a.n_rows = n_rows;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.V = V;
  a.T = T;
  constexpr int64_t step = 8 * kFilterBlock;
  a.slab = step * (((int64_t)V + step * kFilterBlock - 1) / (step * kFilterBlock));
  int bits = 0;  // V * 2^shift stays below 2^62
  while (((int64_t)1 << bits) < V) ++bits;
  a.shift = std::min(62 - bits, 50);
  return SVD_OK;
}

// A row in one workgroup's registers, or in as many passes over memory as there are
// searches (kr_filter_row.hpp), or by the passes that take any row (kr_filter.hpp): for
// vocabularies that are past a row's records, and for many rows of small ones, where four
// workgroups share a CU.  Top-k and top-p of bf16, held against passes: one row of 8192 12
// against 37 us, of 512 11 against 20; 256 rows of 8192 17 against 39, of 512 16 against 21;
// 2048 rows of 8192 115 against 110, of 512 100 against 55; 8192 rows of 2048 405 against 218.
// Above 8192 tokens a row is held whatever the number of rows: 8192 rows of 16384 463 against
// 633, 2304 of 32000 154 against 357 (fp32 333 against 683), 512 of 64000 49 against 214.  Top-p
// alone: 507 against 526, 165 against 290 (322 against 470), 52 against 180; 8192 rows of 8193, at
// the border, 561 against 498.
constexpr int64_t kFilterSmall = 8192, kFilterRound = 256;  // tokens; rows, one per CU

template <typename E, int NV>
int filter_held(const void *logits, void *out, const FilterArgs &a, int64_t rows, hipStream_t s) {
  using T_ = typename E::elem;
  CallTimer tm;
  if (out) {
    SVD_LAUNCH(tm, SVD_KERNEL_FILTER, s, kr_filter<E, kFilterBlock, NV>, dim3((unsigned)rows),
               dim3(kFilterBlock), s, static_cast<const T_ *>(logits), static_cast<T_ *>(out), a);
  } else {
    SVD_LAUNCH(tm, SVD_KERNEL_SAMPLE, s, kr_sample<E, kFilterBlock, NV>, dim3((unsigned)rows),
               dim3(kFilterBlock), s, static_cast<const T_ *>(logits), a);
  }
  return SVD_OK;
}

template <typename E, bool kVec, int NT>
int filter_passes(const void *logits, void *out, const FilterArgs &a, int64_t rows,
                  hipStream_t s) {
  using T_ = typename E::elem;
  CallTimer tm;
  if (out) {
    SVD_LAUNCH(tm, SVD_KERNEL_FILTER, s, kr_filter_any<E, kVec, NT>, dim3((unsigned)rows), dim3(NT),
               s, static_cast<const T_ *>(logits), static_cast<T_ *>(out), a);
  } else {
    SVD_LAUNCH(tm, SVD_KERNEL_SAMPLE, s, kr_sample_any<E, kVec, NT>, dim3((unsigned)rows), dim3(NT),
               s, static_cast<const T_ *>(logits), a);
  }
  return SVD_OK;
}

// out: nullptr for a sample call.
template <typename E>
int filter_rows(const void *logits, void *out, const FilterArgs &a, int64_t rows, hipStream_t s) {
  constexpr int64_t es = sizeof(typename E::elem), P = E::kPerVec, step = P * kFilterBlock;
  const bool alike = !out || ((uintptr_t)logits - (uintptr_t)out) % 16 == 0;
  const int64_t most = a.V + P - 1;  // tokens of whole 16-byte pieces
  const bool passes = a.V <= kFilterSmall && rows > kFilterRound;
  if (alike && !passes) {
    if (es == 2) {
      if (most <= 5 * step) return filter_held<BF16, 5>(logits, out, a, rows, s);
      if (most <= 10 * step) return filter_held<BF16, 10>(logits, out, a, rows, s);
      if (most <= 19 * step) return filter_held<BF16, 19>(logits, out, a, rows, s);
    }
    if (most <= 64 * step) return filter_held<E, 0>(logits, out, a, rows, s);
  }
  if (!passes) return filter_passes<E, false, kFilterBlock>(logits, out, a, rows, s);
  const bool vec = a.V * es % 16 == 0 && ((uintptr_t)logits) % 16 == 0 &&
                   ((uintptr_t)out) % 16 == 0;
  return vec ? filter_passes<E, true, 256>(logits, out, a, rows, s)
             : filter_passes<E, false, 256>(logits, out, a, rows, s);
}

// Rows of a workgroup of the shared part: 256, or 64 with the tokens split over its waves
// where groups have no more on average (the host knows no group's own length, and a tile has
// rows of one group alone).  Whole calls with 32 query and 8 kv heads of 128, one token a
// sequence, 64 rows against 256: 4 sequences over 32000 shared bf16 tokens 56 and 66 us, over
// 8192 34 and 37, over 1024 28 either way; 64 groups of 2, 4 and 8 sequences over 8192 shared
// E4M3 tokens each 437 and 612, 471 and 640, 525 and 694, in workspaces of 28 to 34 MB and of
// 104 to 111.
int share_rows(int64_t B, int32_t T, int64_t group, int64_t G) {
  constexpr int few = SharedShape<128, 4, 2>::M, many = SharedShape<128, 8, 1>::M;
  return B * T * group <= few * G ? few : many;
}

template <int D, bool kE4M3, int NW, int WT>
int shared_launch(const CacheView &c, const AttnArgs &a, int64_t G, float *o, float *ms,
                  hipStream_t s) {
  CallTimer tm;
  auto go = [&](auto *kernel) -> int {
    SVD_LAUNCH(tm, SVD_KERNEL_SHARED_ATTENTION, s, kernel, dim3(kShareWorkgroups),
               dim3(64 * NW), s, c, a, G, o, ms);
    return SVD_OK;
  };
  if (a.slopes) return go(kr_shared_attention<D, kE4M3, NW, WT, kSloped>);
  return a.cap_in > 0.0f ? go(kr_shared_attention<D, kE4M3, NW, WT, kCapped>)
                         : go(kr_shared_attention<D, kE4M3, NW, WT, kPlain>);
}

template <int D, bool kE4M3>
int shared_rows(const CacheView &c, const AttnArgs &a, int64_t G, float *o, float *ms,
                hipStream_t s) {
  return a.share_rows == 64 ? shared_launch<D, kE4M3, 4, 2>(c, a, G, o, ms, s)
                            : shared_launch<D, kE4M3, 8, 1>(c, a, G, o, ms, s);
}

int shared_kind(const svd_cache_t *cache, const CacheView &c, const AttnArgs &a, int64_t G,
                float *o, float *ms, hipStream_t s) {
  if (cache->dtype == SVD_CACHE_E4M3)
    return cache->head_dim == 64 ? shared_rows<64, true>(c, a, G, o, ms, s)
                                 : shared_rows<128, true>(c, a, G, o, ms, s);
  return cache->head_dim == 64 ? shared_rows<64, false>(c, a, G, o, ms, s)
                               : shared_rows<128, false>(c, a, G, o, ms, s);
}

constexpr float kMostCap = 16384.0f;

struct PrefixLayout {
  size_t seqs, groups, cut, nodes, share_o, share_ms, part_o, part_ms, total;
};

// The call's sizes, and its workspace; false: sizes out of range.
bool prefix_layout(int64_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t D, int64_t room,
                   int64_t G, PrefixLayout &l) {
  if (!attn_sizes_ok(B, T, Hq, Hkv, D, room) || G < 0 || G > B) return false;
  const int64_t group = Hq / Hkv;
  size_t off = 0;
  l = PrefixLayout{};
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes);
    return at;
  };
  if (G > 0) {
    if (B * T >= ((int64_t)1 << 31) / group) return false;
    const int64_t rows = share_rows(B, T, group, G);
    // every unit, and every piece of the line, begins a part at most
    const int64_t units = (B * T * group / rows + G) * Hkv;
    if (units >= (int64_t)1 << 30) return false;
    const size_t parts = (size_t)(units + kShareWorkgroups) * rows;
    l.seqs = take((size_t)B * sizeof(ShareSeq));
    l.groups = take((size_t)G * sizeof(ShareGroup));
    l.cut = take(sizeof(ShareCut));
    l.nodes = take((size_t)(B * T) * sizeof(int32_t));
    l.share_o = take(parts * D * sizeof(float));
    l.share_ms = take(parts * 2 * sizeof(float));
  }
  const int S = attn_plan(B, T, Hq, Hkv, D, room).S;
  if (S > 1) {
    const size_t rows = (size_t)(B * T) * Hq * S;
    l.part_o = take(rows * D * sizeof(float));
    l.part_ms = take(rows * 2 * sizeof(float));
  }
  l.total = std::max(off, kAlign);
  return true;
}

}  // namespace

extern "C" {

size_t svd_cache_pages_workspace_bytes(int64_t B) {
  if (B < 1 || B >= (int64_t)1 << 31) return 0;
  return align_up(sizeof(PageHead)) + align_up((size_t)B * sizeof(PagePlan));
}

int svd_cache_pages(const int32_t *length, const int32_t *shared, int64_t B, int32_t max_pages,
                    int32_t page, int64_t n_pages, int32_t *free_ring, const int32_t *state,
                    const int32_t *held, const int32_t *block_table, int32_t *state_out,
                    int32_t *held_out, int32_t *table_out, int32_t *room, void *workspace,
                    size_t workspace_bytes, void *hip_stream) {
  if (!length || !free_ring || !state || !held || !block_table || !state_out || !held_out ||
      !table_out || !room || !workspace)
    return SVD_EINVAL;
  if (!pages_sizes_ok(B, max_pages, page, n_pages)) return SVD_EINVAL;
  if (((uintptr_t)workspace) % kAlign != 0) return SVD_EINVAL;
  if (workspace_bytes < svd_cache_pages_workspace_bytes(B)) return SVD_EWORKSPACE;
  const int64_t entries = B * max_pages;
  // in place, or apart
  if ((state != state_out && overlap(state, 8, state_out, 8)) ||
      (held != held_out && overlap(held, 4 * (uint64_t)B, held_out, 4 * (uint64_t)B)) ||
      (block_table != table_out &&
       overlap(block_table, 4 * (uint64_t)entries, table_out, 4 * (uint64_t)entries)))
    return SVD_EINVAL;
  const int64_t blocks = (entries + kPagesMoveBlock - 1) / kPagesMoveBlock;
  if (!grid_ok(blocks, kPagesMoveBlock)) return SVD_EINVAL;
  PagesArgs a;
  a.length = length;
  a.shared = shared;
  a.held = held;
  a.table = block_table;
  a.state = state;
  a.held_out = held_out;
  a.table_out = table_out;
  a.state_out = state_out;
  a.room = room;
  a.ring = free_ring;
  a.B = B;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.page_shift = __builtin_ctz((unsigned)page);
  a.head = static_cast<PageHead *>(workspace);
  a.plan = reinterpret_cast<PagePlan *>(static_cast<char *>(workspace) + align_up(sizeof(PageHead)));
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  CallTimer tm;
  SVD_LAUNCH(tm, SVD_KERNEL_PAGES, s, kr_pages_plan, dim3(1), dim3(kPagesBlock), s, a);
  SVD_LAUNCH(tm, SVD_KERNEL_PAGES, s, kr_pages_move, dim3((unsigned)blocks),
             dim3(kPagesMoveBlock), s, a);
  return SVD_OK;
}

int svd_cache_slots(const int32_t *ctx_len, const int32_t *n_new, const int32_t *block_table,
                    int64_t B, int32_t max_pages, int32_t page, int64_t n_pages, int64_t N,
                    int32_t *row_off, int32_t *seq, int32_t *pos, int64_t *slot,
                    void *hip_stream) {
  if (!ctx_len || !n_new || !block_table || !row_off || !seq || !pos || !slot) return SVD_EINVAL;
  if (!pages_sizes_ok(B, max_pages, page, n_pages) || N < 1 || N >= (int64_t)1 << 31)
    return SVD_EINVAL;
  SlotsArgs a;
  a.ctx_len = ctx_len;
  a.n_new = n_new;
  a.table = block_table;
  a.B = B;
  a.N = N;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.page_shift = __builtin_ctz((unsigned)page);
  a.row_off = row_off;
  a.seq = seq;
  a.pos = pos;
  a.slot = slot;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  CallTimer tm;
  SVD_LAUNCH(tm, SVD_KERNEL_SLOTS, s, kr_slots, dim3((unsigned)((N + kSlotsBlock - 1) / kSlotsBlock)),
             dim3(kSlotsBlock), s, a);
  return SVD_OK;
}

int svd_cache_write_slots(const svd_cache_t *cache, const void *k, const void *v,
                          svd_dtype_t dtype, int64_t k_stride, int64_t v_stride,
                          const int64_t *slot, int64_t N, void *hip_stream) {
  CacheView c;
  const int rc = cache_view(cache, c, false);
  if (rc != SVD_OK) return rc;
  if (!k || !v || !slot) return SVD_EINVAL;
  if (dtype != SVD_F32 && dtype != SVD_BF16) return SVD_EDTYPE;
  if (N < 1 || N >= (int64_t)1 << 31) return SVD_EINVAL;
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
    return vec ? write_slot_kind<BF16, true>(e4m3, D, k, v, k_stride, v_stride, slot, N, c, s)
               : write_slot_kind<BF16, false>(e4m3, D, k, v, k_stride, v_stride, slot, N, c, s);
  return vec ? write_slot_kind<F32, true>(e4m3, D, k, v, k_stride, v_stride, slot, N, c, s)
             : write_slot_kind<F32, false>(e4m3, D, k, v, k_stride, v_stride, slot, N, c, s);
}

int svd_filter_logits(const void *logits, void *out, svd_dtype_t dtype, int64_t B, int32_t T,
                      int32_t V, const int32_t *n_rows, const float *temperature,
                      const int32_t *top_k, const float *top_p, const float *min_p,
                      void *hip_stream) {
  if (!out) return SVD_EINVAL;
  FilterArgs a;
  const int rc = filter_args(a, dtype, B, T, V, logits, n_rows, temperature, top_k, top_p, min_p);
  if (rc != SVD_OK) return rc;
  const size_t es = dtype == SVD_F32 ? 4 : 2;
  if (((uintptr_t)out) % es != 0) return SVD_EINVAL;
  const uint64_t bytes = (uint64_t)(B * T) * (uint64_t)V * es;
  if (out != logits && overlap(out, bytes, logits, bytes)) return SVD_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  return dtype == SVD_BF16 ? filter_rows<BF16>(logits, out, a, B * T, s)
                           : filter_rows<F32>(logits, out, a, B * T, s);
}

int svd_sample(const void *logits, svd_dtype_t dtype, int64_t B, int32_t T, int32_t V, int32_t K,
               const int32_t *n_rows, const float *temperature, const int32_t *top_k,
               const float *top_p, const float *min_p, const double *uniforms, uint64_t seed,
               uint64_t row_base, int32_t *token, float *logprob, void *hip_stream) {
  if (!token) return SVD_EINVAL;
  FilterArgs a;
  const int rc = filter_args(a, dtype, B, T, V, logits, n_rows, temperature, top_k, top_p, min_p);
  if (rc != SVD_OK) return rc;
  if (K < 1 || K > SVD_MAX_K || B * T >= ((int64_t)1 << 31) / K) return SVD_EINVAL;
  a.K = K;
  a.u = uniforms;
  a.seed = seed;
  a.row_base = row_base;
  a.token = token;
  a.logprob = logprob;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  return dtype == SVD_BF16 ? filter_rows<BF16>(logits, nullptr, a, B * T, s)
                           : filter_rows<F32>(logits, nullptr, a, B * T, s);
}

size_t svd_prefix_attention_workspace_bytes(int64_t B, int32_t T, int32_t q_heads,
                                            int32_t kv_heads, int32_t head_dim, int64_t max_len,
                                            int64_t n_groups) {
  PrefixLayout l;
  return prefix_layout(B, T, q_heads, kv_heads, head_dim, max_len, n_groups, l) ? l.total : 0;
}

int svd_prefix_attention(const svd_cache_t *cache, const void *q, int64_t q_stride,
                         const int32_t *ctx_len, const int32_t *n_nodes, const uint32_t *anc,
                         const int32_t *depth, const int32_t *share_off, int64_t n_groups,
                         float scale, float cap, const float *slopes, int64_t B, int32_t T,
                         int32_t q_heads, void *out, float *lse, void *workspace,
                         size_t workspace_bytes, void *hip_stream) {
  CacheView c;
  int rc = cache_view(cache, c);
  if (rc != SVD_OK) return rc;
  const int D = cache->head_dim;
  const int64_t room = (int64_t)c.max_pages << c.page_shift;
  float cs;
  rc = attn_check(c, D, q, q_stride, ctx_len, scale, B, T, q_heads, out, workspace, cs);
  if (rc != SVD_OK) return rc;
  if ((share_off != nullptr) != (n_groups > 0)) return SVD_EINVAL;
  if (slopes && anc && !depth) return SVD_EINVAL;  // a tree's distances need its depths
  // a capped score is off by up to 2^-21 of the cap, 2^-7 at kMostCap: past it by too much
  if (!(cap >= 0.0f && cap <= kMostCap)) return SVD_EINVAL;
  float cap_in = 0.0f, cap_out = 0.0f;
  if (cap > 0.0f) {
    cap_in = (float)(2.0 * 1.4426950408889634 * (double)scale / (double)cap);
    cap_out = (float)(1.4426950408889634 * (double)cap);
    if (!(std::isnormal(cap_in) && std::isnormal(cap_out)))
      return SVD_EINVAL;
  }
  PrefixLayout l;
  if (!prefix_layout(B, T, q_heads, c.Hkv, D, room, n_groups, l)) return SVD_EINVAL;
  if (workspace_bytes < l.total) return SVD_EWORKSPACE;
  if (attn_overlap(q, q_stride, out, B * T, (uint64_t)q_heads * D * 2)) return SVD_EINVAL;
  char *const ws = static_cast<char *>(workspace);
  AttnArgs a = attn_args(c, q, q_stride, ctx_len, n_nodes, anc, cs, B, T, q_heads, out, lse);
  a.cap_in = cap_in;
  a.cap_out = cap_out;
  a.slopes = slopes;
  a.depth = anc ? depth : nullptr;  // a chain's depths are its nodes' numbers
  a.part_o = reinterpret_cast<float *>(ws + l.part_o);
  a.part_ms = reinterpret_cast<float *>(ws + l.part_ms);
  const AttnPlan own = attn_plan(B, T, q_heads, c.Hkv, D, room);
  attn_split(a, own, B * c.Hkv * own.S);
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if (n_groups > 0) {
    ShareArgs sh;
    sh.off = share_off;
    sh.ctx_len = ctx_len;
    sh.n_nodes = n_nodes;
    sh.table = c.table;
    sh.B = B;
    sh.G = n_groups;
    sh.room = room;
    sh.T = T;
    sh.max_pages = c.max_pages;
    sh.page_shift = c.page_shift;
    sh.group = a.group;
    sh.heads = c.Hkv;
    sh.m_rows = share_rows(B, T, a.group, n_groups);
    sh.tile = kSharedTile;
    sh.seqs = reinterpret_cast<ShareSeq *>(ws + l.seqs);
    sh.nodes = reinterpret_cast<int32_t *>(ws + l.nodes);
    sh.groups = reinterpret_cast<ShareGroup *>(ws + l.groups);
    sh.cut = reinterpret_cast<ShareCut *>(ws + l.cut);
    CallTimer tm;
    SVD_LAUNCH(tm, SVD_KERNEL_SHARE, s, kr_share, dim3((unsigned)n_groups), dim3(kShareBlock), s,
               sh);
    if (n_groups > 1)
      SVD_LAUNCH(tm, SVD_KERNEL_SHARE, s, kr_share_cut, dim3(1), dim3(kShareBlock), s, sh);
    a.seqs = sh.seqs;
    a.groups = sh.groups;
    a.cut = sh.cut;
    a.nodes = sh.nodes;
    a.share_rows = sh.m_rows;
    float *const o = reinterpret_cast<float *>(ws + l.share_o);
    float *const ms = reinterpret_cast<float *>(ws + l.share_ms);
    a.share_o = o;
    a.share_ms = ms;
    rc = shared_kind(cache, c, a, n_groups, o, ms, s);
    if (rc != SVD_OK) return rc;
  }
  return cap > 0.0f || slopes ? attn_kind<kShaped>(cache, own, c, a, q_heads, s)
                              : attn_kind<kTree>(cache, own, c, a, q_heads, s);
}

}  // extern "C"
