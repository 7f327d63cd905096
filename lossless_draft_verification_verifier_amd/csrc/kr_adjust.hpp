// kr_adjust.hpp -- penalties, biases and grammar masks on logit rows.
//
// Row (b, t) predicts the token after node t of prefix b's tree.  A token that
// occurs in the prefix's history or on the node's path gets
//   z = z > 0 ? z / r : z * r                     (repetition)
//   z = z - f * count - pr * [count > 0]          (frequency, presence; count:
//       occurrences in the generated part of the history and on the path)
// then every token its bias, and -inf where the row's grammar mask forbids it.
//
// Bound by HBM: each row is read and written once (in place: only the 16-byte
// vectors that change).  A workgroup takes one prefix and a range of the
// vocabulary and counts the history's tokens of that range in LDS: dense
// integer counters, so a repeated token needs no search and the order of the
// additions cannot show.  A thread then holds the adjustments of its few
// vocabulary columns in registers for all rows of the prefix, as one factor and
// one summand per token, and the row loop touches memory for logits only.  Path
// tokens differ from row to row; the few nodes whose token falls into the range
// are kept as a list, the row loop passes their tokens through as they are, and
// a pass over (row, node) pairs sets them afterwards.
//
// Workgroups of 256 threads over 4096 tokens keep 8 of them on a CU.  2304 bf16 rows
// of 152064 (256 prefixes of 9 nodes, histories of 512 to 1024, a quarter of the rows
// masked): 268 us, 5.3 TB/s, against 334 for 512 threads over 8192 tokens and 288 for a
// copy of the rows.  516 fp32 rows of 100003 with histories to 32768, 300 biases and a
// mask on every row: 129 us, 3.2 TB/s.  Setting up a range is paid there once per chunk of
// its rows, of which there are ten so that the GPU is full: without the counts of the
// history it takes 115.
#pragma once

#include "kr_cache.hpp"
#include "svd_device.hpp"

namespace svd {

constexpr int kAdjBlock = 256;
constexpr int kAdjRange = 4096;      // most vocabulary tokens per workgroup
constexpr int kAdjRangeMin = 1024;   // a workgroup's range when there are few rows
constexpr int kAdjRowsMax = 256;     // most rows per workgroup
constexpr int kAdjPathSmall = 256;   // trees of at most this many nodes keep a short list
constexpr int kAdjPathMax = 4096;
constexpr uint32_t kAdjSeen = 1u << 31;   // the token occurs in the history
constexpr uint32_t kAdjPath = 1u << 30;   // some node holds the token
constexpr uint32_t kAdjCount = (1u << 30) - 1;

struct AdjustArgs {
  const int32_t *n_rows;
  const int32_t *history;
  int64_t hist_stride;
  const int32_t *hist_len, *prompt_len;
  const int32_t *tokens;
  const uint32_t *anc;
  const float *repetition, *frequency, *presence;
  const int32_t *bias_off, *bias_tok;
  const float *bias_val;
  int64_t n_bias;
  const uint32_t *allow;
  const int32_t *allow_index;
  int n_masks;
  int T, V, range, n_ranges, row_step, n_chunks;
  bool in_place;
};

// a load or store of 16 bytes at an address that is a multiple of the element only
typedef vec16 __attribute__((aligned(2))) vec16_at2;
typedef vec16 __attribute__((aligned(4))) vec16_at4;
template <typename E, bool kVec>
struct AdjVec;
template <typename E>
struct AdjVec<E, true> { using type = vec16; };
template <>
struct AdjVec<BF16, false> { using type = vec16_at2; };
template <>
struct AdjVec<F32, false> { using type = vec16_at4; };

// a vector of one value
template <typename E>
__device__ __forceinline__ vec16 adj_fill(float x) {
  const uint32_t u = sizeof(typename E::elem) == 4 ? __float_as_uint(x) : pack_bf16(x, x);
  return vec16{u, u, u, u};
}

// element i of a where bit i of m is set, of b elsewhere
template <typename E>
__device__ __forceinline__ vec16 adj_select(uint32_t m, const vec16 &a, const vec16 &b) {
  vec16 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t k;
    if constexpr (E::kPerVec == 4) {
      k = ((m >> j) & 1) ? 0xffffffffu : 0u;
    } else {
      k = (((m >> (2 * j)) & 1) ? 0x0000ffffu : 0u) | (((m >> (2 * j + 1)) & 1) ? 0xffff0000u : 0u);
    }
    r[j] = (a[j] & k) | (b[j] & ~k);
  }
  return r;
}

// grid: prefix x range x row chunk.  kVec: rows start 16-byte aligned.  In
// both forms a column is the 16 bytes of kPerVec tokens; the last, partial
// column of an odd vocabulary goes element by element.
template <typename E, bool kVec, bool kBias, int PATH>
__global__ __launch_bounds__(kAdjBlock) void kr_adjust(const typename E::elem *logits,
                                                       typename E::elem *out, AdjustArgs a) {
  using T_ = typename E::elem;
  using V_ = typename AdjVec<E, kVec>::type;
  constexpr int P = E::kPerVec;
  __shared__ uint32_t cnt[kAdjRange];
  __shared__ float bias[kBias ? kAdjRange : 1];
  __shared__ uint32_t path[PATH];  // node << 12 | token - v0; the top bit: an earlier entry has the token
  __shared__ int row_mask[kAdjRowsMax];  // the rows' masks: -1 for none, n_masks for a bad index
  __shared__ int n_path, dup;
  const int tid = threadIdx.x;
  const int per_b = a.n_ranges * a.n_chunks;
  const int64_t b = blockIdx.x / per_b;
  const int rem = blockIdx.x % per_b;
  const int v0 = (rem % a.n_ranges) * a.range;
  const int nv = min(a.range, a.V - v0);
  const int t0 = (rem / a.n_ranges) * a.row_step;
  const int T = a.T, W = (T + 31) / 32;
  const int rows_b = a.n_rows ? a.n_rows[b] : T;
  const int hlen = a.history ? a.hist_len[b] : 0;
  // a prefix whose lengths are out of range: NaN rows, which a verification reports as -1
  const bool no_rows = rows_b < 0 || rows_b > T;
  const bool bad = no_rows || hlen < 0 || hlen > a.hist_stride;
  const int t1 = min(t0 + a.row_step, no_rows ? T : rows_b);
  if (t0 >= t1) return;
  const T_ *src = logits + b * T * (int64_t)a.V + v0;
  T_ *dst = out + b * T * (int64_t)a.V + v0;
  const float nan = __uint_as_float(0x7fc00000u);
  if (bad) {
    for (int t = t0; t < t1; ++t)
      for (int i = tid; i < nv; i += kAdjBlock) {
        if constexpr (sizeof(T_) == 4) dst[(int64_t)t * a.V + i] = nan;
        else dst[(int64_t)t * a.V + i] = 0x7fc0;
      }
    return;
  }

  // counts, path list and biases of the range
  for (int i = tid; i < nv; i += kAdjBlock) {
    cnt[i] = 0;
    if constexpr (kBias) bias[i] = 0.0f;  // a count of 0, first
  }
  if (a.allow)
    for (int i = tid; i < t1 - t0; i += kAdjBlock)
      row_mask[i] = min(max(a.allow_index[b * T + t0 + i], -1), a.n_masks);
  if (tid == 0) n_path = dup = 0;
  __syncthreads();
  if (hlen > 0) {
    const int32_t *h = a.history + b * a.hist_stride;
    const int made = a.prompt_len ? a.prompt_len[b] : 0;
    for (int i0 = tid; i0 < hlen; i0 += 8 * kAdjBlock) {
      int x[8];  // loads of 8 tokens in flight
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = i0 + k * kAdjBlock < hlen ? h[i0 + k * kAdjBlock] : -1;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t v = (uint32_t)(x[k] - v0);
        if (x[k] >= 0 && v < (uint32_t)nv) {
          atomicOr(&cnt[v], kAdjSeen);
          if (i0 + k * kAdjBlock >= made) atomicAdd(&cnt[v], 1u);
        }
      }
    }
  }
  if (a.tokens) {
    for (int t = tid; t < rows_b; t += kAdjBlock) {
      const int x = a.tokens[b * T + t];
      const uint32_t v = (uint32_t)(x - v0);
      if (x >= 0 && v < (uint32_t)nv) {
        atomicOr(&cnt[v], kAdjPath);
        path[atomicAdd(&n_path, 1)] = ((uint32_t)t << 12) | v;
      }
    }
  }
  if constexpr (kBias) {
    const int64_t lo = max((int64_t)a.bias_off[b], (int64_t)0);
    const int64_t hi = min((int64_t)a.bias_off[b + 1], a.n_bias);
    // entries of a token named more than once add in the list's order: first
    // see whether there is one, counting in the array that will hold the sums
    uint32_t *seen = reinterpret_cast<uint32_t *>(bias);
    for (int64_t i = lo + tid; i < hi; i += kAdjBlock) {
      const int x = a.bias_tok[i];
      const uint32_t v = (uint32_t)(x - v0);
      if (x >= 0 && v < (uint32_t)nv && atomicAdd(&seen[v], 1u) != 0) dup = 1;
    }
    __syncthreads();
    const bool ordered = dup != 0;
    for (int i = tid; i < nv; i += kAdjBlock) bias[i] = -0.0f;
    __syncthreads();
    if (!ordered) {
      for (int64_t i = lo + tid; i < hi; i += kAdjBlock) {
        const int x = a.bias_tok[i];
        const uint32_t v = (uint32_t)(x - v0);
        if (x >= 0 && v < (uint32_t)nv) bias[v] = a.bias_val[i];
      }
    } else {  // each token has one thread, which walks the list
      for (int64_t i = lo; i < hi; ++i) {
        const int x = a.bias_tok[i];
        const uint32_t v = (uint32_t)(x - v0);
        if (x >= 0 && v < (uint32_t)nv && (int)(v % kAdjBlock) == tid) bias[v] += a.bias_val[i];
      }
    }
  }
  __syncthreads();

  const float r = a.repetition ? a.repetition[b] : 1.0f;
  const float inv = 1.0f / r;
  const float f = a.frequency ? a.frequency[b] : 0.0f;
  const float pr = a.presence ? a.presence[b] : 0.0f;
  const bool rep = r != 1.0f;
  const int MW = (int)(((int64_t)a.V + 31) / 32);  // V goes up to 2^31 - 1
  const int np = n_path;

  // what n counted occurrences and the bias add to token v; -0, which changes no value, is nothing
  auto summand = [&](int n, int v) {
    float x = n > 0 ? -(f * (float)n) - pr : -0.0f;
    if constexpr (kBias) x += bias[v];
    return x;
  };
  auto scaled = [&](float z, float add) {  // one rounding after the factor's
    return __builtin_fmaf(z, z > 0.0f ? inv : r, add);
  };
  // the mask of row t, the same for all lanes: nullptr for none; poison: an index behind the last
  auto mask_row = [&](int t, bool &poison) -> const uint32_t * {
    const int m = __builtin_amdgcn_readfirstlane(row_mask[t - t0]);
    poison = m >= a.n_masks;
    return m >= 0 && !poison ? a.allow + (int64_t)m * MW : nullptr;
  };

  for (int i = tid; i < np; i += kAdjBlock) {  // order of the list: any, the sums are whole numbers
    bool again = false;
    for (int j = 0; j < i; ++j) again |= ((path[j] ^ path[i]) & 4095u) == 0;
    if (again) atomicOr(&path[i], 0x80000000u);
  }

  constexpr uint32_t kAll = (1u << P) - 1;
  const int ncol = nv / P;
  for (int col = tid; col < ncol; col += kAdjBlock) {
    const int v = col * P;
    float add[P];
    uint32_t seen = 0, mine = 0, paths = 0;  // a bit per token
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const uint32_t c = cnt[v + i];
      add[i] = summand((int)(c & kAdjCount), v + i);
      const uint32_t on = (c & kAdjPath) != 0;
      paths |= on << i;
      seen |= (uint32_t)(rep && (c & kAdjSeen)) << i;
      mine |= (uint32_t)(!on && ((rep && (c & kAdjSeen)) || add[i] != 0.0f)) << i;
    }
    for (int t = t0; t < t1; ++t) {
      uint32_t ok = kAll;
      bool poison = false;
      if (a.allow) {
        const uint32_t *m = mask_row(t, poison);
        if (m) ok = ((m[(v0 + v) >> 5] >> ((v0 + v) & 31)) | paths) & kAll;
      }
      // in place, a vector that nothing changes is not touched
      if (a.in_place && !mine && !poison && ok == kAll) continue;
      vec16 w = __builtin_nontemporal_load(
          reinterpret_cast<const V_ *>(src + (int64_t)t * a.V + v));
      if (mine) {
        float x[P];
        E::unpack(w, x);
#pragma unroll
        for (int i = 0; i < P; ++i)
          x[i] = ((seen >> i) & 1) ? scaled(x[i], add[i]) : x[i] + add[i];
        vec16 y;
        if constexpr (P == 4) {
          y = vec16{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                    __float_as_uint(x[3])};
        } else {
          y = vec16{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4 % P], x[5 % P]),
                    pack_bf16(x[6 % P], x[7 % P])};
        }
        w = adj_select<E>(mine, y, w);
      }
      if (ok != kAll) w = adj_select<E>(ok, w, adj_fill<E>(kNegInf));
      if (poison) w = adj_select<E>(paths, w, adj_fill<E>(nan));
      __builtin_nontemporal_store(w, reinterpret_cast<V_ *>(dst + (int64_t)t * a.V + v));
    }
  }
  __syncthreads();
  // one element from its source value: token v with m nodes of its own on the row's path
  auto element = [&](int t, int v, int m) {
    const int64_t at = (int64_t)t * a.V + v;
    const uint32_t c = cnt[v];
    bool ok = true, poison = false;
    if (a.allow) {
      const int k = row_mask[t - t0];
      poison = k >= a.n_masks;
      if (k >= 0 && !poison)
        ok = (a.allow[(int64_t)k * MW + ((v0 + v) >> 5)] >> ((v0 + v) & 31)) & 1u;
    }
    T_ e = src[at];
    const int n = (int)(c & kAdjCount) + m;
    const float add = summand(n, v), z = E::at(src, at);
    const bool times = rep && (m > 0 || (c & kAdjSeen));
    float y = times ? scaled(z, add) : z + add;
    if (!ok) y = kNegInf;
    if (poison) y = nan;
    if (times || add != 0.0f || !ok || poison) {
      if constexpr (sizeof(T_) == 4) e = y;
      else e = (T_)pack_bf16(y, y);
    }
    dst[at] = e;
  };
  // tokens that nodes hold, once each: the row loop has left their source values
  for (int k = tid; k < np * (t1 - t0); k += kAdjBlock) {
    const int t = t0 + k / np;
    const uint32_t mine = path[k % np], v = mine & 4095u;
    if (mine >> 31) continue;
    int m = 0;
    for (int i = 0; i < np; ++i) {
      const uint32_t e = path[i];
      if ((e & 4095u) != v) continue;
      const int node = (int)((e & 0x7fffffffu) >> 12);
      m += a.anc ? (int)((a.anc[(b * T + t) * W + (node >> 5)] >> (node & 31)) & 1u) : node <= t;
    }
    element(t, (int)v, m);
  }
  // the elements behind the last whole column that no node holds
  const int left = nv - ncol * P;
  for (int i = tid; i < left * (t1 - t0); i += kAdjBlock) {
    const int t = t0 + i / left, v = ncol * P + i % left;
    if (!(cnt[v] & kAdjPath)) element(t, v, 0);
  }
}

}  // namespace svd
