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
// vocabulary columns in registers for all rows of the prefix, and the row loop
// touches memory for logits only.  Path tokens differ from row to row; the few
// nodes whose token falls into the range are kept as a list, and the columns
// that hold one look through it row by row.
#pragma once

#include "svd_device.hpp"

namespace svd {

constexpr int kAdjBlock = 512;
constexpr int kAdjRange = 8192;      // most vocabulary tokens per workgroup
constexpr int kAdjRangeMin = 1024;   // a workgroup's range when there are few rows
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

__device__ __forceinline__ uint16_t adj_bf16(float x) {
  return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// element i of a 16-byte vector
template <typename E>
__device__ __forceinline__ void adj_set(vec16 &w, int i, float x) {
  if constexpr (sizeof(typename E::elem) == 4) {
    w[i] = __float_as_uint(x);
  } else {
    const uint32_t h = adj_bf16(x);
    const uint32_t old = w[i >> 1];
    w[i >> 1] = (i & 1) ? (old & 0xffffu) | (h << 16) : (old & 0xffff0000u) | h;
  }
}

__device__ __forceinline__ float adj_apply(float z, bool seen, int count, float r, float f,
                                           float pr) {
  if (seen) z = z > 0.0f ? z / r : z * r;
  if (count > 0) z = (z - f * (float)count) - pr;
  return z;
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
  __shared__ uint32_t path[PATH];  // node << 13 | token - v0
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
  const bool bad = rows_b < 0 || rows_b > T || hlen < 0 || hlen > a.hist_stride;
  const int t1 = min(t0 + a.row_step, bad ? T : rows_b);
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
    if constexpr (kBias) bias[i] = 0.0f;
  }
  if (tid == 0) n_path = dup = 0;
  __syncthreads();
  if (hlen > 0) {
    const int32_t *h = a.history + b * a.hist_stride;
    const int made = a.prompt_len ? a.prompt_len[b] : 0;
    for (int i = tid; i < hlen; i += kAdjBlock) {
      const uint32_t v = (uint32_t)(h[i] - v0);
      if (h[i] >= 0 && v < (uint32_t)nv) {
        atomicOr(&cnt[v], kAdjSeen);
        if (i >= made) atomicAdd(&cnt[v], 1u);
      }
    }
  }
  if (a.tokens) {
    for (int t = tid; t < rows_b; t += kAdjBlock) {
      const int x = a.tokens[b * T + t];
      const uint32_t v = (uint32_t)(x - v0);
      if (x >= 0 && v < (uint32_t)nv) {
        atomicOr(&cnt[v], kAdjPath);
        path[atomicAdd(&n_path, 1)] = ((uint32_t)t << 13) | v;
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
    for (int i = tid; i < nv; i += kAdjBlock) bias[i] = 0.0f;
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
  const float f = a.frequency ? a.frequency[b] : 0.0f;
  const float pr = a.presence ? a.presence[b] : 0.0f;
  const bool rep = a.repetition != nullptr;
  const int MW = (a.V + 31) / 32;
  const int np = n_path;

  // how often token v of the range is on row t's path
  auto on_path = [&](int t, uint32_t v) {
    int n = 0;
    for (int i = 0; i < np; ++i) {
      const uint32_t e = path[i];
      if ((e & 8191u) != v) continue;
      const int node = (int)(e >> 13);
      n += a.anc ? (int)((a.anc[(b * T + t) * W + (node >> 5)] >> (node & 31)) & 1u) : node <= t;
    }
    return n;
  };
  auto adjust = [&](float z, int t, int v, uint32_t c) {
    int n = (int)(c & kAdjCount);
    bool seen = (c & kAdjSeen) != 0;
    if (c & kAdjPath) {
      const int m = on_path(t, (uint32_t)v);
      n += m;
      seen |= m > 0;
    }
    z = adj_apply(z, rep && seen, n, r, f, pr);
    if constexpr (kBias) z += bias[v];
    return z;
  };

  const int ncol = nv / P;
  for (int col = tid; col < ncol; col += kAdjBlock) {
    const int v = col * P;
    uint32_t c[P];
    bool touched = false;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      c[i] = cnt[v + i];
      touched |= c[i] != 0;
      if constexpr (kBias) touched |= bias[v + i] != 0.0f;
    }
    for (int t = t0; t < t1; ++t) {
      uint32_t ok = (1u << P) - 1;
      bool poison = false;
      if (a.allow) {
        const int m = a.allow_index[b * T + t];
        if (m >= a.n_masks) poison = true;
        else if (m >= 0)
          ok &= a.allow[(int64_t)m * MW + ((v0 + v) >> 5)] >> ((v0 + v) & 31);
      }
      if (a.in_place && !touched && !poison && ok == (1u << P) - 1) continue;
      const int64_t at = (int64_t)t * a.V + v;
      vec16 w = *reinterpret_cast<const V_ *>(src + at);
      if (touched) {
        float x[P];
        E::unpack(w, x);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          bool mine = c[i] != 0;
          if constexpr (kBias) mine |= bias[v + i] != 0.0f;
          if (mine) adj_set<E>(w, i, adjust(x[i], t, v + i, c[i]));
        }
      }
      if (ok != (1u << P) - 1) {
#pragma unroll
        for (int i = 0; i < P; ++i)
          if (!((ok >> i) & 1)) adj_set<E>(w, i, kNegInf);
      }
      if (poison) {
#pragma unroll
        for (int i = 0; i < P; ++i) adj_set<E>(w, i, nan);
      }
      *reinterpret_cast<V_ *>(dst + at) = w;
    }
  }
  // the elements behind the last whole column
  const int left = nv - ncol * P;
  for (int i = tid; i < left * (t1 - t0); i += kAdjBlock) {
    const int t = t0 + i / left, v = ncol * P + i % left;
    const int64_t at = (int64_t)t * a.V + v;
    bool ok = true, poison = false;
    if (a.allow) {
      const int m = a.allow_index[b * T + t];
      if (m >= a.n_masks) poison = true;
      else if (m >= 0) ok = (a.allow[(int64_t)m * MW + ((v0 + v) >> 5)] >> ((v0 + v) & 31)) & 1u;
    }
    T_ e = src[at];
    uint32_t c = cnt[v];
    bool mine = c != 0;
    if constexpr (kBias) mine |= bias[v] != 0.0f;
    float z = adjust(E::at(src, at), t, v, c);
    if (!ok) z = kNegInf;
    if (poison) z = nan;
    if (mine || !ok || poison) {
      if constexpr (sizeof(T_) == 4) e = z;
      else e = adj_bf16(z);
    }
    dst[at] = e;
  }
}

}  // namespace svd
