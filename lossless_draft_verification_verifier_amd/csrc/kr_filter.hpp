// kr_filter.hpp -- the tokens that temperature, min-p, top-k and top-p keep of a row of
// logits, and draws among them.
//
// With w_i = exp((z_i - max z) / T), a token is kept when w_i >= min_p; of those the
// first top_k by falling logit, the lower index first among equal ones; of those the
// shortest beginning of that order whose mass is at least top_p of the mass of all of
// them.  So what is kept is a threshold: every token above a key, and the first few of
// those at it.  Both cuts are the same search, for the place where a running sum over
// falling keys (of ones, of weights) reaches a target: a histogram over the leading bits
// of the keys, the bin that the target falls into, then the same over its next bits.
//
// Weights are whole numbers: w_i * 2^s rounded once, s = 62 - ceil(log2 V) (at most 50), from
// an fp64 exponential.  Their sums are exact, so that neither the atomics' order nor how
// a row is divided can change a result; the rounding is 2^-45 of the largest weight at
// V = 152064, less than what fp64 sums of that many terms lose.
//
// One workgroup per row.  These passes take any row; kr_filter_row.hpp's are faster but for
// more than 256 rows of a small vocabulary, where four of these share a CU: 8192 rows of 2048
// bf16 tokens, top-k and top-p, in 218 us, 67 MB moved.  The searches' LDS counts and scans, one
// after another, bound them, not the bytes.
#pragma once

#include "kr_draw.hpp"

namespace svd {

constexpr int kFilterBlock = 1024;
constexpr int kFilterBins = 4096;   // of the first search step
constexpr uint64_t kSample = 4;     // the purpose of a draw's uniforms (after kBonus)

struct FilterArgs {
  const int32_t *n_rows, *top_k;
  const float *temperature, *top_p, *min_p;
  int64_t V, slab;  // slab: tokens of a part, a multiple of 8 * kFilterBlock
  int T, K, shift;  // shift: weights are multiples of 2^-shift
  const double *u;        // [B][K][T] or null: the counter hash
  uint64_t seed, row_base;
  int32_t *token;         // [B][K][T]
  float *logprob;         // [B][K][T] or null
};

// An order-preserving key of a logit: larger keys for larger values, one for both zeros.
__device__ __forceinline__ uint32_t logit_key(float z) {
  const uint32_t u = __float_as_uint(z + 0.0f);
  return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k);
}

// What a row keeps: keys above `key`, and of the tokens at it those below index `tie`.
struct Kept {
  uint32_t key;
  int64_t tie;
  __device__ bool has(uint32_t k, int64_t i) const { return k > key || (k == key && i < tie); }
};

template <int NT>
struct FilterLds {
  unsigned long long hist[kFilterBins];
  unsigned long long slabs[NT];
  unsigned long long wave[NT / 64 + 1];
  unsigned long long found[4];
  float red[NT / 64 + 1];
  int flag;
  ExpTable tab;
};

// The sums of x over the threads before this one; total: over all of them.
template <int NT>
__device__ __forceinline__ unsigned long long block_scan(unsigned long long x,
                                                         unsigned long long &total,
                                                         unsigned long long *lds /* NT / 64 */) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  unsigned long long up = x;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const unsigned long long p = __shfl_up(up, off, 64);
    if (lane >= off) up += p;
  }
  if (lane == 63) lds[w] = up;
  __syncthreads();
  unsigned long long before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) {
    if (i == w) before = all;
    all += lds[i];
  }
  __syncthreads();
  total = all;
  return before + up - x;
}

// The logits of a row, f(index, value) for every token: with kVec a 16-byte piece of P tokens
// per thread and NT * P at a time, else one per thread and NT at a time.
template <typename E, bool kVec, int NT, typename F>
__device__ __forceinline__ void filter_visit(const typename E::elem *row, int64_t lo, int64_t hi,
                                             F &&f) {
  if constexpr (kVec) {
    constexpr int P = E::kPerVec;
    for (int64_t i = lo + (int64_t)threadIdx.x * P; i < hi; i += (int64_t)NT * P) {
      float x[P];
      E::unpack(*reinterpret_cast<const vec16 *>(row + i), x);
#pragma unroll
      for (int e = 0; e < P; ++e) f(i + e, x[e]);
    }
  } else {
    for (int64_t i = lo + threadIdx.x; i < hi; i += NT) f(i, E::at(row, i));
  }
}

template <typename E, bool kVec, int NT>
struct FilterRow {
  const typename E::elem *row;
  const FilterArgs &a;
  FilterLds<NT> &l;
  float m;        // the largest logit
  double c;       // 256 log2(e) / temperature
  double unit;    // 2^shift

  __device__ unsigned long long weight(float z) const {
    const double x = ((double)z - (double)m) * c;
    const double w = __builtin_fma(exp2_256(x, l.tab), unit, 0x1p52);
    return __builtin_bit_cast(unsigned long long, w) & 0xfffffffffffffull;
  }

  // The key at which the sum of weigh(token) over falling keys, tokens with
  // take(token) only, reaches `target` (1 at least, the total at most), and the sum
  // above that key.
  template <typename Take, typename Weigh>
  __device__ void search(unsigned long long target, Take &&take, Weigh &&weigh, uint32_t &key,
                         unsigned long long &above) {
    constexpr bool kShort = sizeof(typename E::elem) == 2;  // bf16: 16 bits of key
    constexpr int kSteps = kShort ? 2 : 3;
    constexpr int first[3] = {12, kShort ? 4 : 10, 10};
    uint32_t prefix = 0;  // the bits found so far, on the left
    int bits = 0;
    above = 0;
#pragma unroll
    for (int step = 0; step < kSteps; ++step) {
      const int nb = first[step], bins = 1 << nb;
      for (int i = threadIdx.x; i < bins; i += NT) l.hist[i] = 0;
      __syncthreads();
      filter_visit<E, kVec, NT>(row, 0, a.V, [&](int64_t i, float z) {
        const uint32_t k = logit_key(z);
        if ((bits == 0 || k >> (32 - bits) == prefix >> (32 - bits)) && take(k, i))
          atomicAdd(&l.hist[(k << bits) >> (32 - nb)], weigh(z));
      });
      __syncthreads();
      // bins by falling key, a run of them per thread
      const int per = (bins + NT - 1) / NT;
      unsigned long long mine = 0, total;
      for (int j = 0; j < per; ++j) {
        const int at = bins - 1 - ((int)threadIdx.x * per + j);
        if (at >= 0) mine += l.hist[at];
      }
      unsigned long long upto = above + block_scan<NT>(mine, total, l.wave);
      if (upto < target && upto + mine >= target) {
        for (int j = 0; j < per; ++j) {
          const int at = bins - 1 - ((int)threadIdx.x * per + j);
          const unsigned long long h = l.hist[at];
          if (upto + h >= target) {
            l.found[0] = at;
            l.found[1] = upto;
            break;
          }
          upto += h;
        }
      }
      __syncthreads();
      prefix |= (uint32_t)l.found[0] << (32 - bits - nb);
      above = l.found[1];
      bits += nb;
      __syncthreads();
    }
    // bf16 keys: the low half is the sign's fill
    key = kShort ? prefix | (prefix >> 31 ? 0u : 0xffffu) : prefix;
  }

  // The sums of weigh(token) over the parts of the row, in l.slabs.
  template <typename Weigh>
  __device__ void slab_sums(Weigh &&weigh) {
    for (int i = threadIdx.x; i < NT; i += NT) l.slabs[i] = 0;
    __syncthreads();
    int s = 0;
    for (int64_t lo = 0; lo < a.V; lo += a.slab, ++s) {
      unsigned long long sum = 0;
      filter_visit<E, kVec, NT>(row, lo, min(lo + a.slab, a.V),
                            [&](int64_t i, float z) { sum += weigh(i, z); });
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
      if ((threadIdx.x & 63) == 0 && sum) atomicAdd(&l.slabs[s], sum);
    }
    __syncthreads();
  }

  // The first index up to which the sum of weigh(token) reaches `target` (1 at least, the
  // total at most), from the parts' sums.
  template <typename Weigh>
  __device__ int64_t locate(unsigned long long target, Weigh &&weigh) {
    const int n = (int)((a.V + a.slab - 1) / a.slab);
    const unsigned long long mine = (int)threadIdx.x < n ? l.slabs[threadIdx.x] : 0;
    unsigned long long total;
    const unsigned long long upto = block_scan<NT>(mine, total, l.wave);
    if (upto < target && upto + mine >= target) {
      l.found[0] = threadIdx.x;
      l.found[1] = upto;
    }
    __syncthreads();
    const int64_t lo0 = (int64_t)l.found[0] * a.slab, hi0 = min(lo0 + a.slab, a.V);
    unsigned long long before = l.found[1];
    __syncthreads();
    constexpr int P = 8;
    for (int64_t lo = lo0; lo < hi0; lo += P * NT) {
      // 8 tokens per thread
      const int64_t i0 = lo + (int64_t)threadIdx.x * P;
      unsigned long long w[P], sum = 0;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        w[e] = i0 + e < hi0 ? weigh(i0 + e, E::at(row, i0 + e)) : 0;
        sum += w[e];
      }
      unsigned long long at = before + block_scan<NT>(sum, total, l.wave);
      if (at < target && at + sum >= target) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
          if (at < target && at + w[e] >= target) l.found[2] = (unsigned long long)(i0 + e);
          at += w[e];
        }
      }
      before += total;
      __syncthreads();
      if (before >= target) break;
    }
    const int64_t r = (int64_t)l.found[2];
    __syncthreads();
    return r;
  }

  // The first index behind the n-th token at `key`.
  __device__ int64_t behind_tie(uint32_t key, unsigned long long n) {
    auto at_key = [&](int64_t, float z) -> unsigned long long { return logit_key(z) == key; };
    slab_sums(at_key);
    return locate(n, at_key) + 1;
  }
};

template <typename E>
__device__ __forceinline__ void fill_nan(typename E::elem *to, int64_t V) {
  typename E::elem nan;
  if constexpr (sizeof(nan) == 2) nan = 0x7fc0;
  else nan = __uint_as_float(0x7fc00000u);
  for (int64_t i = threadIdx.x; i < V; i += blockDim.x) to[i] = nan;
}

// Draw k of row (b, t): its uniform; the sum it is drawn at, 1 to total; its outputs.
__device__ __forceinline__ double draw_uniform(const FilterArgs &a, int64_t b, int k, int t) {
  if (a.u) return a.u[(b * a.K + k) * a.T + t];
  return counter_uniform(a.seed, a.row_base + (uint64_t)b,
                         (uint64_t)k * (uint64_t)a.T + (uint64_t)t, kSample);
}
__device__ __forceinline__ unsigned long long draw_target(double u, unsigned long long total) {
  const unsigned long long x = (unsigned long long)(u * (double)total);
  return x < total ? x + 1 : total;
}
__device__ __forceinline__ void put_draw(const FilterArgs &a, int64_t b, int k, int t, int64_t v,
                                         float z, float m, float temp, unsigned long long total) {
  const int64_t at = (b * a.K + k) * a.T + t;
  a.token[at] = (int32_t)v;
  if (a.logprob)
    a.logprob[at] = v < 0 ? __uint_as_float(0x7fc00000u)
                          : (float)(((double)z - (double)m) / (double)temp -
                                    log(ldexp((double)total, -a.shift)));
}

// What a prefix asks for, and whether a row of it has an answer.
struct FilterAsk {
  float t, p, least;
  int64_t k;
  bool bad;
};
__device__ __forceinline__ FilterAsk filter_ask(const FilterArgs &a, int64_t b) {
  FilterAsk q;
  q.t = a.temperature ? a.temperature[b] : 1.0f;
  q.p = a.top_p ? a.top_p[b] : 1.0f;
  q.least = a.min_p ? a.min_p[b] : 0.0f;
  q.k = a.top_k ? a.top_k[b] : 0;
  const int n = a.n_rows ? a.n_rows[b] : a.T;
  q.bad = !(q.t >= 0.0f && q.t < __builtin_huge_valf()) || q.p != q.p || q.least != q.least ||
          n < 0 || n > a.T;
  if (q.t == 0.0f) {  // the most likely token alone
    q.t = 1.0f;
    q.k = 1;
  }
  return q;
}

// The largest logit of a row and what it keeps; false: no answer (a NaN, +inf, or all -inf).
template <typename E, bool kVec, int NT>
__device__ __forceinline__ bool filter_row(FilterRow<E, kVec, NT> &r, const FilterAsk &q, Kept &kept) {
  FilterLds<NT> &l = r.l;
  const FilterArgs &a = r.a;
  exp_table_init<NT>(l.tab);
  if (threadIdx.x == 0) l.flag = 0;
  __syncthreads();
  float m = kNegInf;
  bool bad = false;
  filter_visit<E, kVec, NT>(r.row, 0, a.V, [&](int64_t, float z) {
    bad |= !(z < __builtin_huge_valf());
    m = fmaxf(m, z);
  });
  if (__any(bad) && (threadIdx.x & 63) == 0) l.flag = 1;
  m = block_max<NT / 64>(m, l.red);
  if (l.flag || m == kNegInf) return false;
  r.m = m;
  r.c = exp2_scale(q.t);
  r.unit = ldexp(1.0, a.shift);
  kept.key = 0;
  kept.tie = a.V;
  uint32_t least = 0;  // the lowest key that min_p leaves
  if (q.least > 0.0f) {
    // the least float z with (z - m) / t >= log(min_p)
    const double zt = (double)m + (double)q.t * log((double)q.least);
    float z = (float)fmax(zt, -3.5e38);
    if ((double)z < zt) z = nextafterf(z, __builtin_huge_valf());
    least = logit_key(fminf(z, m));
  }
  auto take_least = [&](uint32_t k, int64_t) { return k >= least; };
  auto one = [](float) { return 1ull; };
  if (q.k > 0 && q.k < a.V) {
    // all of them when there are no more than k
    unsigned long long n = 0, total;
    filter_visit<E, kVec, NT>(r.row, 0, a.V, [&](int64_t, float z) { n += logit_key(z) >= least; });
    block_scan<NT>(n, total, l.wave);
    if (total > (unsigned long long)q.k) {
      uint32_t key;
      unsigned long long above;
      r.search((unsigned long long)q.k, take_least, one, key, above);
      kept.key = key;
      kept.tie = r.behind_tie(key, (unsigned long long)q.k - above);
    }
  }
  if (kept.key < least) {
    kept.key = least;  // the tokens at it included
    kept.tie = a.V;
  }
  if (q.p < 1.0f) {
    const Kept k0 = kept;
    auto take = [&](uint32_t k, int64_t i) { return k0.has(k, i); };
    unsigned long long sum = 0, total;
    filter_visit<E, kVec, NT>(r.row, 0, a.V, [&](int64_t i, float z) {
      if (take(logit_key(z), i)) sum += r.weight(z);
    });
    block_scan<NT>(sum, total, l.wave);
    const double want = ceil(fmax((double)q.p, 0.0) * (double)total);
    unsigned long long target = (unsigned long long)want;
    target = target < 1 ? 1 : target > total ? total : target;
    uint32_t key;
    unsigned long long above;
    r.search(target, take, [&](float z) { return r.weight(z); }, key, above);
    const unsigned long long w = r.weight(key_logit(key));
    const unsigned long long n = (target - above + w - 1) / w;  // tokens at the key
    const int64_t tie = r.behind_tie(key, n);
    kept.tie = key == k0.key ? min(tie, k0.tie) : tie;
    kept.key = key;
  }
  return true;
}

// ---------------------------------------------------------------------------
// A row by any number of passes over memory: vocabularies of any size, values of any size.

template <typename E, bool kVec, int NT>
__device__ __forceinline__ void filter_any(const typename E::elem *logits, typename E::elem *out,
                                           const FilterArgs &a, const FilterAsk &q, int64_t bt,
                                           FilterLds<NT> &lds) {
  using elem = typename E::elem;
  const int64_t off = bt * a.V;
  FilterRow<E, kVec, NT> r{logits + off, a, lds, 0.0f, 0.0, 0.0};
  Kept kept;
  const bool ok = !q.bad && filter_row<E, kVec>(r, q, kept);
  elem *const to = out + off;
  if (!ok) return fill_nan<E>(to, a.V);
  const elem none = sizeof(elem) == 2 ? (elem)0xff80 : (elem)kNegInf;
  if constexpr (kVec) {
    constexpr int P = E::kPerVec;
    for (int64_t i = (int64_t)threadIdx.x * P; i < a.V; i += (int64_t)NT * P) {
      const vec16 w = *reinterpret_cast<const vec16 *>(r.row + i);
      float x[P];
      E::unpack(w, x);
      elem y[P];
      __builtin_memcpy(y, &w, 16);
#pragma unroll
      for (int e = 0; e < P; ++e)
        if (!kept.has(logit_key(x[e]), i + e)) y[e] = none;
      vec16 v;
      __builtin_memcpy(&v, y, 16);
      *reinterpret_cast<vec16 *>(to + i) = v;
    }
  } else {
    for (int64_t i = threadIdx.x; i < a.V; i += NT)
      to[i] = kept.has(logit_key(E::at(r.row, i)), i) ? r.row[i] : none;
  }
}

template <typename E, bool kVec, int NT>
__device__ __forceinline__ void sample_any(const typename E::elem *logits, const FilterArgs &a,
                                           const FilterAsk &q, int64_t b, int t, FilterLds<NT> &lds) {
  FilterRow<E, kVec, NT> r{logits + (b * a.T + t) * a.V, a, lds, 0.0f, 0.0, 0.0};
  Kept kept;
  const bool ok = !q.bad && filter_row<E, kVec>(r, q, kept);
  auto weigh = [&](int64_t i, float z) -> unsigned long long {
    return kept.has(logit_key(z), i) ? r.weight(z) : 0ull;
  };
  unsigned long long total = 0;
  if (ok) {
    r.slab_sums(weigh);
    block_scan<NT>(lds.slabs[threadIdx.x], total, lds.wave);
  }
  for (int k = 0; k < a.K; ++k) {
    const double u = draw_uniform(a, b, k, t);
    int64_t v = -1;
    if (ok && u >= 0.0 && u < 1.0) v = r.locate(draw_target(u, total), weigh);
    if (threadIdx.x == 0)
      put_draw(a, b, k, t, v, v < 0 ? 0.0f : E::at(r.row, v), r.m, q.t, total);
  }
}

template <typename E, bool kVec, int NT>
__global__ __launch_bounds__(NT) void kr_filter_any(const typename E::elem *logits,
                                                              typename E::elem *out,
                                                              FilterArgs a) {
  __shared__ FilterLds<NT> lds;
  const int64_t b = blockIdx.x / a.T;
  const FilterAsk q = filter_ask(a, b);
  if (!q.bad && a.n_rows && (int)(blockIdx.x % a.T) >= a.n_rows[b]) return;
  filter_any<E, kVec, NT>(logits, out, a, q, blockIdx.x, lds);
}

template <typename E, bool kVec, int NT>
__global__ __launch_bounds__(NT) void kr_sample_any(const typename E::elem *logits,
                                                              FilterArgs a) {
  __shared__ FilterLds<NT> lds;
  const int64_t b = blockIdx.x / a.T;
  const int t = (int)(blockIdx.x % a.T);
  const FilterAsk q = filter_ask(a, b);
  if (!q.bad && a.n_rows && t >= a.n_rows[b]) return;
  sample_any<E, kVec, NT>(logits, a, q, b, t, lds);
}

}  // namespace svd
