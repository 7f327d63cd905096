// kr_filter_row.hpp -- filtered and sampled logits, a row held by one workgroup: the same
// results as kr_filter.hpp's passes, which are what a row falls back to.
//
// The search for a cut needs the tokens' counts and weights by falling logit.  Logits of
// bf16 have few values, so one pass counts every value there is: a counter in LDS for
// each upper half of a logit's bits between 2^-26 and 2^9 in magnitude, positive and
// negative (the counters' addresses are the bits themselves, less a constant), and one
// for zero.  The rest is a scan over 8961 counters: the weight of a value times its count
// is exact, so top-k, min-p and top-p are decided without looking at a token again.
// fp32 logits are counted (top-k) and weighed (top-p) by the same upper halves, and the
// tokens in the counter that holds the cut are gathered and searched by their lower
// halves.  Which of the tokens at the cut are kept goes by index: their number in each
// wave's share of the row, a scan, one wave's share again.
//
// A token at -2^9 or below has no counter.  That is no matter while it has no weight and no
// cut reaches down to it.  Where it does, and with other values outside the range (2^9 or
// more, or below 2^-26 but for zero) or more tokens around an fp32 cut than the list holds,
// the row falls back.
//
// NV > 0: the row's logits stay in registers, NV 16-byte pieces per thread (bf16 up to
// 155641 tokens, one workgroup per CU), and memory is read once, but for pieces with a token
// that has no counter, or a zero: these come again, token by token.  So rows behind a mask take
// longer, top-k and top-p of 2304 rows of 152064 bf16 logits 338 us with no -inf, 401 with one
// token of a hundred at -inf, 548 with half of them, 527 with 99 of a hundred (256 rows 41, 47,
// 63 and 61; in fp32 144, 155, 177 and 174).  NV = 0: every pass reads them again, which the
// 256 MB last-level cache serves.
//
// Bounds, on one MI355X.  2304 rows of 152064 bf16 logits, every prefix with settings of its
// own: 1.40 GB in 306 us, 4.6 TB/s, for 285 at a copy's rate (the general passes: 1151).  One
// round of 256 rows by time stamps: loads and counts 11 us, the scan of the counters 2, weights
// 1, the cut 3, ties 7, the store 7.  516 rows of 100003 fp32 logits, top-p alone: 257 us, the
// weights' exponentials (230 cycles per 64 tokens), three rounds (general: 783).  256 rows of
// bf16, 8 draws each: 53 us, half of them the second look at every token's weight (general:
// 236).  One row, one draw: 26 us (general: 163).
#pragma once

#include "kr_filter.hpp"

namespace svd {

constexpr int kSideBins = 35 << 7;           // counters of one sign
constexpr int kBinLo = (127 - 26) << 7;      // the upper half of 2^-26
constexpr int kRanks = 2 * kSideBins + 1;    // by falling value: positive, zero, negative
constexpr float kBinTop = 512.0f;            // magnitudes below it have counters
// Weights are found by a token's upper half with few steps: of each sign a slot for zero,
// one per counter, and one, without weight, for what lies past them.
constexpr int kSideSlots = kSideBins + 2;
constexpr int kSlots = 2 * kSideSlots;
constexpr int kRowEntries = 1024;            // (step, wave) records of a row at most

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// All waves arrive, and what they wrote to LDS is there; loads from memory stay on their way.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Inclusive sums over a wave's lanes by lane exchanges that stay in the vector unit: shifts
// inside rows of 16 lanes, then the last lane of a row, or of two, to those behind it.
template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t lanes_from(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kCtrl, kRows, 0xf, false);
}
template <int kCtrl, int kRows>
__device__ __forceinline__ unsigned long long lanes_from(unsigned long long x) {
  return (unsigned long long)lanes_from<kCtrl, kRows>((uint32_t)(x >> 32)) << 32 |
         lanes_from<kCtrl, kRows>((uint32_t)x);
}
template <typename T>
__device__ __forceinline__ T wave_scan(T x) {
  x += lanes_from<0x111, 0xf>(x);
  x += lanes_from<0x112, 0xf>(x);
  x += lanes_from<0x114, 0xf>(x);
  x += lanes_from<0x118, 0xf>(x);
  x += lanes_from<0x142, 0xa>(x);
  x += lanes_from<0x143, 0xc>(x);
  return x;
}
__device__ __forceinline__ uint32_t lane_value(uint32_t x, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)x, lane);
}
__device__ __forceinline__ unsigned long long lane_value(unsigned long long x, int lane) {
  return (unsigned long long)lane_value((uint32_t)(x >> 32), lane) << 32 |
         lane_value((uint32_t)x, lane);
}

// The largest of a wave's lanes, in lane 63.
__device__ __forceinline__ uint32_t wave_most(uint32_t x) {
  x = max(x, lanes_from<0x111, 0xf>(x));
  x = max(x, lanes_from<0x112, 0xf>(x));
  x = max(x, lanes_from<0x114, 0xf>(x));
  x = max(x, lanes_from<0x118, 0xf>(x));
  x = max(x, lanes_from<0x142, 0xa>(x));
  return max(x, lanes_from<0x143, 0xc>(x));
}

// The sums of x over the threads before this one; total: over all of them.
template <int NT, typename T>
__device__ __forceinline__ T row_scan(T x, T &total, unsigned long long *lds /* NT / 64 */) {
  constexpr int NW = NT / 64;
  static_assert(NW <= 16, "one row of lanes");
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const T up = wave_scan(x);
  if (lane == 63) lds[w] = up;
  lds_barrier();
  T of = (T)lds[lane & (NW - 1)];
  if (lane >= NW) of = 0;
  of = wave_scan(of);
  total = lane_value(of, NW - 1);
  const T before = w ? lane_value(of, w ? w - 1 : 0) : (T)0;
  lds_barrier();
  return before + up - x;
}

template <int NT>
struct RowLds {
  // counters: word u - kBinLo for an upper half u, so negative ones from 32768 on; before
  // these the zeros' one
  static constexpr int kNeg = 32768;
  static constexpr int kWords = kNeg + kSideBins;
  // in the gap between them: weights by slot, then the keys gathered around a cut
  static constexpr int kMassAt = kSideBins;
  static constexpr int kListAt = kMassAt + 2 * kSlots;
  static constexpr int kListCap = kNeg - 1 - kListAt;
  static_assert(kMassAt % 2 == 0 && kListCap >= 4096, "");
  uint32_t h[kWords];
  unsigned long long sums[kRowEntries];      // of the records, then of what is before each
  unsigned long long wave[NT / 64];
  unsigned long long found[2];               // a target's place: what is above it
  int rank, n_list, tie;
  uint32_t flags, best;
  ExpTable tab;
  __device__ unsigned long long *mass() {
    return reinterpret_cast<unsigned long long *>(h + kMassAt);
  }
  __device__ uint32_t *list() { return h + kListAt; }
};
enum : uint32_t { kRowBad = 1, kRowOdd = 2, kRowLow = 4 };

// The upper half of the logits of rank r, and the word of its counter.
__device__ __forceinline__ uint32_t rank_bits(int r) {
  return r < kSideBins ? (uint32_t)(kBinLo + kSideBins - 1 - r)
                       : r == kSideBins ? 0u : 0x8000u | (uint32_t)(kBinLo + r - kSideBins - 1);
}
__device__ __forceinline__ int rank_word(int r) {
  return r < kSideBins ? kSideBins - 1 - r : RowLds<1024>::kNeg - 1 + (r - kSideBins);
}
__device__ __forceinline__ float rank_value(int r) { return __uint_as_float(rank_bits(r) << 16); }
__device__ __forceinline__ int bits_slot(uint32_t u) {
  const int a = (int)(u & 0x7fffu) - kBinLo;
  return (int)(u >> 15) * kSideSlots + 1 + min(max(a, -1), kSideBins);
}
__device__ __forceinline__ int rank_slot(int r) { return bits_slot(rank_bits(r)); }

template <typename E, int NT, int NV>
struct HeldRow {
  using elem = typename E::elem;
  using Lds = RowLds<NT>;
  static constexpr int P = E::kPerVec;
  static constexpr bool kShort = sizeof(elem) == 2;
  static constexpr int PT = (kRanks + NT - 1) / NT;  // ranks per thread
  const elem *row;
  const FilterArgs &a;
  Lds &l;
  int shift;          // elements before the row in its first 16 bytes
  int at;             // the first token of this thread's first piece
  int n;              // tokens
  int steps;          // pieces per thread
  float m;            // the largest logit
  double c, unit;
  vec16 r[NV ? NV : 1];

  __device__ __forceinline__ HeldRow(const elem *p, const FilterArgs &args, Lds &lds)
      : row(p), a(args), l(lds), m(0.0f), c(0.0), unit(0.0) {
    shift = (int)(((uintptr_t)p & 15) / sizeof(elem));
    at = (int)threadIdx.x * P - shift;
    n = (int)a.V;
    steps = NV ? NV : (n + shift + NT * P - 1) / (NT * P);
  }

  __device__ __forceinline__ int first(int j) const { return j * (NT * P) + at; }
  __device__ __forceinline__ bool whole(int i) const { return i >= 0 && i + P <= n; }

  // The piece at token i; places outside the row hold -inf, which nothing counts.
  __device__ __forceinline__ vec16 piece(int i) const {
    if (whole(i)) return *reinterpret_cast<const vec16 *>(row + i);
    vec16 v = nothing();
    if (i + P > 0 && i < n) {
      elem y[P];
      __builtin_memcpy(y, &v, 16);
#pragma unroll
      for (int e = 0; e < P; ++e)
        if (i + e >= 0 && i + e < n) y[e] = row[i + e];
      __builtin_memcpy(&v, y, 16);
    }
    return v;
  }
  // The row's first (k = 0) or last (k = 1) piece, where it is not whole: its step, for all
  // lanes of its wave, or -1.  mine: whether it is this thread's.
  __device__ __forceinline__ int part(int k, bool &mine) const {
    const int last = (n + shift) / P, at = k ? last : 0;
    mine = at % NT == (int)threadIdx.x;
    if (k ? (n + shift) % P == 0 || (last == 0 && shift) : shift == 0) return -1;
    return at % NT / 64 == (int)(threadIdx.x >> 6) ? at / NT : -1;
  }
  __device__ __forceinline__ static vec16 nothing() {
    constexpr uint32_t none = kShort ? 0xff80ff80u : 0xff800000u;
    return vec16{none, none, none, none};
  }
  // Held rows hold whole pieces only.
  __device__ __forceinline__ void fetch() {
    if constexpr (NV > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        r[j] = nothing();
        if (whole(first(j))) r[j] = *reinterpret_cast<const vec16 *>(row + j * (NT * P) + at);
      }
    }
  }
  // f(j, piece) over this thread's pieces, all lanes of a wave at once.  kAgain: from memory
  // even so, for what is too much code to have it once for every piece held.  Without kParts
  // a held row's first and last piece come as nothing where they are not whole.
  template <bool kAgain = false, bool kParts = true, typename F>
  __device__ __forceinline__ void each(F &&f) const {
    if constexpr (NV > 0 && !kAgain) {
#pragma unroll
      for (int j = 0; j < NV; ++j) f(j, r[j]);
#pragma unroll 1
      for (int k = 0; kParts && k < 2; ++k) {
        bool mine;
        const int j = part(k, mine);
        if (j >= 0) f(j, mine ? piece(first(j)) : nothing());
      }
    } else {
      constexpr int U = 4;  // loads on their way at a time
#pragma unroll 1
      for (int j = 0; j < steps; j += U) {
        vec16 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = piece(j + u < steps ? first(j + u) : n);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (j + u < steps) f(j + u, v[u]);
      }
    }
  }

  __device__ __forceinline__ unsigned long long weight(float z) const {
    const double x = ((double)z - (double)m) * c;
    const double w = __builtin_fma(exp2_256(x, l.tab), unit, 0x1p52);
    return __builtin_bit_cast(unsigned long long, w) & 0xfffffffffffffull;
  }

  // A token that has no counter: what it means for the row.
  __device__ __forceinline__ uint32_t strange(float z) const {
    if (z == kNegInf) return 0;
    if (!(z < __builtin_huge_valf())) return kRowBad;
    return z <= -kBinTop ? kRowLow : kRowOdd;
  }
  // Whether every token of a piece has a counter; then, with kCount, they are counted.
  template <bool kCount>
  __device__ __forceinline__ bool take(const vec16 &v) const {
    if constexpr (kShort) {
      u16x2 rel[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        rel[i] = __builtin_bit_cast(u16x2, v[i] & 0x7fff7fffu) - (unsigned short)kBinLo;
      const u16x2 x = __builtin_elementwise_max(__builtin_elementwise_max(rel[0], rel[1]),
                                                __builtin_elementwise_max(rel[2], rel[3]));
      if (!(x[0] < kSideBins && x[1] < kSideBins)) return false;
      if constexpr (kCount) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          atomicAdd(&l.h[(v[i] & 0xffffu) - kBinLo], 1u);
          atomicAdd(&l.h[(v[i] >> 16) - kBinLo], 1u);
        }
      }
    } else {
      uint32_t rel[4], x = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        rel[i] = ((v[i] >> 16) & 0x7fffu) - kBinLo;
        x = max(x, rel[i]);
      }
      if (x >= (uint32_t)kSideBins) return false;
      if constexpr (kCount) {
#pragma unroll
        for (int i = 0; i < 4; ++i) atomicAdd(&l.h[(v[i] >> 16) - kBinLo], 1u);
      }
    }
    return true;
  }
  template <bool kCount>
  __device__ __forceinline__ uint32_t take_one(uint32_t bits) const {
    const uint32_t u = bits >> 16, rel = (u & 0x7fffu) - kBinLo;
    if (rel < (uint32_t)kSideBins) {
      if constexpr (kCount) atomicAdd(&l.h[u - kBinLo], 1u);
      return 0;
    }
    if ((bits & 0x7fffffffu) == 0) {
      if constexpr (kCount) atomicAdd(&l.h[Lds::kNeg - 1], 1u);
      return 0;
    }
    return strange(__uint_as_float(bits));
  }
  // All of this thread's pieces; returns flags.  Pieces with tokens that have no counter
  // come again, token by token.
  template <bool kCount, typename F>
  __device__ __forceinline__ uint32_t take_all(F &&look) const {
    uint64_t again = 0;
    each<false, false>([&](int j, const vec16 &v) {
      if (!take<kCount>(v) && first(j) < n) again |= 1ull << j;
      look(v);
    });
    uint32_t flags = 0;
#pragma unroll 1
    while (again) {
      const int j = __builtin_ctzll(again);
      again &= again - 1;
      const vec16 v = piece(first(j));
      tokens(v, [&](int, uint32_t bits) { flags |= take_one<kCount>(bits); });
      look(v);
    }
    return flags;
  }

  // f(e, bits of the fp32 value) over the tokens of a piece
  template <typename F>
  __device__ __forceinline__ static void tokens(const vec16 &v, F &&f) {
    if constexpr (kShort) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f(2 * i, v[i] << 16);
        f(2 * i + 1, v[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) f(i, v[i]);
    }
  }
  // The largest token of a piece.
  __device__ __forceinline__ static float top(const vec16 &v) {
    float x = kNegInf;
    tokens(v, [&](int, uint32_t bits) { x = fmaxf(x, __uint_as_float(bits)); });
    return x;
  }

  // This thread's ranks are PT from the PT-th of its number on; f(i, rank) over those that
  // exist.
  template <typename F>
  __device__ __forceinline__ static void ranks(F &&f) {
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      const int rank = (int)threadIdx.x * PT + i;
      if (rank < kRanks) f(i, rank);
    }
  }
  // The first rank at which the running sum of x(rank) reaches the target
  // that want(whole sum) names (0: none) goes to l.rank, the sum above it to l.found[0].
  // mine: the sum of x(rank) over this thread's ranks.
  template <typename T, typename F, typename G>
  __device__ __forceinline__ void cross(T mine, F &&want, G &&x) {
    T total;
    T upto = row_scan<NT>(mine, total, l.wave);
    const T target = want(total);
    if (target && upto < target && upto + mine >= target) {
#pragma unroll 1
      for (int i = 0; i < PT; ++i) {
        const int rank = (int)threadIdx.x * PT + i;
        const T s = x(rank);
        if (upto + s >= target) {
          l.rank = rank;
          l.found[0] = upto;
          break;
        }
        upto += s;
      }
    }
    lds_barrier();
  }

  // The record that `target` falls into (l.found[0]: the sum before it), from their sums.
  __device__ __forceinline__ int find_record(unsigned long long target) {
    lds_barrier();
    constexpr int R = kRowEntries / NT;
    const int records = steps * (NT / 64);
    unsigned long long x[R], mine = 0, total;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int at = (int)threadIdx.x * R + i;
      x[i] = at < records ? l.sums[at] : 0;
      mine += x[i];
    }
    unsigned long long upto = row_scan<NT>(mine, total, l.wave);
    if (upto < target && upto + mine >= target) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (upto < target && upto + x[i] >= target) {
          l.rank = (int)threadIdx.x * R + i;
          l.found[0] = upto;
        }
        upto += x[i];
      }
    }
    lds_barrier();
    return l.rank;
  }

  // The index behind the nth token of value z.
  __device__ __forceinline__ int behind_tie(float z, uint32_t nth) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    auto hits = [&](const vec16 &v) -> uint32_t {
      if constexpr (kShort) {
        // halves that differ from z's: 1 each (both zeros are one value)
        const uint32_t mask = z == 0.0f ? 0x7fff7fffu : 0xffffffffu;
        const uint32_t u = (__float_as_uint(z) >> 16) & (mask & 0xffffu), both = u | u << 16;
        u16x2 off = {0, 0};
        const u16x2 one = {1, 1};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          off += __builtin_elementwise_min(__builtin_bit_cast(u16x2, (v[i] & mask) ^ both), one);
        return 8u - off[0] - off[1];
      } else {
        uint32_t k = 0;
        tokens(v, [&](int, uint32_t bits) { k += __uint_as_float(bits) == z; });
        return k;
      }
    };
    for (int i = threadIdx.x; i < steps * (NT / 64); i += NT) l.sums[i] = 0;
    lds_barrier();
    each([&](int j, const vec16 &v) {
      const uint32_t k = hits(v);
      if (k) atomicAdd(&l.sums[j * (NT / 64) + w], (unsigned long long)k);
    });
    const int rec = find_record((unsigned long long)nth);
    if (w == 0) {
      const int i0 = (rec * 64 + lane) * P - shift;
      const vec16 v = piece(i0);
      const uint32_t mine = hits(v), want = nth - (uint32_t)l.found[0];
      uint32_t upto = wave_scan(mine) - mine;
      if (upto < want && upto + mine >= want)
        tokens(v, [&](int e, uint32_t bits) {
          if (__uint_as_float(bits) == z && ++upto == want) l.tie = i0 + e + 1;
        });
    }
    lds_barrier();
    return l.tie;
  }

  // fp32: the value at which the running sum of the tokens of one rank, those above zt and at
  // it below index tie only, by falling value, reaches target, the sum above it and the
  // number of tokens at it.  kWeigh: sums of weights, else of ones.  false: they are too many.
  template <bool kWeigh>
  __device__ __forceinline__ bool refine(int rank, float zt, int tie, unsigned long long target,
                                         float &z, unsigned long long &above, uint32_t &n_at) {
    const uint32_t u = rank_bits(rank);
    if (threadIdx.x == 0) l.n_list = 0;
    lds_barrier();
    uint32_t *const list = l.list();
    each([&](int j, const vec16 &v) {
      uint32_t in = 0;
      tokens(v, [&](int e, uint32_t bits) {
        const bool hit = u ? bits >> 16 == u : (bits & 0x7fffffffu) == 0;
        in |= (uint32_t)hit << e;
      });
      if (!in) return;
      tokens(v, [&](int e, uint32_t bits) {
        const float x = __uint_as_float(bits);
        if (!(x > zt || (x == zt && first(j) + e < tie))) in &= ~(1u << e);
      });
      int to = atomicAdd(&l.n_list, (int)__popc(in));
      tokens(v, [&](int e, uint32_t bits) {
        if (in >> e & 1) {
          if (to < Lds::kListCap) list[to] = logit_key(__uint_as_float(bits));
          ++to;
        }
      });
    });
    lds_barrier();
    const int listed = l.n_list;
    if (listed > Lds::kListCap) return false;
    uint32_t prefix = 0;
    above = 0;
    // the upper halves are one: two steps over the lower
#pragma unroll 1
    for (int step = 0; step < 2; ++step) {
      for (int i = threadIdx.x; i < 256; i += NT) l.sums[i] = 0;
      lds_barrier();
      for (int i = threadIdx.x; i < listed; i += NT) {
        const uint32_t k = list[i];
        if (step == 0 || ((k >> 8) & 255u) == prefix)
          atomicAdd(&l.sums[step == 0 ? (k >> 8) & 255u : k & 255u],
                    kWeigh ? weight(key_logit(k)) : 1ull);
      }
      lds_barrier();
      const unsigned long long mine = threadIdx.x < 256 ? l.sums[255 - threadIdx.x] : 0;
      unsigned long long total;
      const unsigned long long upto = above + row_scan<NT>(mine, total, l.wave);
      if (upto < target && upto + mine >= target) {
        l.rank = 255 - (int)threadIdx.x;
        l.found[0] = upto;
        l.found[1] = mine;
      }
      lds_barrier();
      prefix = step == 0 ? (uint32_t)l.rank : prefix << 8 | (uint32_t)l.rank;
      above = l.found[0];
    }
    const uint32_t key = (listed ? list[0] & 0xffff0000u : 0u) | prefix;
    z = key_logit(key);
    n_at = (uint32_t)(l.found[1] / (kWeigh ? weight(z) : 1ull));
    lds_barrier();
    return true;
  }
};

// What the row keeps (tokens above zt, and those at it below index tie) and its largest
// logit.  bf16: the weights of the kept ranks are in l.mass() if they were needed (for top_p,
// or with `weights`).  Returns flags: 0, kRowBad or kRowOdd.
template <typename E, int NT, int NV>
__device__ __forceinline__ uint32_t held_cut(HeldRow<E, NT, NV> &r, const FilterAsk &q,
                                             bool weights, float &zt, int &tie) {
  using Row = HeldRow<E, NT, NV>;
  using Lds = RowLds<NT>;
  Lds &l = r.l;
  const FilterArgs &a = r.a;
  const bool by_k = q.k > 0 && q.k < a.V, by_p = q.p < 1.0f, by_least = q.least > 0.0f;
  const bool counts = by_k || by_p || (Row::kShort && (by_least || weights));
  if (counts) {
    for (int i = threadIdx.x; i < kSideBins; i += NT) {
      l.h[i] = 0;
      l.h[Lds::kNeg + i] = 0;
    }
  }
  if (threadIdx.x < kExpTab) l.tab.t[threadIdx.x] = kExp2Frac[threadIdx.x];
  if (threadIdx.x == 0) {
    l.h[Lds::kNeg - 1] = 0;
    l.flags = 0;
    l.best = 0;
  }
  lds_barrier();
  r.fetch();
  float m = kNegInf;
  uint32_t flags;
  auto look = [&](const vec16 &v) {
    if (!(Row::kShort && counts)) m = fmaxf(m, Row::top(v));
  };
  flags = counts ? r.template take_all<true>(look) : r.template take_all<false>(look);
  if (!(Row::kShort && counts)) {
    const uint32_t most = wave_most(m == kNegInf ? 0u : logit_key(m));
    if ((threadIdx.x & 63) == 63) atomicMax(&l.best, most);
  }
  if (flags) atomicOr(&l.flags, flags);
  lds_barrier();
  flags = l.flags;
  zt = kNegInf;
  tie = r.n;
  if (flags & kRowBad) return kRowBad;
  r.unit = ldexp(1.0, a.shift);
  r.c = exp2_scale(q.t);
  uint32_t n_in = 0;
  int rank_k = kRanks;                // top_k's cut: the first n_k tokens of this rank
  uint32_t n_k = 0, all_k = 0;
  if (counts) {
    if (flags & kRowOdd) return kRowOdd;
    uint32_t mine = 0;
    int best = kRanks;
    Row::ranks([&](int, int rank) {
      const uint32_t k = l.h[rank_word(rank)];
      mine += k;
      best = best == kRanks && k ? rank : best;
    });
    if constexpr (Row::kShort) {  // the largest logit: the first rank that has tokens
      const unsigned long long who = __ballot(best < kRanks);
      if (who && (threadIdx.x & 63) == (unsigned)__builtin_ctzll(who))
        atomicMax(&l.best, (uint32_t)(kRanks - best));
    }
    r.cross(mine, [&](uint32_t total) -> uint32_t {
      n_in = total;
      return by_k && (uint32_t)q.k <= total ? (uint32_t)q.k : 0u;
    }, [&](int rank) { return l.h[rank_word(rank)]; });
    if (n_in == 0) return flags & kRowLow ? kRowOdd : kRowBad;
    rank_k = by_k && (uint32_t)q.k <= n_in ? l.rank : kRanks;
    n_k = rank_k < kRanks ? (uint32_t)q.k - (uint32_t)l.found[0] : 0u;
    m = Row::kShort ? rank_value(kRanks - (int)l.best) : key_logit(l.best);
    if (by_k && (uint32_t)q.k > n_in && (flags & kRowLow) && !by_least) return kRowOdd;
  } else {
    if (l.best == 0) return kRowBad;
    m = key_logit(l.best);
    if (Row::kShort) return 0;  // nothing asked
  }
  r.m = m;
  if ((flags & kRowLow) && (m <= -kBinTop || r.weight(-kBinTop) != 0)) return kRowOdd;
  float least = kNegInf;
  if (by_least) {
    // the least float z with (z - m) / t >= log(min_p)
    const double d = (double)m + (double)q.t * log((double)q.least);
    least = (float)fmax(d, -3.5e38);
    if ((double)least < d) least = nextafterf(least, __builtin_huge_valf());
    least = fminf(least, m);
    if ((flags & kRowLow) && least <= -kBinTop) return kRowOdd;
    zt = least;
  }
  // what min_p leaves is a beginning of the same order as what top_k does: the shorter one
  if constexpr (Row::kShort) {
    if (rank_k < kRanks && rank_value(rank_k) >= least) {
      zt = rank_value(rank_k);
      all_k = l.h[rank_word(rank_k)];
    } else {
      rank_k = kRanks;
    }
    if (!by_p && n_k < all_k) tie = r.behind_tie(zt, n_k);
    if (!by_p && !weights) return 0;
    // weights by rank, of what is left
    unsigned long long mine = 0;
    unsigned long long *const mass = l.mass();
    Row::ranks([&](int, int rank) {
      uint32_t k = l.h[rank_word(rank)];
      if (rank >= rank_k) k = rank == rank_k ? n_k : 0u;
      unsigned long long w = 0;
      if (k) {
        const float z = rank_value(rank);
        if (z >= least) w = r.weight(z);
      }
      mass[rank_slot(rank)] = w;
      mine += k * w;
    });
    if (threadIdx.x < 2) mass[threadIdx.x * kSideSlots + kSideSlots - 1] = 0;
    lds_barrier();
    if (threadIdx.x == 0) mass[kSideSlots] = mass[0];  // -0.0
    if (!by_p) {
      lds_barrier();
      return 0;
    }
    unsigned long long target = 0;
    r.cross(mine, [&](unsigned long long total) {
      target = (unsigned long long)ceil(fmax((double)q.p, 0.0) * (double)total);
      return target = target < 1 ? 1 : target > total ? total : target;
    }, [&](int rank) {
      return mass[rank_slot(rank)] * (rank == rank_k ? n_k : l.h[rank_word(rank)]);
    });
    const int rank = l.rank;
    target -= l.found[0];  // of this rank
    const unsigned long long w = mass[rank_slot(rank)];
    const uint32_t k = (uint32_t)((target + w - 1) / w);
    zt = rank_value(rank);
    if (k < l.h[rank_word(rank)]) tie = r.behind_tie(zt, k);
    return 0;
  } else {
    if (rank_k < kRanks) {
      float z;
      unsigned long long above;
      if (!r.template refine<false>(rank_k, kNegInf, r.n, n_k, z, above, all_k)) return kRowOdd;
      if (z >= least) {
        zt = z;
        n_k -= (uint32_t)above;
        if (n_k < all_k) tie = r.behind_tie(z, n_k);
      }
    }
    if (!by_p) return 0;
    unsigned long long *const mass = l.mass();
    for (int i = threadIdx.x; i < kSlots; i += NT) mass[i] = 0;
    lds_barrier();
    r.each([&](int j, const vec16 &v) {
      const int i0 = r.first(j);
      Row::tokens(v, [&](int e, uint32_t bits) {
        const float z = __uint_as_float(bits);
        if ((z > zt || (z == zt && i0 + e < tie)) && z > -kBinTop) {
          const unsigned long long w = r.weight(z);
          if (w) atomicAdd(&mass[bits_slot(bits >> 16)], w);
        }
      });
    });
    lds_barrier();
    unsigned long long mine = 0;
    if (threadIdx.x == 0) mass[0] += mass[kSideSlots];  // one rank for both zeros
    lds_barrier();
    Row::ranks([&](int, int rank) { mine += mass[rank_slot(rank)]; });
    unsigned long long target = 0;
    r.cross(mine, [&](unsigned long long total) {
      target = (unsigned long long)ceil(fmax((double)q.p, 0.0) * (double)total);
      return target = target < 1 ? 1 : target > total ? total : target;
    }, [&](int rank) { return mass[rank_slot(rank)]; });
    const int rank = l.rank;
    target -= l.found[0];
    float z;
    unsigned long long above;
    uint32_t n_at;
    if (!r.template refine<true>(rank, zt, tie, target, z, above, n_at)) return kRowOdd;
    target -= above;
    const unsigned long long w = r.weight(z);
    const uint32_t k = (uint32_t)((target + w - 1) / w);
    if (k < n_at) tie = r.behind_tie(z, k);
    else if (z > zt) tie = r.n;
    zt = z;
    return 0;
  }
}

// -inf for the tokens of a piece below lim.
template <typename E>
__device__ __forceinline__ vec16 held_mask(const vec16 &v, float lim) {
  vec16 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (E::kPerVec == 8) {
      const float lo = __uint_as_float(v[i] << 16), hi = __uint_as_float(v[i] & 0xffff0000u);
      y[i] = (lo >= lim ? v[i] & 0xffffu : 0xff80u) | (hi >= lim ? v[i] & 0xffff0000u : 0xff800000u);
    } else {
      y[i] = __uint_as_float(v[i]) >= lim ? v[i] : 0xff800000u;
    }
  }
  return y;
}

template <typename E, int NT, int NV>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(NT / 256, NT / 256)))
void kr_filter(const typename E::elem *logits, typename E::elem *out, FilterArgs a) {
  using Row = HeldRow<E, NT, NV>;
  using elem = typename E::elem;
  constexpr int P = Row::P;
  __shared__ union {
    RowLds<NT> row;
    FilterLds<NT> any;
  } lds;
  const int64_t b = blockIdx.x / a.T;
  const FilterAsk q = filter_ask(a, b);
  if (!q.bad && a.n_rows && (int)(blockIdx.x % a.T) >= a.n_rows[b]) return;
  const int64_t off = (int64_t)blockIdx.x * a.V;
  if (q.bad) return fill_nan<E>(out + off, a.V);
  Row r(logits + off, a, lds.row);
  float zt;
  int tie;
  const uint32_t flags = held_cut(r, q, false, zt, tie);
  if (flags & kRowBad) return fill_nan<E>(out + off, a.V);
  if (flags & kRowOdd) {
    lds_barrier();
    return filter_any<E, false, NT>(logits, out, a, q, blockIdx.x, lds.any);
  }
  elem *const to = out + off;
  // all of a piece's tokens are on one side of tie, but for one piece of the row, which is
  // done token by token like the row's first and last ones where they are not whole
  const float above = nextafterf(zt, __builtin_huge_valf());
  int split = (tie + r.shift) / P;
  split = tie < r.n && (tie + r.shift) % P && split % NT == (int)threadIdx.x ? split / NT : -1;
  if (split >= 0 && !r.whole(r.first(split))) split = -1;
  r.template each<false, false>([&](int j, const vec16 &v) {
    const int i = r.first(j);
    if (r.whole(i) && j != split) {
      const vec16 y = held_mask<E>(v, i + P <= tie ? zt : above);
      *reinterpret_cast<vec16 *>(to + j * (NT * P) + r.at) = y;
    }
  });
#pragma unroll 1
  for (int k = 0; k < 3; ++k) {
    bool mine = true;
    const int j = k < 2 ? r.part(k, mine) : split;
    if (j < 0 || !mine) continue;
#pragma unroll 1
    for (int e = 0; e < P; ++e) {
      const int i = r.first(j) + e;
      if (i < 0 || i >= r.n) continue;
      const float z = E::at(r.row, i);
      const elem none = Row::kShort ? (elem)0xff80 : (elem)kNegInf;
      to[i] = z > zt || (z == zt && i < tie) ? r.row[i] : none;
    }
  }
}

template <typename E, int NT, int NV>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(NT / 256, NT / 256)))
void kr_sample(const typename E::elem *logits, FilterArgs a) {
  using Row = HeldRow<E, NT, NV>;
  __shared__ union {
    RowLds<NT> row;
    FilterLds<NT> any;
  } lds;
  const int64_t b = blockIdx.x / a.T;
  const int t = (int)(blockIdx.x % a.T);
  const FilterAsk q = filter_ask(a, b);
  if (!q.bad && a.n_rows && t >= a.n_rows[b]) return;
  RowLds<NT> &l = lds.row;
  Row r(logits + (int64_t)blockIdx.x * a.V, a, l);
  float zt = 0.0f;
  int tie = 0;
  const uint32_t flags = q.bad ? (uint32_t)kRowBad : held_cut(r, q, true, zt, tie);
  if (flags & kRowOdd) {
    lds_barrier();
    return sample_any<E, false, NT>(logits, a, q, b, t, lds.any);
  }
  if (flags & kRowBad) {
    for (int k = threadIdx.x; k < a.K; k += NT) put_draw(a, b, k, t, -1, 0.0f, 0.0f, 1.0f, 1);
    return;
  }
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  // the sums of the kept weights in every wave's piece; most pieces have none
  unsigned long long *const mass = l.mass();
  if constexpr (Row::kShort) {  // ranks below the cut have none
    Row::ranks([&](int, int rank) {
      if (rank_value(rank) < zt) mass[rank_slot(rank)] = 0;
    });
    if (threadIdx.x == 0 && 0.0f < zt) mass[kSideSlots] = 0;
    lds_barrier();
  }
  auto weigh = [&](int i, uint32_t bits) -> unsigned long long {
    const float z = __uint_as_float(bits);
    if constexpr (Row::kShort) {
      return z == zt && i >= tie ? 0ull : mass[bits_slot(bits >> 16)];
    } else {
      if (!(z > zt || (z == zt && i < tie)) || !(z > -kBinTop)) return 0;
      return r.weight(z);
    }
  };
  auto sum_of = [&](int i0, const vec16 &v) {
    unsigned long long s = 0;
    Row::tokens(v, [&](int e, uint32_t bits) { s += weigh(i0 + e, bits); });
    return s;
  };
  const float lim = fmaxf(zt, -kBinTop);
  for (int i = threadIdx.x; i < r.steps * (NT / 64); i += NT) l.sums[i] = 0;
  lds_barrier();
  r.template each<true>([&](int j, const vec16 &v) {
    if (!__any(Row::top(v) >= lim)) return;
    const unsigned long long s = wave_scan(sum_of(r.first(j), v));
    if (lane == 63 && s) atomicAdd(&l.sums[j * (NT / 64) + w], s);
  });
  lds_barrier();
  // what is before each record
  constexpr int R = kRowEntries / NT;
  const int n = r.steps * (NT / 64);
  unsigned long long x[R], mine = 0, total;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    x[i] = (int)threadIdx.x * R + i < n ? l.sums[threadIdx.x * R + i] : 0;
    mine += x[i];
  }
  unsigned long long upto = row_scan<NT>(mine, total, l.wave);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if ((int)threadIdx.x * R + i < n) l.sums[threadIdx.x * R + i] = upto;
    upto += x[i];
  }
  lds_barrier();
  // a wave per draw: the record that it falls into, then the token
#pragma unroll 1
  for (int k = w; k < a.K; k += NT / 64) {
    const double u = draw_uniform(a, b, k, t);
    if (!(u >= 0.0 && u < 1.0)) {
      if (lane == 0) put_draw(a, b, k, t, -1, 0.0f, 0.0f, 1.0f, 1);
      continue;
    }
    const unsigned long long target = draw_target(u, total);
    int lo = 0, hi = n - 1;  // the last record with less than target before it
#pragma unroll 1
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (l.sums[mid] < target) lo = mid;
      else hi = mid - 1;
    }
    const int i0 = (lo * 64 + lane) * Row::P - r.shift;
    const vec16 v = r.piece(i0);
    const unsigned long long s = sum_of(i0, v);
    unsigned long long at = wave_scan(s) + l.sums[lo] - s;
    if (at < target && at + s >= target) {
      int token = 0;
      uint32_t z = 0;
      Row::tokens(v, [&](int e, uint32_t bits) {
        const unsigned long long x_ = weigh(i0 + e, bits);
        if (at < target && at + x_ >= target) {
          token = i0 + e;
          z = bits;
        }
        at += x_;
      });
      put_draw(a, b, k, t, token, __uint_as_float(z), r.m, q.t, total);
    }
  }
}

}  // namespace svd
