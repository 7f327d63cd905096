// kr_pages.hpp -- block tables and slot maps of the paged cache, from the lengths that
// the requests shall have.
//
// Free pages are a ring: state holds its first place and its count.  A call takes the
// pages that growing sequences need from the ring's head, in sequence order, and puts the
// pages that shrinking ones give back behind its end.  The two ranges never meet (free and
// returned pages together are at most as many as the ring has places), so that pages move
// in one pass without an order among them, and what a call does is a function of its
// inputs alone.
//
//   kr_pages_plan  one workgroup: the pages every sequence needs, two running sums over
//                  the batch (grants and returns), who fits, and the new lengths;
//   kr_pages_move  a thread per table entry: copies it, grants it or returns it.
//   kr_slots       packed tokens: a running sum over the batch in every workgroup, then a
//                  search for each token's sequence.
// One workgroup plans, since every place follows from sums over the whole batch and 1024
// sequences are one round of it: 3.8 us for 8 sequences, 6.0 for 1024.  The move is bound by
// its bytes only where the tables are wide: 16.8 MB in 6.7 us for 1024 rows of 2048 entries
// (2.5 TB/s, out of the last-level cache in part), 2.0 us for 8 rows of 64.  kr_slots: 3.7 us
// for a few tokens, 4.9 for 41000 of 32 sequences.
#pragma once

#include "kr_cache.hpp"
#include "svd_device.hpp"

namespace svd {

constexpr int kPagesBlock = 1024;
constexpr int kPagesMoveBlock = 256;

struct PagePlan {      // one sequence
  int32_t was, now;    // entries of its row in use before and after; -1: out of range
  int32_t off;         // places of the ring from its head (grants) or its end (returns) on
  int32_t pad;
};
struct PageHead {
  int32_t head, count, ok, pad;  // the ring as it was; ok: the call moves pages at all
};

struct PagesArgs {
  const int32_t *length, *shared, *held, *table, *state;
  int32_t *held_out, *table_out, *state_out, *room, *ring;
  int64_t B, n_pages;
  int max_pages, page_shift;
  PageHead *head;
  PagePlan *plan;
};

// Inclusive sums of x over the workgroup's threads, and the total: two scans in one.
template <int NT>
__device__ __forceinline__ void block_scan2(int64_t &x, int64_t &y, int64_t &tx, int64_t &ty,
                                            int64_t (*lds)[2] /* NT / 64 + 1 */) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t px = __shfl_up(x, off, 64), py = __shfl_up(y, off, 64);
    if (lane >= off) {
      x += px;
      y += py;
    }
  }
  if (lane == 63) {
    lds[w][0] = x;
    lds[w][1] = y;
  }
  __syncthreads();
  tx = ty = 0;
  int64_t bx = 0, by = 0;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) {
    if (i == w) {
      bx = tx;
      by = ty;
    }
    tx += lds[i][0];
    ty += lds[i][1];
  }
  x += bx;
  y += by;
  __syncthreads();
}

__global__ __launch_bounds__(kPagesBlock) void kr_pages_plan(PagesArgs a) {
  __shared__ int64_t lds[kPagesBlock / 64][2];
  __shared__ unsigned long long taken;  // the most that a sequence's grant reaches up to
  const int64_t head = a.state[0], count = a.state[1];
  const bool ring_ok = head >= 0 && head < a.n_pages && count >= 0 && count <= a.n_pages;
  if (threadIdx.x == 0) taken = 0;
  __syncthreads();
  int64_t grows = 0, gives = 0;  // of the sequences before this chunk
  for (int64_t b0 = 0; b0 < a.B; b0 += kPagesBlock) {
    const int64_t b = b0 + threadIdx.x;
    int64_t was = 0, now = -1, grow = 0, give = 0;
    if (b < a.B) {
      const int64_t n = a.length[b], sh = a.shared ? a.shared[b] : 0;
      was = a.held[b];
      const int64_t need = max(sh, (n + (1ll << a.page_shift) - 1) >> a.page_shift);
      if (n >= 0 && need <= a.max_pages && was >= 0 && was <= a.max_pages && sh >= 0 && sh <= was) {
        now = need;
        grow = max(need - was, (int64_t)0);
        give = max(was - need, (int64_t)0);
      }
    }
    int64_t up = grow, gone = give, all_up, all_gone;
    block_scan2<kPagesBlock>(up, gone, all_up, all_gone, lds);
    up += grows;
    gone += gives;
    if (b < a.B) {
      if (grow > 0 && up > count) now = was;  // it does not fit: nothing of it changes
      else if (grow > 0) atomicMax(&taken, (unsigned long long)up);
      PagePlan p;
      p.was = (int32_t)was;
      p.now = (int32_t)now;
      p.off = (int32_t)(grow > 0 ? up - grow : gone - give);
      p.pad = 0;
      a.plan[b] = p;
    }
    grows += all_up;
    gives += all_gone;
  }
  __syncthreads();
  const bool ok = ring_ok && count + gives <= a.n_pages;
  if (threadIdx.x == 0) {
    a.head->head = (int32_t)head;
    a.head->count = (int32_t)count;
    a.head->ok = ok;
    const int64_t g = (int64_t)taken;
    a.state_out[0] = (int32_t)(ok ? (head + g) % a.n_pages : head);
    a.state_out[1] = (int32_t)(ok ? count - g + gives : count);
  }
  for (int64_t b = threadIdx.x; b < a.B; b += kPagesBlock) {
    const PagePlan p = a.plan[b];  // this thread's own
    const bool move = ok && p.now >= 0;
    a.held_out[b] = move ? p.now : p.was;
    a.room[b] = move ? p.now << a.page_shift : -1;
  }
}

__global__ __launch_bounds__(kPagesMoveBlock) void kr_pages_move(PagesArgs a) {
  const int64_t i = (int64_t)blockIdx.x * kPagesMoveBlock + threadIdx.x;
  if (i >= a.B * a.max_pages) return;
  const int64_t b = i / a.max_pages;
  const int j = (int)(i % a.max_pages);
  const PageHead h = *a.head;
  const PagePlan p = a.plan[b];
  const bool move = h.ok && p.now >= 0;
  const bool in_place = a.table == a.table_out;
  if (move && j >= p.was && j < p.now) {
    a.table_out[i] = a.ring[((int64_t)h.head + p.off + (j - p.was)) % a.n_pages];
  } else if (move && j >= p.now && j < p.was) {
    a.ring[((int64_t)h.head + h.count + p.off + (j - p.now)) % a.n_pages] = a.table[i];
    a.table_out[i] = -1;
  } else if (!in_place) {
    a.table_out[i] = a.table[i];
  }
}

// ---------------------------------------------------------------------------
// Packed tokens.

constexpr int kSlotsBlock = 1024;   // tokens of a workgroup, and sequences of a chunk

struct SlotsArgs {
  const int32_t *ctx_len, *n_new, *table;
  int64_t B, N, n_pages;
  int max_pages, page_shift;
  int32_t *row_off, *seq, *pos;
  int64_t *slot;
};

__global__ __launch_bounds__(kSlotsBlock) void kr_slots(SlotsArgs a) {
  __shared__ int64_t lds[kSlotsBlock / 64][2];
  __shared__ int64_t ends[kSlotsBlock];  // behind the last token of each sequence of a chunk
  const int64_t i = (int64_t)blockIdx.x * kSlotsBlock + threadIdx.x;
  const int64_t i_hi = min((int64_t)(blockIdx.x + 1) * kSlotsBlock, a.N);
  const bool all = blockIdx.x == 0;  // writes the sequences' offsets
  int32_t seq = -1, pos = -1;
  int64_t slot = -1;
  int64_t before = 0;
  for (int64_t b0 = 0; b0 < a.B && (all || before < i_hi); b0 += kSlotsBlock) {
    const int64_t b = b0 + threadIdx.x;
    int64_t n = 0;
    if (b < a.B) {
      const int64_t c = a.ctx_len[b], m = a.n_new[b];
      n = c >= 0 && m >= 0 && c + m < (1ll << 31) ? m : 0;  // lengths out of range: no tokens
    }
    int64_t up = n, none = 0, total, none_;
    block_scan2<kSlotsBlock>(up, none, total, none_, lds);
    up += before;
    ends[threadIdx.x] = up;
    if (all && b < a.B) a.row_off[b] = (int32_t)min(up - n, (int64_t)0x7fffffff);
    __syncthreads();
    if (i < i_hi && i >= before && i < before + total) {
      int lo = 0, hi = kSlotsBlock - 1;  // the first sequence that ends behind token i
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (ends[mid] > i) hi = mid;
        else lo = mid + 1;
      }
      const int64_t s = b0 + lo, first = lo ? ends[lo - 1] : before;
      const int64_t p = a.ctx_len[s] + (i - first);
      seq = (int32_t)s;
      pos = (int32_t)p;
      const int64_t col = p >> a.page_shift;
      if (col < a.max_pages) {
        const int64_t pg = a.table[s * a.max_pages + col];
        if (pg >= 0 && pg < a.n_pages)
          slot = (pg << a.page_shift) + (p & ((1 << a.page_shift) - 1));
      }
    }
    before += total;
    __syncthreads();
  }
  if (all && threadIdx.x == 0) a.row_off[a.B] = (int32_t)min(before, (int64_t)0x7fffffff);
  if (i < i_hi) {
    a.seq[i] = seq;
    a.pos[i] = pos;
    a.slot[i] = slot;
  }
}

}  // namespace svd
