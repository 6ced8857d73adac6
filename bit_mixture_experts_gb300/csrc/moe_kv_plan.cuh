// How an attention call's work is dealt to its CTAs, worked out on the device
// (the lengths are never read by the host).
//
// Query rows are packed per KV head: row r of a 128-row tile is token r / G,
// query head r % G of the head's group of G (tpt = 128 / G tokens per tile), so
// every key is read once for all query heads that share it.  An item is one
// (sequence, KV head, pair of tiles); its units are the 128-key tiles that the
// pair's last token sees, after START more for what an item costs whatever its
// length.  All units of a call in the order sequence, head, pair, key tile are
// one line, of which CTA c of n takes [W c / n, W (c+1) / n):
// even shares whatever the lengths, an item being cut where a share ends
// (its parts are merged afterwards).  Where all items are short it goes whole to
// the CTA whose share it starts in: nothing to merge.  A pair that sees no key counts one unit,
// which writes its zeros.  Where a pair has rows in its first tile alone (the
// last of a sequence, and every decode step), the second tile's half of the CTA
// takes every other key tile instead.
#pragma once
#include "moe_kv_dev.cuh"

namespace moe {
namespace kv {

constexpr int TILE = 128;  // query rows of a tile, keys of a tile
constexpr int START = 2;   // an item's start and end (its queries, its output), in key tiles

// Sum of floor((a i + b) / TILE) for i = 0 .. n-1, n <= 2^20, a <= 2 TILE (the Euclid-like recursion
// on the slope).  After the first step every term but the sum itself fits 32 bits.
__device__ __forceinline__ long long floor_sum(int n_, int a_, long long b_) {
  static_assert(TILE == 128, "shift");
  unsigned long long n = static_cast<unsigned>(n_);
  long long ans = static_cast<long long>(n * (n - 1) / 2) * (a_ >> 7) + static_cast<long long>(n) * (b_ >> 7);
  if (n_ == 0) return 0;
  uint32_t m = TILE, a = a_ & (TILE - 1), b = static_cast<uint32_t>(b_) & (TILE - 1);
  for (;;) {
    const uint32_t y = a * static_cast<uint32_t>(n) + b;
    if (y < m) return ans;
    n = y / m;
    b = y % m;
    const uint32_t t = m;
    m = a;
    a = t;
    ans += static_cast<long long>(n * (n - 1) / 2) * (a / m) + static_cast<long long>(n) * (b / m);
    a %= m;
    b %= m;
  }
}

// A sequence's pairs: M of them of tp tokens (the last may have fewer).
struct Pairs {
  int n, base, tp, M;  // new tokens; keys before them (negative: more new tokens than positions)

  __device__ __forceinline__ Pairs(const Seq& s, int tp_) : n(s.n), base(s.len - s.n), tp(tp_), M(ceil_div(s.n, tp_)) {}

  // Key tiles of pair mp.
  __device__ __forceinline__ int tiles(int mp) const {
    const int last = static_cast<int>(min(static_cast<long long>(n), (mp + 1ll) * tp));
    return max(1, ceil_div(max(0, base + last), TILE));
  }

  // Units of the pairs before mp (mp < M, so all of them are full).
  __device__ __forceinline__ long long before(int mp) const {
    if (mp == 0) return 0;
    int z = 0;  // pairs that see nothing
    if (base < 0) z = min(mp, -base / tp);
    const long long first = base + (z + 1ll) * tp + TILE - 1;
    return static_cast<long long>(mp) * START + z + floor_sum(mp - z, tp, first);
  }

  __device__ __forceinline__ long long units() const {
    return M == 0 ? 0 : before(M - 1) + START + tiles(M - 1);
  }

  // The pair that unit r (of one head) belongs to, and the units before it, by a whole warp: each lane tries
  // one of 32 places in the range left (one place at a time, a 512-token prompt's plan took 3 us longer).
  __device__ __forceinline__ int find(long long r, long long* units_before) const {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = M - 1;  // before(lo) <= r
    long long at = 0;
    while (lo < hi) {
      const int step = (hi - lo + 31) >> 5, mid = lo + (lane + 1) * step;
      long long x = 0;
      if (mid <= hi) x = before(mid);
      const int n = __popc(__ballot_sync(0xffffffffu, mid <= hi && x <= r));
      if (n > 0) at = __shfl_sync(0xffffffffu, x, n - 1);
      lo += n * step;
      hi = min(hi, lo + step - 1);
    }
    *units_before = at;
    return lo;
  }
};

// A run of key tiles [t0, t1) of one item: sequence b (first row row0, len tokens), KV head h, tokens
// i0 .. i0 + ntok - 1 of its new ones, the first of which sits at position base; nt: the item's tiles.
struct Seg {
  int row0, len, b, h, i0, ntok, base, t0, t1, nt;
};

// Quotient of two counts that nearly always fit 32 bits (a 64-bit division costs several times as much).
__device__ __forceinline__ long long divide(long long x, long long y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// Walks the segments of units [u, end), starting in sequence b whose first unit is b_lo; by a whole warp.
struct Walk {
  const Args* a;
  int tp, b;
  long long u, end, b_lo, b_hi, per_head;
  long long item_end;  // the last segment's item's last unit, plus one
  Seq s;
  bool whole;

  __device__ __forceinline__ Walk(const Args& a_, int tp_, long long u_, long long end_, int b_, long long b_lo_,
                                  bool whole_)
      : a(&a_), tp(tp_), b(b_ - 1), u(u_), end(end_), b_lo(0), b_hi(b_lo_), per_head(0), item_end(0), whole(whole_) {}

  // `whole`: items that start in [u, end), each in full; otherwise the key tiles among units [u, end).
  __device__ __forceinline__ bool next(Seg& g) {
    for (;;) {
      if (u >= end) return false;
      while (u >= b_hi) {
        s = load_seq(*a, ++b);
        per_head = Pairs(s, tp).units();
        b_lo = b_hi;
        b_hi += per_head * a->heads;
      }
      const Pairs p(s, tp);
      const long long v = u - b_lo, h = divide(v, per_head), r = v - h * per_head;
      long long first;
      const int mp = p.find(r, &first), off = static_cast<int>(r - first);
      g.row0 = s.row0;
      g.len = s.len;
      g.b = b;
      g.h = static_cast<int>(h);
      g.i0 = mp * tp;
      g.ntok = min(tp, s.n - g.i0);
      g.base = s.len - s.n + g.i0;
      g.nt = p.tiles(mp);
      item_end = u - off + START + g.nt;
      const long long stop = whole ? item_end : min(item_end, end);
      g.t0 = max(0, off - START);
      g.t1 = static_cast<int>(off - START + (stop - u));
      u = stop;
      if (whole ? off == 0 : g.t1 > g.t0) return true;
    }
  }
};

// How a call's line of units is dealt out: as evenly as can be.
struct Share {
  long long total, each;
  int ctas, more;  // CTAs with work; how many of them take one unit more than `each`
  bool whole;

  // `merge`: what writing and merging parts costs, in key tiles.  Cut, the call takes about an even share
  // and that; whole, the longest item where every item has a CTA, and up to that more than a share else.
  __device__ __forceinline__ void set(long long units, int longest, int items, int grid, int merge) {
    total = units;
    ctas = static_cast<int>(min(static_cast<long long>(grid), units));
    each = ctas ? divide(units, ctas) : 0;
    more = static_cast<int>(units - each * ctas);
    whole = longest <= merge + (items <= grid ? each : each / 16);
  }
  __device__ __forceinline__ long long lo(int c) const { return each * c + min(c, more); }
  // The CTA whose share holds unit u.
  __device__ __forceinline__ int of(long long u) const {
    const long long edge = (each + 1) * more;
    return static_cast<int>(u < edge ? divide(u, each + 1) : more + divide(u - edge, each));
  }
};

// A unit's sequence and that sequence's first unit.
struct Start {
  long long b_lo;
  int b;
};

// Sets `share` and finds the sequence that holds unit share.lo(cut), if there is such a share.  All
// threads of the block, or up to 32 sequences any whole warps of it; `scratch`: 66 long longs of shared
// memory, free again on return.  Up to 32 sequences every warp works it out for itself, a sequence per lane;
// more are dealt to the block's threads.
template <int NT>
__device__ __forceinline__ Start locate(const Args& a, int tp, int grid, int merge, int cut, long long* scratch,
                                        Share& share) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool small = a.B <= 32;
  const int per = small ? 1 : ceil_div(a.B, NT);
  const int b0 = min((small ? lane : tid) * per, a.B), b1 = min(b0 + per, a.B);
  long long mine = 0;
  int longest = 0, items = 0;
  for (int b = b0; b < b1; ++b) {
    const Pairs p(load_seq(a, b), tp);
    mine += p.units() * a.heads;
    if (p.M > 0) longest = max(longest, p.tiles(p.M - 1));
    items += p.M * a.heads;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  items = __reduce_add_sync(0xffffffffu, items);
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  Start found = {0, 0};
  if (small) {
    share.set(__shfl_sync(0xffffffffu, incl, 31), longest, items, grid, merge);
    const long long want = share.lo(cut);
    const uint32_t past = __ballot_sync(0xffffffffu, incl > want);  // sequences that end after it
    if (cut < share.ctas) {
      found.b = __ffs(past) - 1;
      found.b_lo = __shfl_sync(0xffffffffu, incl - mine, found.b);
    }
    return found;
  }
  int* more = reinterpret_cast<int*>(scratch + 32);
  if (lane == 31) {
    scratch[warp] = incl;
    more[warp] = longest;
    more[32 + warp] = items;
  }
  __syncthreads();
  long long off = 0, total = 0;
  items = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const long long x = scratch[w];
    if (w < warp) off += x;
    total += x;
    longest = max(longest, more[w]);
    items += more[32 + w];
  }
  share.set(total, longest, items, grid, merge);
  const long long want = share.lo(cut);
  long long lo = off + incl - mine;
  Start* shared = reinterpret_cast<Start*>(scratch + 64);
  if (cut < share.ctas && want >= lo && want < lo + mine) {
    int b = b0;
    for (;; ++b) {
      const long long n = Pairs(load_seq(a, b), tp).units() * a.heads;
      if (want < lo + n) break;
      lo += n;
    }
    shared->b = b;
    shared->b_lo = lo;
  }
  __syncthreads();
  if (cut < share.ctas) found = *shared;
  return found;
}

}  // namespace kv
}  // namespace moe
