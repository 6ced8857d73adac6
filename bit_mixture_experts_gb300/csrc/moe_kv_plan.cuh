// How an attention call's work is dealt to its CTAs, worked out on the device
// (the lengths are never read by the host).
//
// Query rows are packed per KV head: row r of a 128-row tile is token r / G,
// query head r % G of the head's group of G (tpt = 128 / G tokens per tile), so
// every key is read once for all query heads that share it.  An item is one
// (sequence, KV head, pair of tiles); its units are the 128-key tiles that the
// pair's last token sees.  All units of a call in the order sequence, head,
// pair, key tile are one line, of which CTA c of n takes [W c / n, W (c+1) / n):
// even shares whatever the lengths, an item being cut where a share ends
// (its parts are merged afterwards).  A pair that sees no key counts one unit,
// which writes its zeros.
#pragma once
#include "moe_kv_dev.cuh"

namespace moe {
namespace kv {

constexpr int TILE = 128;  // query rows of a tile, keys of a tile

// Sum of floor((a i + b) / m) for i = 0 .. n-1 (the Euclid-like recursion on the slope a / m).
__device__ __forceinline__ long long floor_sum(unsigned long long n, unsigned m, unsigned a, unsigned long long b) {
  unsigned long long ans = 0;
  while (n > 0) {
    ans += n * (n - 1) / 2 * (a / m);
    a %= m;
    ans += n * (b / m);
    b %= m;
    const unsigned long long y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const unsigned t = m;
    m = a;
    a = t;
  }
  return static_cast<long long>(ans);
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
    return z + floor_sum(mp - z, TILE, tp, first);
  }

  __device__ __forceinline__ long long units() const { return M == 0 ? 0 : before(M - 1) + tiles(M - 1); }

  // The pair that unit r (of one head) belongs to.
  __device__ __forceinline__ int find(long long r) const {
    int lo = 0, hi = M - 1;  // before(lo) <= r
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before(mid) <= r)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }
};

// A run of key tiles [t0, t1) of one item.
struct Seg {
  Seq s;
  int b, h, i0, ntok;  // sequence, KV head, first token of the pair, tokens in it
  int t0, t1, nt;      // nt: the item's tiles
};

// Walks the segments of units [u, end), starting in sequence b whose first unit is b_lo.
struct Walk {
  const Args& a;
  int tp, b;
  long long u, end, b_lo, b_hi, per_head;
  Seq s;

  __device__ __forceinline__ Walk(const Args& a_, int tp_, long long u_, long long end_, int b_, long long b_lo_)
      : a(a_), tp(tp_), b(b_ - 1), u(u_), end(end_), b_lo(0), b_hi(b_lo_), per_head(0) {}

  __device__ __forceinline__ bool next(Seg& g) {
    if (u >= end) return false;
    while (u >= b_hi) {
      s = load_seq(a, ++b);
      per_head = Pairs(s, tp).units();
      b_lo = b_hi;
      b_hi += per_head * a.heads;
    }
    const Pairs p(s, tp);
    const long long v = u - b_lo, r = v % per_head;
    const int mp = p.find(r);
    g.s = s;
    g.b = b;
    g.h = static_cast<int>(v / per_head);
    g.i0 = mp * tp;
    g.ntok = min(tp, s.n - g.i0);
    g.nt = p.tiles(mp);
    g.t0 = static_cast<int>(r - p.before(mp));
    g.t1 = static_cast<int>(min(static_cast<long long>(g.nt), g.t0 + (end - u)));
    u += g.t1 - g.t0;
    return true;
  }
};

// Where a call's line of units is cut.
struct Share {
  long long total;  // W
  int ctas;         // n: CTAs with work
  __device__ __forceinline__ long long lo(int c) const { return total * c / ctas; }
};

struct Start {
  long long b_lo;
  int b;
};

// Block-wide: the total of all sequences' units, then (for the unit that `pick` returns for that
// total; negative: none) the sequence that holds it.  `scratch`: 33 long longs and a Start in shared
// memory, free again on return.  NT threads.
template <int NT, typename Pick>
__device__ __forceinline__ long long locate(const Args& a, int tp, long long* scratch, Start* found, Pick pick) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = ceil_div(a.B, NT);
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += Pairs(load_seq(a, b), tp).units() * a.heads;
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  long long off = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const long long x = scratch[w];
    if (w < warp) off += x;
    total += x;
  }
  const long long want = pick(total);
  long long lo = off + incl - mine;
  if (want >= lo && want < lo + mine) {
    int b = b0;
    for (;; ++b) {
      const long long n = Pairs(load_seq(a, b), tp).units() * a.heads;
      if (want < lo + n) break;
      lo += n;
    }
    found->b = b;
    found->b_lo = lo;
  }
  __syncthreads();
  return total;
}

}  // namespace kv
}  // namespace moe
