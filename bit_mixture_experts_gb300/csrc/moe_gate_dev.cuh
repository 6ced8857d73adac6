// The choice of tokens' experts by a warp, for routers with sigmoid or
// softmax scores, a bias that takes part in the choice alone, groups of experts
// of which the best stay, and weights that are renormalised and scaled:
//
//   s_e = sigmoid(l_e)  or  exp(l_e - m) / sum_i exp(l_i - m)
//   v_e = s_e + b_e;  chosen: the k largest v_e of the groups that stay, in
//   descending order, equal ones by index
//   w_j = scale s_j / (sum of the chosen s, or 1), by ratios of the s
//
// The choice has to be what exact scores give, and FP32 scores can be off by
// more than two experts differ.  So values are compared as integers m, v in
// units of 2^-23 (2^-21 above 256 experts) of the range that v can have, and
// where two neighbours of the sorted choice, the last one chosen and any other
// expert, or the last group that stays and the first that does not are not
// further apart than their errors, the token is done again with scores of twice
// the length, off by less than 2^-40 (256 experts, 8 chosen: one token in 200 to
// 1000; 1024 experts, softmax: one in 25 to 50 with 16 chosen, one in 10 with 32).  Experts
// whose logit and bias are the same bits tie in any precision and need no second look.  Without a bias
// the scores are monotone in the logits, which are then compared themselves: m
// is the upper 23 (21) bits of the logit, and the second look is at all of it.
//
// m and the expert's index make one key (equal m: lower index first), 31 bits,
// so that a round of the choice is one redux.sync over the lanes' largest keys
// below the last one chosen.  A warp takes up to four tokens at a time: what
// concerns a token's k choices or its groups needs fewer lanes than a warp has,
// and is done for all of them at once.
//
// What bounds it: 262144 tokens of 256 experts (sigmoid, bias, four of eight
// groups, eight chosen) take 129 us where the bytes of their logits take 42.  The
// ALU pipe, which does minima, maxima and compares at half rate, is 65 % busy, the
// issue slots are 58 %.  A single token takes 3.0 us, a chain of latencies.
#pragma once
#include <float.h>

#include "moe_common.cuh"
#include "moe_route_dev.cuh"

namespace moe {
namespace gate_dev {

using route_dev::float_key;
using route_dev::FULL;
using route_dev::key_float;

struct Gate {
  const float* bias;  // [E] or null
  int E, k, groups, per_group, top_groups;
  // lane / lanes is the lane's group, of whose per_group experts it has `width` consecutive ones
  int lanes_log, width;
  bool softmax, top2, renorm;
  bool by_logit;  // the logits themselves are compared
  float scale;
};

// Experts a lane holds, at most (groups of any number up to 32, E <= 1024).
constexpr int MAX_WIDTH = 64;

enum Mode { BY_LOGIT, SIGMOID, SOFTMAX };  // what is compared; SOFTMAX also where weights need the sum over all

__device__ __forceinline__ float available(float l) {  // NaN counts as -inf, +inf as the largest number
  return l > -INFINITY ? fminf(l, FLT_MAX) : -INFINITY;
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A lane's share of the experts.
struct Lane {
  int group, first, n;
  __device__ __forceinline__ Lane(const Gate& g, int lane) {
    const int sub = lane & ((1 << g.lanes_log) - 1);
    group = lane >> g.lanes_log;
    first = group * g.per_group + sub * g.width;
    n = group < g.groups ? min(max(g.per_group - sub * g.width, 0), g.width) : 0;
  }
};

// ---- The second look: scores as pairs of floats (high part, rest), about 45 bits, on the FP32 pipe, by the known
// error-free sums (fast two-sum: Dekker; two-sum: Knuth) and the product whose rest an FMA gives.  (In
// 64-bit floats, of which an SM does one a clock, a token's 256 exponentials took 9000 cycles, all of its
// second look 29000.)
struct Pair {
  float h, l;
};

__device__ __forceinline__ Pair fast_sum(float a, float b) {  // |a| >= |b| or a = 0: exact
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}

__device__ __forceinline__ Pair sum(float a, float b) {  // exact
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}

__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = sum(a.h, b.h);
  return fast_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}

__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  const float p = __fmul_rn(a.h, b.h);
  return fast_sum(p, __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, __fmaf_rn(a.h, b.h, -p))));
}

// e^x for x <= 0, 0 below about -87: x = n ln 2 + r with ln 2 in three parts (the first has ten bits, so that
// its product with n is exact), e^r by its Taylor series, the terms from r^7 on as floats.
__device__ __forceinline__ Pair exp_pair(Pair x) {
  if (x.h < -150.f) x = {-150.f, 0.f};
  const float n = rintf(x.h * 1.44269504f);
  Pair r = sum(__fmaf_rn(n, -0.693359375f, x.h), x.l);
  const float p = __fmul_rn(n, 0x1.bd01060000000p-13f);
  r = add(r, {p, __fmaf_rn(n, -0x1.cf79ac0000000p-40f, __fmaf_rn(n, 0x1.bd01060000000p-13f, -p))});
  float t = 1.0f / 479001600.0f;
  t = fmaf(t, r.h, 1.0f / 39916800.0f);
  t = fmaf(t, r.h, 1.0f / 3628800.0f);
  t = fmaf(t, r.h, 1.0f / 362880.0f);
  t = fmaf(t, r.h, 1.0f / 40320.0f);
  t = fmaf(t, r.h, 1.0f / 5040.0f);
  Pair q = add({0x1.6c16c20000000p-10f, -0x1.27d27e0000000p-35f}, mul(r, {t, 0.f}));
  q = add({0x1.1111120000000p-7f, -0x1.ddddde0000000p-32f}, mul(r, q));
  q = add({0x1.5555560000000p-5f, -0x1.5555560000000p-30f}, mul(r, q));
  q = add({0x1.5555560000000p-3f, -0x1.5555560000000p-28f}, mul(r, q));
  q = add({0.5f, 0.f}, mul(r, q));
  q = add({1.0f, 0.f}, mul(r, q));
  q = add({1.0f, 0.f}, mul(r, q));
  const float f = n < -126.f ? 0.f : __uint_as_float(static_cast<uint32_t>(static_cast<int>(n) + 127) << 23);
  return {q.h * f, q.l * f};
}

__device__ __forceinline__ Pair reciprocal(Pair d) {  // of 1 and more
  const float q = __frcp_rn(d.h);
  return fast_sum(q, __fmul_rn(q, __fmaf_rn(-q, d.l, __fmaf_rn(-q, d.h, 1.0f))));
}

__device__ __forceinline__ Pair sigmoid_pair(float l) {
  const Pair e = exp_pair({-fabsf(l), 0.f});
  const Pair d = fast_sum(1.0f, e.h), q = reciprocal(fast_sum(d.h, __fadd_rn(d.l, e.l)));
  return l >= 0.f ? q : mul(e, q);
}

// Pairs in their order as integers: of -inf 0x007fffff80000000, of all others more.
__device__ __forceinline__ uint64_t pair_key(Pair x) { return static_cast<uint64_t>(float_key(x.h)) << 32 | float_key(x.l); }
__device__ __forceinline__ Pair key_pair(uint64_t k) {
  return {key_float(static_cast<uint32_t>(k >> 32)), key_float(static_cast<uint32_t>(k))};
}
constexpr uint64_t NOT_AVAILABLE = 0x007fffff80000000ull;

// The largest of the lanes' x, by two reductions of 32 bits.
__device__ __forceinline__ uint64_t warp_max_u64(uint64_t x) {
  const uint32_t hi = static_cast<uint32_t>(x >> 32), top = __reduce_max_sync(FULL, hi);
  const uint32_t lo = __reduce_max_sync(FULL, hi == top ? static_cast<uint32_t>(x) : 0u);
  return static_cast<uint64_t>(top) << 32 | lo;
}

// What softmax's scores hang on, by the whole warp: the largest logit and 1 / sum.
struct Scale {
  float top;
  Pair inv;
};

__device__ __forceinline__ Scale softmax_scale(const float* row, const Lane& me) {
  float top = -INFINITY;
#pragma unroll 4
  for (int i = 0; i < me.n; ++i) top = fmaxf(top, available(__ldg(row + me.first + i)));
  __syncwarp();
  top = key_float(__reduce_max_sync(FULL, float_key(top)));
  Pair total = {0.f, 0.f};
#pragma unroll 2
  for (int i = 0; i < me.n; ++i) {
    const float l = available(__ldg(row + me.first + i));
    if (l != -INFINITY) total = add(total, exp_pair(sum(l, -top)));
  }
  __syncwarp();
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1)
    total = add(total, {__shfl_xor_sync(FULL, total.h, m), __shfl_xor_sync(FULL, total.l, m)});
  return {top, reciprocal(total)};
}

// The value of expert e, logit l.
template <Mode MODE>
__device__ __forceinline__ uint64_t value_of(float l, int e, const Gate& g, const Scale& s) {
  if (l == -INFINITY) return NOT_AVAILABLE;
  Pair v = {l, 0.f};
  if (MODE != BY_LOGIT) {
    v = MODE == SOFTMAX ? mul(exp_pair(sum(l, -s.top)), s.inv) : sigmoid_pair(l);
    if (g.bias) v = add(v, {__ldg(g.bias + e), 0.f});
    if (!(fabsf(v.h) < INFINITY)) {  // a bias that is not finite
      if (!(v.h > 0.f)) return NOT_AVAILABLE;
      v = {FLT_MAX, 0.f};
    }
  }
  return pair_key(v);
}

// Whether the lane's group stays, by the whole warp.
template <Mode MODE>
__device__ __forceinline__ bool group_stays(const float* row, const Lane& me, const Gate& g, const Scale& s) {
  uint64_t c1 = 0, c2 = 0;
#pragma unroll 2
  for (int i = 0; i < me.n; ++i) {
    const uint64_t x = value_of<MODE>(available(__ldg(row + me.first + i)), me.first + i, g, s), lo = min(c1, x);
    c1 = max(c1, x);
    c2 = max(c2, lo);
  }
  __syncwarp();
  for (int m = 1; m < 1 << g.lanes_log; m <<= 1) {
    const uint64_t o1 = __shfl_xor_sync(FULL, c1, m), o2 = __shfl_xor_sync(FULL, c2, m);
    c2 = max(min(c1, o1), max(c2, o2));
    c1 = max(c1, o1);
  }
  const uint64_t mine = g.top2 && c2 > NOT_AVAILABLE ? pair_key(add(key_pair(c1), key_pair(c2))) : c1;
  int ahead = 0;
  for (int m = 1; m << g.lanes_log < 32; ++m) {
    const uint64_t o = __shfl_xor_sync(FULL, mine, m << g.lanes_log);
    ahead += o > mine || (o == mine && (me.group ^ m) < me.group);
  }
  return ahead < g.top_groups && me.group < g.groups;
}

// The choice among the groups that stay with every value worked out anew for each of the k: for tokens of
// which more experts are close to the last one chosen than a warp has lanes, or, with 32 chosen, any other.  Slow:
// 400 tokens of 1024 experts, 32 chosen, take 437 us (softmax; with 31 chosen 29), for one to three tokens of them.
template <Mode MODE>
__device__ __forceinline__ int choose_slowly(const float* row, const Lane& me, bool stays, const Gate& g, const Scale& s,
                                             int lane) {
  uint64_t last = ~0ull;
  int last_e = -1, id = 0;
#pragma unroll 1
  for (int j = 0; j < g.k; ++j) {
    uint64_t best = 0;
    int at = 0;
#pragma unroll 1
    for (int i = 0; stays && i < me.n; ++i) {
      const int e = me.first + i;
      const uint64_t x = value_of<MODE>(available(__ldg(row + e)), e, g, s);
      if (x > best && (x < last || (x == last && e > last_e))) {
        best = x;
        at = e;
      }
    }
    __syncwarp();
    const uint64_t most = warp_max_u64(best);
    const int win = __ffs(__ballot_sync(FULL, best == most)) - 1;
    last = most;
    last_e = __shfl_sync(FULL, at, win);
    if (lane == j) id = last_e;
  }
  return id;
}

// m of experts that are not available, and of none that is.
template <int IDX, Mode MODE>
__host__ __device__ constexpr uint32_t not_available_m() {
  return MODE == BY_LOGIT ? 0x007fffffu >> (IDX + 1) : 1u;
}

// What a warp keeps from token to token: its experts' biases in units, and what a unit is.
//   m = s a + base_e,  base_e = (b_e - least bias) a + 2,  below 2^(31 - IDX)
// computed as FP32 numbers of 2^23 and more, whose lower bits are the integer.
template <int EPL, int IDX, Mode MODE>
struct Units {
  static constexpr bool KEEP = EPL <= 8;
  float a, least;
  float base[KEEP ? EPL : 1];

  __device__ __forceinline__ float at(float b) const { return fmaf(b - least, a, 8388608.0f + 2.0f); }

  __device__ __forceinline__ Units(const Gate& g, const Lane& me) : a(0.f), least(0.f) {
    if (MODE == BY_LOGIT) return;
    float most = 0.f;
    if (g.bias) {
      float lo = INFINITY, hi = -INFINITY;
      bool nan = false;
      for (int i = 0; i < me.n; ++i) {
        const float b = __ldg(g.bias + me.first + i);
        lo = fminf(lo, b);
        hi = fmaxf(hi, b);
        nan |= b != b;
      }
      least = key_float(__reduce_min_sync(FULL, float_key(lo)));
      most = __any_sync(FULL, nan) ? INFINITY : key_float(__reduce_max_sync(FULL, float_key(hi)));
    }
    // (a range that is not finite leaves nothing to compare: every token is then done in 64 bits)
    const float range = most - least + 1.0f;
    if (range < 1e30f) {
      a = (static_cast<float>(1 << (31 - IDX)) - 16.0f) / range;
    } else {
      least = 0.f;
    }
    if (KEEP) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) base[KEEP ? i : 0] = at(g.bias && a > 0.f && i < me.n ? __ldg(g.bias + me.first + i) : least);
    }
  }
};

// Loads a lane's logits; VEC: they start on 16 bytes and are a multiple of four.  (By way of L1, which has them
// still when the chosen ones are read again.)
template <int EPL, bool VEC>
__device__ __forceinline__ void load_logits(const float* row, const Lane& me, float (&l)[EPL]) {
#pragma unroll
  for (int i = 0; i < EPL; ++i) l[i] = -INFINITY;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4)
      if (i < me.n) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(row + me.first + i));
        l[i] = x.x, l[i + 1] = x.y, l[i + 2] = x.z, l[i + 3] = x.w;
      }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (i < me.n) l[i] = __ldg(row + me.first + i);
  }
}

// The largest of the lane's keys below `under`, less `under` (modulo 2^32); minus: 0 - under.  Keys are 31 bits:
// of a key below the difference has its top bit set, of all others not.
template <int EPL>
__device__ __forceinline__ uint32_t below(const uint32_t (&key)[EPL], uint32_t minus) {
  uint32_t d = key[0] + minus;
#pragma unroll
  for (int i = 1; i < EPL; ++i) d = __viaddmax_u32(key[i], minus, d);
  return d;
}

// How many tokens a warp does together: as many as have room for their k choices side by side in its lanes,
// and for a group's score each in the group's lanes.
__host__ __device__ inline int batch_of(const Gate& g, int width) {
  int n = g.k <= 8 ? 4 : g.k <= 16 ? 2 : 1;
  if (g.top_groups < g.groups && n > 1 << g.lanes_log) n = 1 << g.lanes_log;
  while (n * width > 32 && n > 1) n >>= 1;
  return n;
}

// The second look at a token whose groups are beyond doubt: those that may be among the k by their keys (the k
// and all within `near` of the last), a lane each, sorted by scores of twice the length.  key: the lane's
// keys, 0 where its group does not stay; blur: the relative error of 1 / sum (softmax).  Lane j < k gets the
// j-th choice; false: more candidates than lanes, or two that the blur could exchange.
template <int EPL, int IDX, Mode MODE>
__device__ __forceinline__ bool choose_close(const float* row, const uint32_t (&key)[EPL], uint32_t near,
                                             const Scale& scale, float blur, const Gate& g, int lane, int* choice) {
  constexpr uint32_t MASK = (1u << IDX) - 1u, OUT = not_available_m<IDX, MODE>();
  uint32_t last = 0x80000000u, kth = 0, mine = 0;
  int n = 0;
#pragma unroll 1
  for (;; ++n) {
    const uint32_t d = __reduce_max_sync(FULL, below(key, 0u - last));
    const uint32_t next = d >> 31 ? last + d : 0u;
    if (n >= g.k && (next >> IDX <= OUT || (kth >> IDX) - (next >> IDX) > near)) break;
    if (n == 32) return false;
    last = next;
    if (n == g.k - 1) kth = last;
    if (lane == n) mine = last;
  }
  const int id = min(static_cast<int>(MASK - (mine & MASK)), g.E - 1);
  const float x = lane < n ? available(__ldg(row + id)) : -INFINITY;
  const float bias = MODE != BY_LOGIT && g.bias && lane < n ? __ldg(g.bias + id) : 0.f;
  if (!__all_sync(FULL, fabsf(bias) < INFINITY)) return false;
  Pair v = {x, 0.f};
  float off = 0.f;
  if (MODE != BY_LOGIT && x != -INFINITY) {
    v = MODE == SOFTMAX ? mul(exp_pair(sum(x, -scale.top)), scale.inv) : sigmoid_pair(x);
    off = blur * v.h;
    v = add(v, {bias, 0.f});
  }
  const uint64_t value = x == -INFINITY ? NOT_AVAILABLE : pair_key(v);
  int ahead = 0;
#pragma unroll 1
  for (int o = 0; o < n; ++o) {
    const uint64_t other = __shfl_sync(FULL, value, o);
    const int e = __shfl_sync(FULL, id, o);
    ahead += other > value || (other == value && e < id);
  }
  // in order: lane j takes over from the lane that has j ahead of it
  int from = lane;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const int o = __ffs(__ballot_sync(FULL, lane < n && ahead == j)) - 1;
    if (lane == j) from = o;
  }
  *choice = __shfl_sync(FULL, id, from);
  if (MODE != SOFTMAX || blur == 0.f) return true;
  // neighbours (every lane takes part in every exchange)
  const int after = __shfl_down_sync(FULL, from, 1);
  const float h = __shfl_sync(FULL, v.h, from), h2 = __shfl_sync(FULL, v.h, after);
  const float l = __shfl_sync(FULL, v.l, from), l2 = __shfl_sync(FULL, v.l, after);
  const float o = __shfl_sync(FULL, off, from), o2 = __shfl_sync(FULL, off, after);
  const float x1 = __shfl_sync(FULL, x, from), x2 = __shfl_sync(FULL, x, after);
  const float b1 = __shfl_sync(FULL, bias, from), b2 = __shfl_sync(FULL, bias, after);
  const bool alike = x1 == x2 && b1 == b2;
  return !__any_sync(FULL, lane + 1 < n && x2 != -INFINITY && !alike && !((h - h2) + (l - l2) > o + o2));
}

// What a warp makes of a token's logits.
struct Made {
  float top, inv;  // softmax: the largest logit, 1 / sum (the largest score)
  uint32_t near;   // the largest difference of two m that errors may account for
};

// Keys of a lane's logits.  `near`: each m is off by its score's error and 1.5 (b - least, base, m).  Sigmoid: the
// fast exponential is off by (2 + 1.16 |l|) 2^-23, which enters s times 1 - s (s (1 - s) <= 1/4, s (1 - s) |l| <=
// 0.224), the sum by 2^-24, the reciprocal by 2^-23: below 5e-7.  Softmax: s times 1.5e-6 and 2^-24 per addition
// (expf 2^-22, its argument 2^-24 (top - l), on average at most ln 1024 2^-24, sum, reciprocal, product), and
// 2^-24 s (top - l) <= 2^-24 0.37 / sum.
template <int EPL, int IDX, Mode MODE, bool WHOLE>
__device__ __forceinline__ Made make_keys(const float (&l)[EPL], const Units<EPL, IDX, MODE>& u, const Gate& g,
                                          const Lane& me, uint32_t (&key)[EPL]) {
  constexpr uint32_t MASK = (1u << IDX) - 1u, OUT = not_available_m<IDX, MODE>();
  Made made = {0.f, 0.f, 0};
  float e[MODE == SOFTMAX ? EPL : 1];
  if (MODE == SOFTMAX || (MODE == BY_LOGIT && g.softmax && !g.renorm)) {
    float most = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) most = fmaxf(most, available(l[i]));
    most = key_float(__reduce_max_sync(FULL, float_key(most)));
    made.top = most == -INFINITY ? 0.f : most;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float x = expf(available(l[i]) - made.top);
      sum += x;
      if (MODE == SOFTMAX) e[MODE == SOFTMAX ? i : 0] = x;
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(FULL, sum, m);
    made.inv = sum > 0.f ? 1.0f / sum : 0.f;
  }
  if (MODE == SIGMOID) made.near = static_cast<uint32_t>(1e-6f * u.a) + 5u;
  if (MODE == SOFTMAX) made.near = static_cast<uint32_t>((3.1e-6f + 1.2e-7f * EPL) * made.inv * u.a) + 5u;
  // (0 x: NaN of what is not finite; a comparison per expert would cost twice as much)
  bool odd = true;
  if (WHOLE && MODE != BY_LOGIT) {
    float zero = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) zero = fmaf(l[i], 0.f, zero);
    odd = __any_sync(FULL, zero != 0.f);
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const uint32_t index = MASK - static_cast<uint32_t>(me.first + i);
    if (MODE == BY_LOGIT) {
      key[i] = (float_key(available(l[i])) >> (IDX + 1) << IDX) | index;
    } else {
      const float s = MODE == SOFTMAX ? e[MODE == SOFTMAX ? i : 0] * made.inv
                                      : fast_rcp(1.0f + fast_exp2(l[i] * -1.44269504f));
      float base;
      if (u.KEEP)
        base = u.base[u.KEEP ? i : 0];
      else
        base = u.at(g.bias && u.a > 0.f && i < me.n ? __ldg(g.bias + me.first + i) : u.least);
      const uint32_t m = __float_as_uint(fmaf(s, u.a, base));
      if (IDX == 8)  // the integer's three bytes and the index's, of which a word holds four
        key[i] = __byte_perm(m, (index + i % 4) * 0x01010101u - 0x03020100u, 0x2104 + i % 4);
      else
        key[i] = (m << IDX) + index;
    }
    if (!WHOLE && i >= me.n) key[i] = 0;
  }
  if (MODE != BY_LOGIT && odd) {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (!(l[i] > -INFINITY) && (WHOLE || i < me.n)) key[i] = (OUT << IDX) + MASK - static_cast<uint32_t>(me.first + i);
  }
  return made;
}

// The logits of tokens t .. t + BATCH - 1 (the last one again for those from T on).
template <int EPL, int BATCH, bool WHOLE>
__device__ __forceinline__ void load_tokens(const float* logits, int t, int T, const Gate& g, const Lane& me,
                                            float (&l)[BATCH][EPL]) {
#pragma unroll
  for (int b = 0; b < BATCH; ++b) load_logits<EPL, WHOLE>(logits + static_cast<size_t>(min(t + b, T - 1)) * g.E, me, l[b]);
}

// Tokens t .. t + BATCH - 1 (those below T) by one warp: lane i (32 / BATCH) + j ends with the j-th choice of
// token t + i and its weight.  l: load_tokens'.  WHOLE: every lane has EPL experts, which start on 16 bytes, or none
// (the last lanes of 232, 240 and 248 experts, or of two groups of 120).  The keys of those that have none name
// experts behind the group's, as not available: behind the 120 or more of the group itself, of which at most 32 are chosen.
template <int EPL, int IDX, Mode MODE, int BATCH, bool WHOLE>
__device__ __forceinline__ void warp_gate(const float* logits, int t, int T, const float (&l)[BATCH][EPL],
                                          const Units<EPL, IDX, MODE>& u, const Gate& g, const Lane& me, int lane,
                                          int* id_out, float* w_out) {
  constexpr uint32_t MASK = (1u << IDX) - 1u, OUT = not_available_m<IDX, MODE>();
  constexpr int SEG = 32 / BATCH;
  const int ti = lane / SEG, tj = lane % SEG;  // whose choice this lane ends with
  uint32_t key[BATCH][EPL];
  float top = 0.f, inv = 0.f;  // this lane's token's
  uint32_t near[BATCH];
  uint32_t c1 = 0, c2 = 0;  // the two largest keys of this lane's group, of token (lane modulo BATCH)
  const bool drop = g.top_groups < g.groups;
  {
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const Made made = make_keys<EPL, IDX, MODE, WHOLE>(l[b], u, g, me, key[b]);
      near[b] = made.near;
      if (ti == b) {
        top = made.top;
        inv = made.inv;
      }
      if (drop) {
        uint32_t a1 = 0, a2 = 0;
#pragma unroll
        for (int i = 0; i < EPL; i += 2) {
          const uint32_t hi = EPL == 1 ? key[b][i] : max(key[b][i], key[b][(i + 1) % EPL]);
          const uint32_t lo = EPL == 1 ? 0u : min(key[b][i], key[b][(i + 1) % EPL]);
          a2 = __vimax3_u32(min(a1, hi), a2, lo);
          a1 = max(a1, hi);
        }
        for (int m = 1; m < 1 << g.lanes_log; m <<= 1) {
          const uint32_t o1 = __shfl_xor_sync(FULL, a1, m), o2 = __shfl_xor_sync(FULL, a2, m);
          a2 = __vimax3_u32(min(a1, o1), a2, o2);
          a1 = max(a1, o1);
        }
        if (BATCH == 1 || (lane & (BATCH - 1)) == b) {
          c1 = a1 >> IDX;
          c2 = a2 >> IDX;
        }
      }
    }
  }
  // tokens whose choice may hang on a rounding, a bit each: that of the groups, or of the experts in them
  uint32_t unsure = 0, close = 0;
  if (MODE != BY_LOGIT && !(u.a > 0.f)) unsure = (1u << BATCH) - 1u;
  // ---- groups: lane's own, of token (lane modulo BATCH)
  uint32_t stays = ~0u;
  if (drop) {
    // The score in units, from 1 on (0: none available), and the group's index.  A sum of two counts from
    // twice the least bias, a lone value from that once.
    uint32_t worth = 0;
    bool doubt = false;
    if (c1 > OUT) {
      worth = c1;
      if (MODE != BY_LOGIT && g.top2) {
        const float from = fminf(fmaxf(rintf(u.least * u.a), -33554432.f), 33554432.f);
        const int up = max(static_cast<int>(from), 0);
        worth = static_cast<uint32_t>(c2 > OUT ? static_cast<int>(c1 + c2) - 3 + up
                                               : max(static_cast<int>(c1) - 1 + up - static_cast<int>(from), 1));
        doubt = c2 <= OUT && fabsf(from) > 16777216.f;
      }
    }
    const uint32_t mine = me.group < g.groups ? (worth + 1u) << 5 | static_cast<uint32_t>(31 - me.group) : 0u;
    // places of the groups, and the best score of those behind this one
    int ahead = 0;
    uint32_t behind = 0;
    for (int m = 1; m << g.lanes_log < 32; ++m) {
      const uint32_t o = __shfl_xor_sync(FULL, mine, m << g.lanes_log);
      ahead += o > mine;
      behind = max(behind, o < mine ? o : 0u);
    }
    // (a group without an available expert is behind all others for sure)
    uint32_t slack = near[0];
    if (MODE == SOFTMAX) {
#pragma unroll
      for (int b = 1; b < BATCH; ++b) slack = (lane & (BATCH - 1)) == b ? near[b] : slack;
    }
    if (ahead == g.top_groups - 1 && behind >> 5 > 1u && (mine >> 5) - (behind >> 5) <= (g.top2 ? 2u * slack + 4u : slack)) doubt = true;
    const uint32_t in = __ballot_sync(FULL, ahead < g.top_groups && me.group < g.groups);
    const uint32_t un = __ballot_sync(FULL, doubt);
    stays = 0;
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      stays |= (in >> ((me.group << g.lanes_log) + b) & 1u) << b;
      uint32_t of_b = 0;  // the lanes that speak for token b
#pragma unroll
      for (int i = b; i < 32; i += BATCH) of_b |= 1u << i;
      if (un & of_b) unsure |= 1u << b;
    }
  }
  // ---- the k largest of each token (side by side: a round is a chain of latencies)
  uint32_t chosen = 0, others = 0, minus[BATCH];  // minus: 0 less the last one chosen
  constexpr uint32_t NO_KEY = 0x7fffffffu;        // above all keys, and so never below one chosen
#pragma unroll
  for (int b = 0; b < BATCH; ++b) {
    minus[b] = 0u - NO_KEY;
    if (drop) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[b][i] = stays >> b & 1u ? key[b][i] : NO_KEY;
    }
  }
#pragma unroll 1
  for (int j = 0; j < g.k; ++j) {
    uint32_t mine = 0;
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      minus[b] -= __reduce_max_sync(FULL, below(key[b], minus[b]));
      if (ti == b) mine = minus[b];
    }
    if (tj == j) chosen = 0u - mine;
  }
#pragma unroll
  for (int b = 0; b < BATCH; ++b) {
    const uint32_t most = __reduce_max_sync(FULL, below(key[b], minus[b])), last = 0u - minus[b];
    const uint32_t next = most >> 31 ? last + most : 0u;
    // every other expert that may be ahead of the last one chosen has to tie with it in logit and bias
    if (next >> IDX > OUT && (last >> IDX) - (next >> IDX) <= near[b]) {
      const float* row = logits + static_cast<size_t>(min(t + b, T - 1)) * g.E;
      const int idk = min(static_cast<int>(MASK - (last & MASK)), g.E - 1);
      const float xk = available(__ldg(row + idk)), bk = g.bias ? __ldg(g.bias + idk) : 0.f;
      bool alike = true;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const uint32_t x = key[b][i];
        if (x >= last || x >> IDX <= OUT || (last >> IDX) - (x >> IDX) > near[b]) continue;
        const float xi = available(__ldg(row + me.first + i)), bi = g.bias ? __ldg(g.bias + me.first + i) : 0.f;
        if (!(xi == xk && bi == bk)) alike = false;
      }
      if (!__all_sync(FULL, alike)) close |= 1u << b;
    }
    if (ti == b) others = near[b];
  }
  int id = min(static_cast<int>(MASK - (chosen & MASK)), g.E - 1);
  const float* row = logits + static_cast<size_t>(min(t + ti, T - 1)) * g.E;
  float x = tj < g.k ? available(__ldg(row + id)) : -INFINITY;
  // ---- neighbours in the choice
  {
    const uint32_t m = chosen >> IDX, m2 = __shfl_down_sync(FULL, m, 1);
    const bool near_by = tj + 1 < g.k && m2 > OUT && m - m2 <= others;
    if (__any_sync(FULL, near_by)) {
      const float bias = g.bias && tj < g.k ? __ldg(g.bias + id) : 0.f;
      const float x2 = __shfl_down_sync(FULL, x, 1), b2 = __shfl_down_sync(FULL, bias, 1);
      const uint32_t un = __ballot_sync(FULL, near_by && !(x == x2 && bias == b2));
#pragma unroll
      for (int b = 0; b < BATCH; ++b)
        if (un >> (b * SEG) & (SEG == 32 ? FULL : (1u << (SEG & 31)) - 1u)) close |= 1u << b;
    }
  }
  const uint32_t here = T - t < BATCH ? (1u << (T - t)) - 1u : (1u << BATCH) - 1u;
  unsure &= here;
  close &= here & ~unsure;
  if (unsure | close) {
#pragma unroll 1
    for (uint32_t left = unsure | close; left; left &= left - 1u) {
      const int b = __ffs(left) - 1;
      const float* at = logits + static_cast<size_t>(t + b) * g.E;
      // (its keys anew: those of groups that do not stay are gone)
      float again[EPL];
      uint32_t own[EPL];
      load_logits<EPL, WHOLE>(at, me, again);
      const Made made = make_keys<EPL, IDX, MODE, WHOLE>(again, u, g, me, own);
      bool in = stays >> b & 1u;
      // softmax: with 1 / sum as it is first, unless the groups need it exact anyway
      Scale scale = {made.top, {made.inv, 0.f}};
      float blur = MODE == SOFTMAX ? 1.5e-6f + 6e-8f * EPL : 0.f;
      bool groups = unsure >> b & 1u, done = false;
      int e = 0;
#pragma unroll 1
      for (int go = 0; go < 2 && !done; ++go) {
        if (MODE == SOFTMAX && (groups || go == 1)) {
          scale = softmax_scale(at, me);
          blur = 0.f;
        }
        if (groups && drop) in = group_stays<MODE>(at, me, g, scale);
        groups = false;
#pragma unroll
        for (int i = 0; i < EPL; ++i) own[i] = in ? own[i] : 0u;
        done = choose_close<EPL, IDX, MODE>(at, own, made.near, scale, blur, g, lane, &e);
        if (blur == 0.f) break;
      }
      if (!done) e = choose_slowly<MODE>(at, me, in, g, scale, lane);
      const int mine = __shfl_sync(FULL, e, tj);
      if (ti == b) id = min(max(mine, 0), g.E - 1);
    }
    if (tj < g.k) x = available(__ldg(row + id));
  }
  // ---- weights
  float z = 0.f, most = x;
  if (g.renorm) {
#pragma unroll
    for (int m = SEG / 2; m >= 1; m >>= 1) most = fmaxf(most, __shfl_xor_sync(FULL, most, m));
  }
  if (g.renorm && (g.softmax || most < 0.f)) {
    // exp(x - the chosen ones' largest), so that scores which 32 bits do not hold keep their ratios; the difference
    // is carried exactly (two-sum).  Sigmoid: e^x / (1 + e^x) over e^most; from 0 on the largest is 1/2 or more.
    const float hi = x - most;
    if (hi > -104.f) {  // (e^-104 is 0 in 32 bits; a difference that overflows leaves a rest that is NaN)
      const float bb = hi - x, lo = (x - (hi - bb)) + (-most - bb);
      z = expf(hi) * (1.0f + lo);
      if (!g.softmax) z /= 1.0f + expf(x);
    }
  } else if (x != -INFINITY) {
    z = g.softmax ? expf(x - top) * inv : 1.0f / (1.0f + expf(-x));
  }
  if (g.renorm) {
    float sum = z;
#pragma unroll
    for (int m = SEG / 2; m >= 1; m >>= 1) sum += __shfl_xor_sync(FULL, sum, m);
    z = sum > 0.f ? z / sum : 0.f;
  }
  *id_out = id;
  *w_out = z * g.scale;
}

}  // namespace gate_dev
}  // namespace moe
