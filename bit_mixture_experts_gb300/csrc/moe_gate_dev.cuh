// The choice of a token's experts by one warp, for routers with sigmoid or
// softmax scores, a bias that takes part in the choice alone, groups of experts
// of which the best stay, and weights that are renormalised and scaled:
//
//   s_e = sigmoid(l_e)  or  exp(l_e - m) / sum_i exp(l_i - m)
//   v_e = s_e + b_e;  chosen: the k largest v_e of the groups that stay, in
//   descending order, equal ones by index
//   w_j = scale s_j / (sum of the chosen s, or 1)
//
// The choice has to be what exact scores give, and FP32 scores can be off by
// more than two experts differ.  So the FP32 choice comes with a bound on the
// error of each v, and where two neighbours of the sorted choice, the last one
// chosen and any other expert, or the last group that stays and the first that
// does not are nearer to each other than their bounds, the token is done again
// in 64 bits (about one token in a thousand at 256 experts).  Experts whose
// logit and bias are the same bits tie in any precision and need no second
// look.  Without a bias the scores are monotone in the logits, which are then
// compared themselves, exactly.
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

// Bound on |s - exact| = rel s + abs.  Sigmoid: the fast exponential is off by (2 + 1.16 |l|) 2^-23, which
// enters s times 1 - s (s (1 - s) <= 1/4, s (1 - s) |l| <= 0.224), the sum by 2^-24, the division by 2^-22.
// Softmax: expf by 2^-22, its argument by 2^-24 (m - l), together at most 2^-24 0.37 / sum that enters
// absolutely (x e^-x <= 0.37); the sum by as much on average (at most ln 1024 2^-24) and its additions.
struct Bound {
  float rel, abs;
};

__device__ __forceinline__ float available(float l) {  // NaN counts as -inf, +inf as the largest number
  return l > -INFINITY ? fminf(l, FLT_MAX) : -INFINITY;
}

__device__ __forceinline__ float fast_sigmoid(float l) { return __fdividef(1.0f, 1.0f + __expf(-l)); }

// ---- the same in 64 bits; lane j < k gets the j-th choice
__device__ __forceinline__ uint64_t double_key(double x) {
  uint64_t u = static_cast<uint64_t>(__double_as_longlong(x));
  if (u == 0x8000000000000000ull) u = 0;
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

__device__ __forceinline__ uint64_t warp_max_u64(uint64_t x) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) {
    const uint64_t o = __shfl_xor_sync(FULL, x, m);
    x = o > x ? o : x;
  }
  return x;
}

static __device__ __noinline__ int choose_exact(const float* row, const Gate& g, int lane) {
  const int L = 1 << g.lanes_log, group = lane >> g.lanes_log, sub = lane & (L - 1);
  const int first = group * g.per_group + sub * g.width;
  const int n = group < g.groups ? min(max(g.per_group - sub * g.width, 0), g.width) : 0;
  const double none = -INFINITY;
  double v[MAX_WIDTH];
  float top = -INFINITY;
  for (int i = 0; i < n; ++i) top = fmaxf(top, available(__ldcg(row + first + i)));
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, m));
  double sum = 0.0;
  for (int i = 0; i < n; ++i) {
    const float l = available(__ldcg(row + first + i));
    v[i] = l == -INFINITY ? none : g.softmax ? exp(static_cast<double>(l) - top) : 1.0 / (1.0 + exp(-static_cast<double>(l)));
    if (v[i] != none) sum += v[i];
  }
  if (g.softmax) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(FULL, sum, m);
  }
  double c1 = none, c2 = none;
  for (int i = 0; i < n; ++i) {
    if (v[i] == none) continue;
    if (g.softmax) v[i] /= sum;
    if (g.bias) v[i] += static_cast<double>(__ldg(g.bias + first + i));
    if (!(v[i] == v[i])) v[i] = none;
    c2 = v[i] > c1 ? c1 : fmax(c2, v[i]);
    c1 = fmax(c1, v[i]);
  }
  bool stays = group < g.groups;
  if (g.top_groups < g.groups) {
    for (int m = 1; m < L; m <<= 1) {
      const double o1 = __shfl_xor_sync(FULL, c1, m), o2 = __shfl_xor_sync(FULL, c2, m);
      c2 = fmax(fmin(c1, o1), fmax(c2, o2));
      c1 = fmax(c1, o1);
    }
    const double mine = g.top2 && c2 != none ? c1 + c2 : c1;
    int ahead = 0;
    for (int o = 0; o < g.groups; ++o) {
      const double other = __shfl_sync(FULL, mine, o << g.lanes_log);
      ahead += other > mine || (other == mine && o < group);
    }
    stays &= ahead < g.top_groups;
  }
  uint64_t taken = 0;
  int id = 0;
  for (int j = 0; j < g.k; ++j) {
    uint64_t best = 0;
    int at = 0;
    for (int i = 0; stays && i < n; ++i) {
      const uint64_t key = double_key(v[i]);
      if (!(taken >> i & 1) && key > best) {
        best = key;
        at = i;
      }
    }
    const uint64_t most = warp_max_u64(best);
    const int win = __ffs(__ballot_sync(FULL, best == most)) - 1;
    if (lane == win) taken |= 1ull << at;
    const int e = __shfl_sync(FULL, first + at, win);
    if (lane == j) id = e;
  }
  return min(id, g.E - 1);
}

// Lane j < k ends with the token's j-th choice and its weight.  EPL >= g.width; VEC: the lane's experts
// start on 16 bytes and are a multiple of four.  The row is read through L2 (it may have been written by
// other CTAs of the same kernel).
template <int EPL, bool VEC>
__device__ __forceinline__ void warp_gate(const float* row, const Gate& g, int lane, int* id_out, float* w_out) {
  const int L = 1 << g.lanes_log, group = lane >> g.lanes_log, sub = lane & (L - 1);
  const int first = group * g.per_group + sub * g.width;
  const int n = group < g.groups ? min(max(g.per_group - sub * g.width, 0), g.width) : 0;
  float v[EPL];  // logits, then what is compared
#pragma unroll
  for (int i = 0; i < EPL; ++i) v[i] = -INFINITY;
  if (VEC) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4)
      if (i < n) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(row + first + i));
        v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
      }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (i < n) v[i] = __ldcg(row + first + i);
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) v[i] = available(v[i]);
  float top = 0.f, inv = 0.f;  // softmax over all experts: the largest logit, 1 / sum (which is the largest score)
  if (g.softmax && !(g.by_logit && g.renorm)) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) top = fmaxf(top, v[i]);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, m));
    if (top == -INFINITY) top = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float e = expf(v[i] - top);
      sum += e;
      if (!g.by_logit && v[i] != -INFINITY) v[i] = e;
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(FULL, sum, m);
    inv = sum > 0.f ? 1.0f / sum : 0.f;
  }
  Bound err = {0.f, 0.f};
  if (!g.by_logit) {
    err = g.softmax ? Bound{1.5e-6f + 6e-8f * EPL, 3e-8f * inv + 1e-37f} : Bound{4e-7f, 1e-7f};
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (v[i] != -INFINITY) {
        const float s = g.softmax ? v[i] * inv : fast_sigmoid(v[i]);
        v[i] = g.bias ? fmaxf(s + __ldg(g.bias + first + i), -INFINITY) : s;
      }
  }
  bool sure = true;  // false: the choice may hang on a rounding
  // ---- groups
  bool stays = true;
  if (g.top_groups < g.groups) {
    float c1 = -INFINITY, c2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      c2 = fmaxf(c2, fminf(c1, v[i]));
      c1 = fmaxf(c1, v[i]);
    }
    for (int m = 1; m < L; m <<= 1) {
      const float o1 = __shfl_xor_sync(FULL, c1, m), o2 = __shfl_xor_sync(FULL, c2, m);
      c2 = fmaxf(fminf(c1, o1), fmaxf(c2, o2));
      c1 = fmaxf(c1, o1);
    }
    const float mine = g.top2 && c2 != -INFINITY ? c1 + c2 : c1;
    int ahead = 0;
    for (int o = 0; o < g.groups; ++o) {
      const float other = __shfl_sync(FULL, mine, o << g.lanes_log);
      ahead += other > mine || (other == mine && o < group);
    }
    stays = ahead < g.top_groups && group < g.groups;
    if (!g.by_logit) {
      const uint32_t key = float_key(mine);
      const float last = key_float(__reduce_min_sync(FULL, stays ? key : 0xffffffffu));
      const float next = key_float(__reduce_max_sync(FULL, stays || group >= g.groups ? 0u : key));
      const float most = g.softmax ? inv : 1.0f;
      const float a1 = c1 == -INFINITY ? 0.f : fabsf(c1), a2 = c2 == -INFINITY ? 0.f : fabsf(c2);
      const float d = 4.f * (err.rel * most + err.abs) + (fabsf(last) + fabsf(next) + 2.f * fmaxf(a1, a2)) * 2.4e-7f;
      // (a group without an available expert is behind all others for sure)
      if (next != -INFINITY && !(last - next > d)) sure = false;
      sure = __all_sync(FULL, sure);
    }
  }
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) key[i] = stays && i < n ? float_key(v[i]) : 0u;
  // ---- the k largest: lower lanes have lower experts
  uint32_t best = 0, my_key = 0;
  int id = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) best = max(best, key[i]);
  for (int j = 0; j < g.k; ++j) {
    const uint32_t most = __reduce_max_sync(FULL, best);
    const int win = __ffs(__ballot_sync(FULL, best == most)) - 1;
    int at = 0;
    if (lane == win) {
      bool done = false;
      best = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (!done && key[i] == most) {
          done = true;
          key[i] = 0;
          at = i;
        }
        best = max(best, key[i]);
      }
    }
    const int e = __shfl_sync(FULL, first + at, win);
    if (lane == j) {
      id = e;
      my_key = most;
    }
  }
  id = min(id, g.E - 1);
  // ---- is the choice beyond doubt?
  if (!g.by_logit) {
    float c = key_float(my_key);
    const float l = available(__ldcg(row + id)), b = g.bias ? __ldg(g.bias + id) : 0.f;
    const float s = l == -INFINITY ? 0.f : g.softmax ? expf(l - top) * inv : fast_sigmoid(l);
    const float dc = err.rel * s + err.abs + fabsf(c) * 1.2e-7f;
    const float c2 = __shfl_down_sync(FULL, c, 1), l2 = __shfl_down_sync(FULL, l, 1), b2 = __shfl_down_sync(FULL, b, 1),
                dc2 = __shfl_down_sync(FULL, dc, 1);
    if (lane + 1 < g.k && c2 != -INFINITY && !(c - c2 > dc + dc2) && !(l == l2 && b == b2)) sure = false;
    // the last one chosen and the others
    const float ck = __shfl_sync(FULL, c, g.k - 1), dk = __shfl_sync(FULL, dc, g.k - 1);
    const float most = g.softmax ? inv : 1.0f;
    const float cu = key_float(best);  // this lane's best other one
    if (__any_sync(FULL, best > 0x007fffffu && !(ck - cu > dk + err.rel * most + err.abs + fabsf(cu) * 1.2e-7f))) {
      const float lk = __shfl_sync(FULL, l, g.k - 1), bk = __shfl_sync(FULL, b, g.k - 1);
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const int e = first + i;
        const float lu = available(__ldcg(row + e)), bu = g.bias ? __ldg(g.bias + e) : 0.f;
        bool out = lu == -INFINITY || !stays;
        const float su = g.softmax ? expf(lu - top) * inv : fast_sigmoid(lu);
        const float vu = fmaxf(su + bu, -INFINITY);
        // (chosen ones are past the last one, or the last one itself)
        out |= vu == -INFINITY || (lu == lk && bu == bk) || vu > ck;
        if (!out && !(ck - vu > dk + err.rel * su + err.abs + fabsf(vu) * 1.2e-7f)) sure = false;
      }
    }
    if (!__all_sync(FULL, sure)) id = choose_exact(row, g, lane);
  }
  // ---- weights
  const float l = available(__ldcg(row + id));
  float z = 0.f;
  if (lane < g.k && l != -INFINITY) {
    if (!g.softmax)
      z = 1.0f / (1.0f + expf(-l));
    else if (!g.renorm)
      z = expf(l - top) * inv;
  }
  if (g.softmax && g.renorm) {
    // exp(l - the chosen ones' largest): the difference carried exactly (two-sum)
    float most = lane < g.k ? l : -INFINITY;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) most = fmaxf(most, __shfl_xor_sync(FULL, most, m));
    if (lane < g.k && l != -INFINITY) {
      const float hi = l - most, bb = hi - l, lo = (l - (hi - bb)) + (-most - bb);
      z = expf(hi) * (1.0f + lo);
    }
  }
  if (g.renorm) {
    float sum = z;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(FULL, sum, m);
    z = sum > 0.f ? z / sum : 0.f;
  }
  *id_out = id;
  *w_out = z * g.scale;
}

}  // namespace gate_dev
}  // namespace moe
