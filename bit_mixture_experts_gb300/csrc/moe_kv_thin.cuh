// The attention of an item with at most 32 query rows (a decode step, a few
// drafted tokens), on mma.sync.
//
// Such an item is bound by reading its keys and values, and a 128-row tile
// would spend its one-thread-per-row softmax on a handful of rows.  Instead the
// eight softmax warps share out the keys: 32 keys per warp and tile, four warps
// to a key tile (with up to 16 rows the other four take the next tile, with more
// they take the other 16 rows), each warp with its own running maximum, sum and
// output, joined once at the end of the item's run.  Keys and values come
// straight from where the copies land: e4m3 codes are expanded in registers,
// their scales applied to the scores and to the weights (powers of two), so the
// result is that of a bf16 cache with the same values, bit for bit while the
// value scales lie between 2^-90 and 2^90: weights are up to 2^8 and then
// rounded to bf16 times the scale, which has to stay a normal number.
//
// Two shapes of the products.  Up to 8 rows (NARROW): S^T = K Q^T and
// O^T = V^T P^T, the queries as the 8-wide operand; a row's scores lie in the
// eight lanes of equal q, and the weights are transposed by movmatrix.  More
// rows: S = Q K^T and O = P V, 16 rows per warp.  With 8 rows the second shape
// spends half of its products and accumulators on rows that do not exist:
// 8 e4m3 sequences over 2K to 32K 31.1 us in it, 29.9 narrow; one of 131071 27.2
// and 26.2.
//
// Fragments (mma.m16n8k16; lane = 4 gr + q): the sum over d may run in any
// order, so lane q of a quad takes d = (D/4) q .. + D/4 - 1 of its key's row as
// contiguous 16-byte loads, four values per step, and Q's fragments likewise.
// For P V the values are read four keys at a time (2q, 2q + 1, 2q + 8, 2q + 9):
// bf16 by ldmatrix.trans, e4m3 as 16-byte (D = 64: 8-byte) pieces whose column
// j + (D/8) gr belongs to step j.
//
// Measured (calls in a row from a CUDA graph, 2 KV heads of 128, 8 query heads
// each): 64 bf16 sequences over 1K to 8K tokens 57 us (floor 45: the keys and
// values at the copy rate), 8 e4m3 sequences 29.7 us (floor 13), of which copies
// alone, nothing computed, take 23, and launch, plan and merge 10.
#pragma once
#include "moe_kv_attn.cuh"

namespace moe {
namespace kv {

constexpr int THIN_ROWS = 32;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t a, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(a)
               : "memory");
}

// The transpose of an 8 x 8 matrix of 16-bit values, a row's pair per lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ float lds_float(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ float2 lds_float2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

// Byte B of x and of y (e4m3 codes) -> a bf16 pair of their values; see expand4.
template <int B>
__device__ __forceinline__ uint32_t expand_pair(uint32_t x, uint32_t y) {
  constexpr uint32_t sel = B | (8 + B) << 4 | (4 + B) << 8 | (12 + B) << 12;
  uint32_t a;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(a) : "r"(x), "r"(y), "n"(sel));
  return bf16x2_mul((a << 4) & 0x87f087f0u, 0x7b807b80u);  // times 2^120
}

// What the roles of the kernel share with the thin form.
struct ThinCtx {
  uint32_t sbase;
  uint8_t* smem;
  volatile int* s_abort;
  int warp, lane;  // warp: 0..7 of the team
};

// One segment by the team's eight warps, whose query rows have landed.  units: ring units before it;
// team_ph: phases of the TEAM barrier so far.  False when a wait gave up.
template <int D, bool Q8, bool NARROW>
__device__ __forceinline__ bool thin_segment(const Args& a, const AttnArgs& g, const Seg& sg, const ThinCtx& x, int cta,
                                             int units, uint32_t& team_ph) {
  using L = Layout<D, Q8>;
  constexpr int STEPS = D / 16, DQ = D / 4, QC = DQ / 8, NT = D / 8;
  constexpr int NO = NARROW ? D / 16 : NT, NF = NARROW ? 2 : 4;  // fragments of the output, of 32 keys
  const int lane = x.lane, gr = lane >> 2, q = lane & 3;
  const uint32_t sbase = x.sbase;
  auto bar = [sbase](int i) -> uint32_t { return sbase + L::BAR_OFF + 8u * static_cast<uint32_t>(i); };
  auto wait = [&](int i, uint32_t parity) -> bool {
    return wait_warp(bar(i), parity, x.s_abort, a.err, g);
  };
  auto team = [&]() -> bool {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar(L::TEAM));
    const bool ok = wait(L::TEAM, team_ph & 1);
    ++team_ph;
    return ok;
  };
  const int rows = sg.ntok * g.group;
  // up to 16 rows: warps 0-3 and 4-7 take alternate tiles; more: all tiles, rows 0-15 and 16-31
  const int groups = rows <= 16 ? 1 : 2;
  const int mg = groups == 1 ? 0 : x.warp >> 2, first_tile = groups == 1 ? x.warp >> 2 : 0, step = 3 - groups;
  const int first_key = (x.warp & 3) * 32;
  const int r0 = NARROW ? 2 * q : mg * 16 + gr, r1 = NARROW ? r0 + 1 : r0 + 8;
  const bool ok0 = r0 < rows, ok1 = r1 < rows;
  const int vis0 = sg.base + 1;  // keys that all rows see; row r sees those before vis0 + its token
  const int see0 = ok0 ? vis0 + r0 / g.group : 0, see1 = ok1 ? vis0 + r1 / g.group : 0;

  auto landed = [&](int i) -> bool { return wait(L::HFULL + i % (2 * L::NH_), (i / (2 * L::NH_)) & 1); };
  // a tile is released by the four warps that read it, or all eight
  auto release = [&](int st) {
    __syncwarp();
    if (lane == 0) mbar_arrive_n(bar(L::HEMPTY + st), step);
  };

  // Q's fragments
  uint32_t qa[STEPS][NARROW ? 2 : 4];
#pragma unroll
  for (int c = 0; c < QC; ++c) {
    const int d = DQ * q + 8 * c;
    const uint32_t at = sbase + L::Q_OFF + (d >> 6) * L::PANEL, ch = (d & 63) >> 3;
    const int ra = NARROW ? gr : r0;
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
    if (ra < rows) v0 = lds128(at + ra * 128 + ((ch ^ (ra & 7)) << 4));
    if constexpr (NARROW) {
      qa[2 * c][0] = v0.x, qa[2 * c][1] = v0.y, qa[2 * c + 1][0] = v0.z, qa[2 * c + 1][1] = v0.w;
    } else {
      if (ok1) v1 = lds128(at + r1 * 128 + ((ch ^ (r1 & 7)) << 4));
      qa[2 * c][0] = v0.x, qa[2 * c][2] = v0.y, qa[2 * c + 1][0] = v0.z, qa[2 * c + 1][2] = v0.w;
      qa[2 * c][1] = v1.x, qa[2 * c][3] = v1.y, qa[2 * c + 1][1] = v1.z, qa[2 * c + 1][3] = v1.w;
    }
  }
  float o[NO][4];
#pragma unroll
  for (int j = 0; j < NO; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  bool bad0 = false, bad1 = false;

  for (int kt = sg.t0 + first_tile; kt < sg.t1; kt += step) {
    const int k0 = kt * TILE, ki = 2 * (units + kt - sg.t0);
    const int ks = ki % L::NH_, vs = (ki + 1) % L::NH_;
    const uint32_t kbase = sbase + L::H_OFF + ks * L::LAND, vbase = sbase + L::H_OFF + vs * L::LAND;
    const bool fix = k0 + TILE > min(vis0, sg.len);
    if (!landed(ki)) return false;
    // ---- scores of 32 keys
    float s[NF][4];
    if constexpr (NARROW) {  // keys gr and gr + 8 of each 16, rows r0 and r1
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        const int kr = first_key + 16 * n + gr;
        if (!Q8) {
#pragma unroll
          for (int c = 0; c < QC; ++c) {
            const int d = DQ * q + 8 * c;
            const uint32_t at = kbase + (d >> 6) * L::PANEL + kr * 128 + ((((d & 63) >> 3) ^ gr) << 4);
            const uint4 v = lds128(at), u = lds128(at + 8 * 128);
            mma16816(s[n], v.x, u.x, v.y, u.y, qa[2 * c][0], qa[2 * c][1]);
            mma16816(s[n], v.z, u.z, v.w, u.w, qa[2 * c + 1][0], qa[2 * c + 1][1]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint32_t at = kbase + (D == 128 ? kr * 128 + (((2 * q + c) ^ gr) << 4)
                                                  : kr * 64 + ((q ^ ((kr >> 1) & 3)) << 4));
            const uint4 v = lds128(at), u = lds128(at + 8 * D);
            const uint32_t vw[4] = {v.x, v.y, v.z, v.w}, uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint2 a = expand4(vw[e], 0x7b807b80u), b = expand4(uw[e], 0x7b807b80u);
              mma16816(s[n], a.x, b.x, a.y, b.y, qa[4 * c + e][0], qa[4 * c + e][1]);
            }
          }
          const uint32_t at = sbase + L::SCALE_OFF + (ks * TILE + kr) * 4;
          const float sa = lds_float(at), sb = lds_float(at + 32);
          s[n][0] *= sa, s[n][1] *= sa, s[n][2] *= sb, s[n][3] *= sb;
        }
      }
    } else {  // keys 2q and 2q + 1 of each 8
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        const int kr = first_key + 8 * n + gr;
        if (!Q8) {
#pragma unroll
          for (int c = 0; c < QC; ++c) {
            const int d = DQ * q + 8 * c;
            const uint4 v = lds128(kbase + (d >> 6) * L::PANEL + kr * 128 + ((((d & 63) >> 3) ^ (kr & 7)) << 4));
            mma16816(s[n], qa[2 * c][0], qa[2 * c][1], qa[2 * c][2], qa[2 * c][3], v.x, v.y);
            mma16816(s[n], qa[2 * c + 1][0], qa[2 * c + 1][1], qa[2 * c + 1][2], qa[2 * c + 1][3], v.z, v.w);
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint32_t at = D == 128 ? kr * 128 + (((2 * q + c) ^ (kr & 7)) << 4)
                                         : kr * 64 + ((q ^ ((kr >> 1) & 3)) << 4);
            const uint4 v = lds128(kbase + at);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint2 b = expand4(w[e], 0x7b807b80u);
              const int st = 4 * c + e;
              mma16816(s[n], qa[st][0], qa[st][1], qa[st][2], qa[st][3], b.x, b.y);
            }
          }
          const float2 sc = lds_float2(sbase + L::SCALE_OFF + (ks * TILE + first_key + 8 * n + 2 * q) * 4);
          s[n][0] *= sc.x, s[n][1] *= sc.y, s[n][2] *= sc.x, s[n][3] *= sc.y;
        }
      }
    }
    release(ks);
    // ---- weights
    float x0, x1;
    if constexpr (NARROW) {
      if (fix) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int p = k0 + first_key + 16 * n + gr;
          if (p >= see0) s[n][0] = -INFINITY;
          if (p >= see1) s[n][1] = -INFINITY;
          if (p + 8 >= see0) s[n][2] = -INFINITY;
          if (p + 8 >= see1) s[n][3] = -INFINITY;
        }
      }
      x0 = max3(fmaxf(s[0][0], s[0][2]), s[1][0], s[1][2]);
      x1 = max3(fmaxf(s[0][1], s[0][3]), s[1][1], s[1][3]);
    } else {
      if (fix) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int p = k0 + first_key + 8 * n + 2 * q;
          if (p >= see0) s[n][0] = -INFINITY;
          if (p + 1 >= see0) s[n][1] = -INFINITY;
          if (p >= see1) s[n][2] = -INFINITY;
          if (p + 1 >= see1) s[n][3] = -INFINITY;
        }
      }
      x0 = max3(max3(s[0][0], s[0][1], s[1][0]), max3(s[1][1], s[2][0], s[2][1]), fmaxf(s[3][0], s[3][1]));
      x1 = max3(max3(s[0][2], s[0][3], s[1][2]), max3(s[1][3], s[2][2], s[2][3]), fmaxf(s[3][2], s[3][3]));
    }
    // a row's keys are spread over the lanes of a quad, or over the eight quads
#pragma unroll
    for (int w = NARROW ? 4 : 1; w <= (NARROW ? 16 : 2); w <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, w));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, w));
    }
    x0 = fmaxf(m0, x0);
    x1 = fmaxf(m1, x1);
    if (kt == sg.t0 + first_tile) {
      m0 = x0;
      m1 = x1;
    } else if (__any_sync(0xffffffffu, fmaxf(x0 - m0, x1 - m1) * g.scale_log2 > 8.f)) {
      const float f0 = x0 == m0 ? 1.f : ex2((m0 - x0) * g.scale_log2);
      const float f1 = x1 == m1 ? 1.f : ex2((m1 - x1) * g.scale_log2);
#pragma unroll
      for (int j = 0; j < NO; ++j)
        o[j][0] *= f0, o[j][1] *= NARROW ? f1 : f0, o[j][2] *= NARROW ? f0 : f1, o[j][3] *= f1;
      l0 *= f0;
      l1 *= f1;
      m0 = x0;
      m1 = x1;
    }
    const float n0 = m0 == -INFINITY ? 0.f : -m0 * g.scale_log2, n1 = m1 == -INFINITY ? 0.f : -m1 * g.scale_log2;
    if (!landed(ki + 1)) return false;
    uint32_t p[NF][2];  // weights as bf16 pairs: of fragment n, row r0 / r1, or (narrow) row gr
    if constexpr (NARROW) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float e0 = ex2(fmaf(s[n][0], g.scale_log2, n0)), e1 = ex2(fmaf(s[n][1], g.scale_log2, n1));
        float e2 = ex2(fmaf(s[n][2], g.scale_log2, n0)), e3 = ex2(fmaf(s[n][3], g.scale_log2, n1));
        l0 += e0 + e2;
        l1 += e1 + e3;
        if (Q8) {
          const uint32_t at = sbase + L::SCALE_OFF + (vs * TILE + first_key + 16 * n + gr) * 4;
          const float sa = lds_float(at), sb = lds_float(at + 32);
          e0 *= sa, e1 *= sa, e2 *= sb, e3 *= sb;
          if (fix) {  // a hidden key's scale may be anything
            const int pos = k0 + first_key + 16 * n + gr;
            if (pos >= see0) e0 = 0.f;
            if (pos >= see1) e1 = 0.f;
            if (pos + 8 >= see0) e2 = 0.f;
            if (pos + 8 >= see1) e3 = 0.f;
          }
        }
        p[n][0] = movmatrix_trans(pack_bf16x2(e0, e1));
        p[n][1] = movmatrix_trans(pack_bf16x2(e2, e3));
      }
    } else {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        float e0 = ex2(fmaf(s[n][0], g.scale_log2, n0)), e1 = ex2(fmaf(s[n][1], g.scale_log2, n0));
        float e2 = ex2(fmaf(s[n][2], g.scale_log2, n1)), e3 = ex2(fmaf(s[n][3], g.scale_log2, n1));
        l0 += e0 + e1;
        l1 += e2 + e3;
        if (Q8) {
          const float2 sc = lds_float2(sbase + L::SCALE_OFF + (vs * TILE + first_key + 8 * n + 2 * q) * 4);
          e0 *= sc.x, e1 *= sc.y, e2 *= sc.x, e3 *= sc.y;
          if (fix) {  // a hidden key's scale may be anything
            const int pos = k0 + first_key + 8 * n + 2 * q;
            if (pos >= see0) e0 = 0.f;
            if (pos + 1 >= see0) e1 = 0.f;
            if (pos >= see1) e2 = 0.f;
            if (pos + 1 >= see1) e3 = 0.f;
          }
        }
        p[n][0] = pack_bf16x2(e0, e1);
        p[n][1] = pack_bf16x2(e2, e3);
      }
    }
    if (!Q8 && fix) {
      // Values that must not reach a row through its zero weights (0 x NaN) are replaced by zeros in
      // this warp's 32 keys: all past the sequence's end, and the elements that are not finite of those
      // that some row does not see yet (rows that do see one take note).  An e4m3 code is always finite.
      constexpr int LANES = D / 8, RPI = 32 / LANES;  // 16-byte pieces of a row, rows at a time
      const int piece = lane % LANES, sub = lane / LANES;
      const int end = min(32, sg.len - k0 - first_key);  // this warp's rows before the sequence's end
      const uint32_t at = vbase + (piece >> 3) * L::PANEL + first_key * 128;
      uint32_t wipe = 0;  // the keys whose values are not all finite
#pragma unroll 1
      for (int rb = max(0, vis0 - k0 - first_key) / RPI * RPI; rb < end; rb += RPI) {
        const int rr = rb + sub;
        uint32_t acc = 0;
        if (k0 + first_key + rr >= vis0 && rr < end) {
          const uint4 v = lds128(at + rr * 128 + (((piece & 7) ^ (rr & 7)) << 4));
          acc = ptx::bf16x2_fma(v.x, 0u, 0u);
          acc = ptx::bf16x2_fma(v.y, 0u, acc);
          acc = ptx::bf16x2_fma(v.z, 0u, acc);
          acc = ptx::bf16x2_fma(v.w, 0u, acc);
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, (acc & 0x7fff7fffu) != 0);  // 0 x Inf, 0 x NaN: NaN
#pragma unroll
        for (int h = 0; h < RPI; ++h) {
          if (hit >> (h * LANES) & ((1u << LANES) - 1u)) {
            const int key = k0 + first_key + rb + h;
            wipe |= 1u << (rb + h);
            bad0 |= key < see0;
            bad1 |= key < see1;
          }
        }
      }
      // where two warps have the same keys, both have looked at them before either replaces any (then both
      // replace the same: it does not matter whose reads and writes come first)
      if (groups == 2 && !team()) return false;
#pragma unroll
      for (int rb = 0; rb < 32; rb += RPI) {
        const int rr = rb + sub;
        if (rr >= end) sts128(at + rr * 128 + (piece & 7) * 16, make_uint4(0, 0, 0, 0));
      }
      if (wipe) {
#pragma unroll 1
        for (int rr = sub; rr < end; rr += RPI) {
          const uint32_t place = at + rr * 128 + (((piece & 7) ^ (rr & 7)) << 4);
          if (wipe >> rr & 1) sts128(place, bf16x8_finite(lds128(place)));
        }
      }
      ptx::fence_proxy_async_smem();  // the copies overwrite what was written here
      __syncwarp();
    }
    // ---- O += P V
#pragma unroll
    for (int n = 0; n < NF; n += NF / 2) {
      const int kb = first_key + 32 / NF * n;
      if (!Q8) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const int row = kb + ((lane >> 3) & 1) * 8 + (lane & 7), ch = 2 * j + (lane >> 4);
          uint32_t v[4];
          ldmatrix_x4_trans(vbase + (ch >> 3) * L::PANEL + row * 128 + (((ch & 7) ^ (row & 7)) << 4), v);
          if constexpr (NARROW) {
            mma16816(o[j], v[0], v[2], v[1], v[3], p[n][0], p[n][1]);
          } else {
            mma16816(o[2 * j], p[n][0], p[n][1], p[n + 1][0], p[n + 1][1], v[0], v[1]);
            mma16816(o[2 * j + 1], p[n][0], p[n][1], p[n + 1][0], p[n + 1][1], v[2], v[3]);
          }
        }
      } else {
        uint32_t v[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = kb + 2 * q + (i & 1) + (i >> 1) * 8;
          if (D == 128) {
            const uint4 w = lds128(vbase + row * 128 + ((gr ^ (row & 7)) << 4));
            v[i][0] = w.x, v[i][1] = w.y, v[i][D / 32 - 2] = w.z, v[i][D / 32 - 1] = w.w;
          } else {
            const uint2 w = lds64(vbase + row * 64 + (((gr >> 1) ^ ((row >> 1) & 3)) << 4) + (gr & 1) * 8);
            v[i][0] = w.x, v[i][1] = w.y;
          }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const uint32_t a0 = expand_pair<0>(v[0][w], v[1][w]), a1 = expand_pair<1>(v[0][w], v[1][w]);
          const uint32_t a2 = expand_pair<2>(v[0][w], v[1][w]), a3 = expand_pair<3>(v[0][w], v[1][w]);
          const uint32_t b0 = expand_pair<0>(v[2][w], v[3][w]), b1 = expand_pair<1>(v[2][w], v[3][w]);
          const uint32_t b2 = expand_pair<2>(v[2][w], v[3][w]), b3 = expand_pair<3>(v[2][w], v[3][w]);
          if constexpr (NARROW) {
            mma16816(o[2 * w], a0, a1, b0, b1, p[n][0], p[n][1]);
            mma16816(o[2 * w + 1], a2, a3, b2, b3, p[n][0], p[n][1]);
          } else {
            mma16816(o[4 * w], p[n][0], p[n][1], p[n + 1][0], p[n + 1][1], a0, b0);
            mma16816(o[4 * w + 1], p[n][0], p[n][1], p[n + 1][0], p[n + 1][1], a1, b1);
            mma16816(o[4 * w + 2], p[n][0], p[n][1], p[n + 1][0], p[n + 1][1], a2, b2);
            mma16816(o[4 * w + 3], p[n][0], p[n][1], p[n + 1][0], p[n + 1][1], a3, b3);
          }
        }
      }
    }
    release(vs);
  }
#pragma unroll
  for (int w = NARROW ? 4 : 1; w <= (NARROW ? 16 : 2); w <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, w);
    l1 += __shfl_xor_sync(0xffffffffu, l1, w);
  }
  // ---- the warps' results joined by way of the query tiles' memory, a region of 16 rows per warp
  float* s_m = reinterpret_cast<float*>(x.smem + L::ML_OFF);
  float* s_l = s_m + 128;
  uint8_t* s_b = x.smem + L::ML_OFF + 8 * TILE;
  float* region = reinterpret_cast<float*>(x.smem + L::Q_OFF);
  // column of o[j][0]: bf16 fragments are natural, e4m3's column 2q of step j is d = j + (D/8) 2q (narrow:
  // row gr of step pair j is d = 2 j + (D/8) gr); its place in the region is swizzled so that a warp's 32
  // stores go to 32 banks
  auto place = [](int row, int col) {
    if constexpr (NARROW)
      return row * D + (Q8 ? col ^ ((col >> 5 & 3) << 2) ^ (row >> 1 & 3) : col ^ ((row >> 1 & 3) << 3));
    else
      return row * D + (Q8 ? col ^ ((col >> 5 & 3) << 3) ^ (row & 7) : col ^ ((row & 3) << 3) ^ (row >> 2 & 1));
  };
  auto at = [&](int j, int e) {
    if constexpr (NARROW)
      return place(r0 + (e & 1), Q8 ? 2 * j + (e >> 1) + NT * gr : 16 * j + gr + 8 * (e >> 1));
    else
      return place(gr + (e >> 1) * 8, Q8 ? j + NT * (2 * q + (e & 1)) : 8 * j + 2 * q + (e & 1));
  };
  // every warp has read its query rows (the first barrier), then their memory is written (the second)
  if (!team()) return false;
  float* mine = region + x.warp * 16 * D;
#pragma unroll
  for (int j = 0; j < NO; ++j) {
    mine[at(j, 0)] = o[j][0];
    mine[at(j, 1)] = o[j][1];
  }
  if (NARROW || rows > 8) {
#pragma unroll
    for (int j = 0; j < NO; ++j) {
      mine[at(j, 2)] = o[j][2];
      mine[at(j, 3)] = o[j][3];
    }
  }
  if (NARROW ? gr == 0 : q == 0) {
    const int a0 = x.warp * 16 + (r0 & 15), a1 = x.warp * 16 + (r1 & 15);
    s_m[a0] = m0 == -INFINITY ? m0 : m0 * g.scale_log2;
    s_m[a1] = m1 == -INFINITY ? m1 : m1 * g.scale_log2;
    s_l[a0] = l0;
    s_l[a1] = l1;
    s_b[a0] = bad0;
    s_b[a1] = bad1;
  }
  if (!team()) return false;
  const bool whole = sg.t0 == 0 && sg.t1 == sg.nt;
  float* slot = g.part + (2ll * cta + (sg.t0 == 0 ? 1 : 0)) * slot_floats<D>();
  // lanes: columns 2 lane, 2 lane + 1 and (D = 128) those 64 further
  for (int r = x.warp; r < rows; r += 8) {
    const int w0 = r >> 4 << 2, n = groups == 1 ? 8 : 4;  // the warps that have this row
    float ml = -INFINITY, l = 0.f;
    bool bad = false;
    for (int w = w0; w < w0 + n; ++w) ml = fmaxf(ml, s_m[w * 16 + (r & 15)]);
    const float top = ml == -INFINITY ? 0.f : ml;
    float2 y[NT / 8];
#pragma unroll
    for (int j = 0; j < NT / 8; ++j) y[j] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int w = w0; w < w0 + n; ++w) {
      const float f = ex2(s_m[w * 16 + (r & 15)] - top);
      l = fmaf(s_l[w * 16 + (r & 15)], f, l);
      bad |= s_b[w * 16 + (r & 15)] != 0;
#pragma unroll
      for (int j = 0; j < NT / 8; ++j) {
        y[j].x = fmaf(region[w * 16 * D + place(r & 15, 64 * j + 2 * lane)], f, y[j].x);
        y[j].y = fmaf(region[w * 16 * D + place(r & 15, 64 * j + 2 * lane + 1)], f, y[j].y);
      }
    }
    const int tok = r / g.group;
    if (!Q8 && bad) {
      // elements that are not finite and that this row sees enter the sums as they are
      for (int p = max(vis0, sg.t0 * TILE); p < min(vis0 + tok, sg.t1 * TILE); ++p) {
        const int page = find_page(a, sg.b, p);
        if (page < 0) continue;
        const size_t row = (static_cast<size_t>(page) * a.heads + sg.h) * a.page_size + p % a.page_size;
#pragma unroll
        for (int j = 0; j < NT / 8; ++j) {
          const uint32_t v = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.v) + row * D + 64 * j + 2 * lane);
          const float lo = __uint_as_float(v << 16), hi = __uint_as_float(v & 0xffff0000u);
          if (!(fabsf(lo) < INFINITY)) y[j].x += lo;
          if (!(fabsf(hi) < INFINITY)) y[j].y += hi;
        }
      }
    }
    if (whole) {
      const float inv = l == 0.f ? 0.f : 1.0f / l;  // no key seen: zero
      const long long row = static_cast<long long>(sg.row0 + sg.i0 + tok) * g.q_heads + sg.h * g.group + r - tok * g.group;
#pragma unroll
      for (int j = 0; j < NT / 8; ++j)
        *reinterpret_cast<uint32_t*>(g.out + row * D + 64 * j + 2 * lane) = pack_bf16x2(y[j].x * inv, y[j].y * inv);
      if (g.lse && lane == 0) g.lse[row] = l == 0.f ? -INFINITY : (ml + log2f(l)) * 0.69314718055994531f;
    } else {
#pragma unroll
      for (int j = 0; j < NT / 8; ++j) *reinterpret_cast<float2*>(slot + r * D + 64 * j + 2 * lane) = y[j];
      if (lane == 0) {
        slot[2 * TILE * D + r] = ml;
        slot[2 * TILE * (D + 1) + r] = l;
      }
    }
  }
  __syncwarp();
  if (lane == 0) {
    ptx::mbar_arrive(bar(L::QEMPTY));
    ptx::mbar_arrive(bar(L::QEMPTY + 1));
  }
  return true;
}

}  // namespace kv
}  // namespace moe
