// Shared by the two forms of the attention over the paged cache: the tile form
// (moe_kv_attn.cu) and the thin one (moe_kv_thin.cuh), which run in one kernel.
#pragma once
#include "moe_kv_plan.cuh"
#include "moe_ptx.cuh"
#include "moe_tc_dev.cuh"

namespace moe {
namespace kv {

struct AttnArgs {
  const uint16_t* q;
  long long q_token, q_head;
  uint16_t* out;
  float* lse;
  int4* joins;  // workspace: per CTA, the item that its last part begins (parts, first row, tokens, KV head)
  float* part;  // and two slots for parts of items
  float scale_log2;
  int q_heads, group, tpt;  // tpt: tokens per query tile
  int tokens;               // per item: of a pair of tiles, or of one
  int merge;                // what cutting items costs, in key tiles
  int chunk, chunk_log;     // rows of one copy (a power of two), divides page_size and TILE
  int per_page;             // copies of a page
  unsigned long long wait_cycles;
  bool poll;  // the limit is too short for waits inside an instruction
};

// A partial result: raw output [256][D], then its rows' maximum (times scale_log2) and sum.
template <int D>
__host__ __device__ constexpr int slot_floats() {
  return 2 * TILE * (D + 2);
}

constexpr int SEGS = 4;  // work segments published ahead

template <int D, bool Q8>
struct Layout {
  static constexpr int THREADS = Q8 ? 512 : 384;
  static constexpr int NH = D / 64;                // 64-wide swizzled panels of a row
  static constexpr int PANEL = TILE * 128;         // bytes of one panel of a tile
  static constexpr int TB = NH * PANEL;            // one bf16 tile of 128 rows
  static constexpr int NS = Q8 ? 3 : (D == 128 ? 5 : 10);  // bf16 key/value tiles in the ring
  static constexpr int NR = Q8 ? (D == 128 ? 3 : 8) : 0;  // e4m3 tiles in front of it
  static constexpr int LAND = Q8 ? TILE * D : TB;  // bytes of a tile as copied
  // The rings that copies land in.  bf16: one.  e4m3: the tile form's (L) in front of its bf16 ring, and the
  // thin form's (H), which takes the memory of both: a segment of the other form starts when the last one's
  // tiles are done with.
  static constexpr int NL = Q8 ? NR : NS;
  static constexpr int NH_ = Q8 ? NS * TB / LAND + NR : NS;
  static constexpr int Q_OFF = 0;
  static constexpr int KV_OFF = 2 * TB;
  static constexpr int RAW_OFF = KV_OFF + NS * TB;
  static constexpr int L_OFF = Q8 ? RAW_OFF : KV_OFF;
  static constexpr int H_OFF = KV_OFF;
  static constexpr int SCALE_OFF = RAW_OFF + NR * LAND;  // TILE scales per landed e4m3 tile
  static constexpr int BAR_OFF = SCALE_OFF + (Q8 ? NH_ * TILE * 4 : 0);
  // Barriers.  LFULL / LEMPTY, HFULL / HEMPTY: the rings that copies land in (the same when there is one);
  // FULL / EMPTY: the e4m3 form's bf16 ring.  A wait by parity is only right if its thread cannot fall two
  // phases behind or get ahead of the phase before it, so
  //  - tile i of a landing ring completes FULL[i % (2 N)], twice as many barriers as slots: a team of the
  //    thin form that waits for tile i skipped the tiles of the other team, but released tile i - 3 or a
  //    later one of its own, whose slot was filled after tile i - 2 N had landed (N >= 3);
  //  - whoever waits for QFULL[0] (the MMA warp and the softmax warps) does so for every segment, and
  //    QEMPTY[0] needs all of them; QFULL[0] needs both loading warps, who wait for every QEMPTY[0].
  static constexpr int LFULL = 0, LEMPTY = LFULL + 2 * NL, HFULL = Q8 ? LEMPTY + NL : LFULL,
                       HEMPTY = Q8 ? HFULL + 2 * NH_ : LEMPTY, FULL = HEMPTY + NH_, EMPTY = FULL + (Q8 ? NS : 0),
                       SFULL = EMPTY + (Q8 ? NS : 0), PREADY = SFULL + 2, QFULL = PREADY + 2, QEMPTY = QFULL + 2,
                       OFULL = QEMPTY + 2, FIX = OFULL + 2, ML = FIX + 2, OBFREE = ML + 1, TEAM = OBFREE + 1,
                       TCDONE = TEAM + 1, SEGF = TCDONE + 1, SEGE = SEGF + SEGS, DRAIN = SEGE + SEGS, NBAR = DRAIN + 1;
  // arrivals that complete a phase of barrier i
  static __device__ __forceinline__ int arrivals(int i) {
    if (i < LEMPTY) return 1;
    if (i < LEMPTY + NL) return Q8 ? 4 : 8;
    if (Q8 && i < HEMPTY) return 1;
    if (i < FULL) return 8;
    if (i < EMPTY) return 4;
    if (i < SFULL) return 1;
    if (i >= PREADY && i < QFULL) return 4;
    if (i == QFULL) return 2;
    if (i >= QEMPTY && i < OFULL) return i == QEMPTY ? 9 : 8;
    if (i >= FIX && i < TEAM) return 4;
    if (i == TEAM) return 8;
    if (i >= SEGE && i < DRAIN) return THREADS / 32 - 1;
    return 1;
  }
  static constexpr int MISC_OFF = BAR_OFF + 8 * NBAR;       // TMEM address, abort flag, bad-row masks
  static constexpr int SEG_OFF = (MISC_OFF + 48 + 15) / 16 * 16;  // SEGS segments of 48 bytes
  static constexpr int ML_OFF = SEG_OFF + 48 * SEGS;        // row maxima and sums (2 x 128 floats), flags (128 bytes)
  static constexpr int BYTES = ML_OFF + 9 * TILE + 1024;    // + alignment
  // registers per thread: 128 (Q8) or 168 at launch, moved to the two softmax warpgroups
  static constexpr int REGS_SOFTMAX = Q8 ? 176 : 208, REGS_ISSUE = Q8 ? 96 : 88, REGS_EXPAND = Q8 ? 64 : 0;
  static_assert(256 * REGS_SOFTMAX + 128 * (REGS_ISSUE + REGS_EXPAND) <= THREADS * (Q8 ? 128 : 168), "register split");
  static_assert(BYTES <= 232448, "shared memory of one CTA");
};

constexpr int TM_S = 0, TM_O = 256;  // TMEM columns: S a, S b (128 each), O a, O b (D each)

// Instruction descriptor of P V: D fp32, A and B bf16, A (P) K-major, B (V, rows of d per key) MN-major.
__device__ __forceinline__ uint32_t idesc_pv(int N) { return ptx::idesc_bf16_f32(TILE, N) | (1u << 16); }

// Descriptor of an MN-major operand in 128-byte swizzled atoms of 8 keys x 64 columns: the next 8 keys
// 1024 bytes on, the next 64 columns one panel on.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t panel) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(panel >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// O += P V: eight K16 steps, P columns 8 and V keys 16 (2048 bytes) further per step; the first step keeps
// O only if `accumulate` is non-zero.
__device__ __forceinline__ void mma_pv_elect(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\t.reg .b32 x1, x2, x3, x4, x5, x6, x7;\n\t"
      ".reg .b64 c1, c2, c3, c4, c5, c6, c7;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %3, 0;\n\t"
      "add.u32 x1, %1, 8;\n\tadd.u32 x2, %1, 16;\n\tadd.u32 x3, %1, 24;\n\tadd.u32 x4, %1, 32;\n\t"
      "add.u32 x5, %1, 40;\n\tadd.u32 x6, %1, 48;\n\tadd.u32 x7, %1, 56;\n\t"
      "add.s64 c1, %2, 128;\n\tadd.s64 c2, %2, 256;\n\tadd.s64 c3, %2, 384;\n\tadd.s64 c4, %2, 512;\n\t"
      "add.s64 c5, %2, 640;\n\tadd.s64 c6, %2, 768;\n\tadd.s64 c7, %2, 896;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x1], c1, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x2], c2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x3], c3, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x4], c4, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x5], c5, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x6], c6, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x7], c7, %3, q;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// S = Q K^T for d = 128: eight K16 steps over two panels (1024 descriptor units apart).
__device__ __forceinline__ void mma_qk2_elect(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\t.reg .b64 a1, a2, a3, a4, a5, a6, a7, c1, c2, c3, c4, c5, c6, c7;\n\t"
      "setp.eq.b32 p, %3, 0;\n\t"
      "setp.ne.b32 q, %3, 0;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\tadd.s64 a4, %1, 1024;\n\t"
      "add.s64 a5, %1, 1026;\n\tadd.s64 a6, %1, 1028;\n\tadd.s64 a7, %1, 1030;\n\t"
      "add.s64 c1, %2, 2;\n\tadd.s64 c2, %2, 4;\n\tadd.s64 c3, %2, 6;\n\tadd.s64 c4, %2, 1024;\n\t"
      "add.s64 c5, %2, 1026;\n\tadd.s64 c6, %2, 1028;\n\tadd.s64 c7, %2, 1030;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, c1, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, c2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, c3, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a4, c4, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a5, c5, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a6, c6, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a7, c7, %3, q;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ float2 unpack2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 16 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// A value that all lanes hold, or one lane (the others 0), as a warp-uniform one: what the copy and MMA
// instructions take without going lane by lane.
__device__ __forceinline__ int uniform(int x) {
  return static_cast<int>(__reduce_or_sync(0xffffffffu, static_cast<uint32_t>(x)));
}

// Bounded wait of a whole warp on phase `parity` of `bar`; false when it gave up (recorded) or another role
// has.  The waiting is done by try_wait with its own time limit, which wakes sooner than one that is told to
// sleep for longer (4096 tokens over 32K, 832 us with that, 798 without): the barriers here are handed over
// every thousand cycles.
__device__ __forceinline__ bool wait_warp_untraced(uint32_t bar, uint32_t parity, volatile int* s_abort, int* err,
                                                   const AttnArgs& g) {
  if (__all_sync(0xffffffffu, g.poll ? ptx::mbar_test_wait(bar, parity) : ptx::mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  for (;;) {
    if (__all_sync(0xffffffffu, g.poll ? ptx::mbar_test_wait(bar, parity) : ptx::mbar_try_wait(bar, parity)))
      return true;
    int give_up = *s_abort;
    if (!give_up && static_cast<unsigned long long>(clock64() - t0) > g.wait_cycles) give_up = 2;
    give_up = __shfl_sync(0xffffffffu, give_up, 0);
    if (give_up) {
      if (give_up == 2 && (threadIdx.x & 31) == 0) {
        set_device_error(err, MOE_DEV_TIMEOUT);
        *s_abort = 1;
      }
      return false;
    }
  }
}

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* s_abort, int* err,
                                          const AttnArgs& g) {
#ifdef MOE_TRACE
  const long long t0 = clock64();
  const bool r = wait_warp_untraced(bar, parity, s_abort, err, g);
  tc_dev::trace_wait(err, t0, clock64());
  return r;
#else
  return wait_warp_untraced(bar, parity, s_abort, err, g);
#endif
}

// Arrive n times.
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

}  // namespace kv
}  // namespace moe
