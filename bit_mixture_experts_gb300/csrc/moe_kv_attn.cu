// Causal attention of new tokens over a paged key/value cache on the tensor
// cores, GQA: o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m), s_j = scale q.k_j.
//
// One pass over the keys with a running maximum and sum per query row.  Query
// rows are packed per KV head (moe_kv_plan.cuh), so a key is read once for its
// whole head group; a work item is a pair of 128-row tiles against a run of
// 128-key tiles, and one persistent CTA per SM takes an even share of all key
// tiles of the call.  An item cut between CTAs leaves partial sums in the
// workspace, which kv_merge_kernel joins.
//
// Per key tile and query tile: S = Q K^T (tcgen05, FP32 in TMEM), one thread
// per row reads its 128 scores, takes the maximum, writes P = exp2(S - m) as
// bf16 over S in TMEM, and O += P V (tcgen05, P from TMEM, FP32 in TMEM).  While
// one tile's threads are at its softmax, the tensor core works for the other:
// PV a, QK a (next key tile), PV b, QK b, ...  O is rescaled only when the
// maximum has grown by more than 2^8 since the last time (P then stays below
// 2^8, which bf16 holds as accurately as numbers below one): rare after the
// first tiles, and it saves a pass over O per key tile.
//
// Roles (warps): 0 copies keys and values (TMA boxes of up to 128 rows of a
// page into 128-byte swizzled tiles), 1 issues the MMAs, 2 and 3 load the two
// query tiles, 4-7 and 8-11 the softmax of the pair's tiles.  With an e4m3
// cache warps 12-15 expand the tiles to bf16: e4m3 times a power of two is
// exact in bf16, so everything after that is the same as for a bf16 cache, to
// the bit.  Every wait is bounded (MOE_DEV_TIMEOUT).
//
// Roundings: P to bf16 (the tensor core's operand; sums are taken of the
// unrounded values), the output to bf16.  All else is FP32.
#include <cuda.h>
#include <string.h>

#include "moe_common.cuh"
#include "moe_kv_plan.cuh"
#include "moe_ptx.cuh"
#include "moe_tc_dev.cuh"
#include "moe_tmap.cuh"

namespace moe {

namespace {

using kv::TILE;

struct AttnArgs {
  const uint16_t* q;
  long long q_token, q_head;
  uint16_t* out;
  float* lse;
  float* part;  // workspace: two slots per CTA
  float scale_log2;
  int q_heads, group, tpt, chunk;  // chunk: rows of one copy, divides page_size and TILE
  unsigned long long wait_cycles;
  uint32_t sleep_ns;
};

// A partial result: raw output [256][D], then its rows' maximum (times scale_log2) and sum.
template <int D>
__host__ __device__ constexpr int slot_floats() {
  return 2 * TILE * (D + 2);
}

template <int D, bool Q8>
struct Layout {
  static constexpr int NH = D / 64;                // 64-wide swizzled panels of a row
  static constexpr int PANEL = TILE * 128;         // bytes of one panel of a tile
  static constexpr int TB = NH * PANEL;            // one bf16 tile of 128 rows
  static constexpr int NS = Q8 ? 3 : (D == 128 ? 5 : 10);  // bf16 key/value tiles in the ring
  static constexpr int RAW = TILE * D + TILE * 4;  // one e4m3 tile and its scales
  static constexpr int NR = Q8 ? (D == 128 ? 3 : 8) : 0;
  static constexpr int Q_OFF = 0;
  static constexpr int KV_OFF = 2 * TB;
  static constexpr int RAW_OFF = KV_OFF + NS * TB;
  static constexpr int BAR_OFF = RAW_OFF + NR * RAW;
  // barriers
  static constexpr int FULL = 0, EMPTY = FULL + NS, RFULL = EMPTY + NS, REMPTY = RFULL + NR, SFULL = REMPTY + NR,
                       PREADY = SFULL + 2, QFULL = PREADY + 2, QEMPTY = QFULL + 2, OFULL = QEMPTY + 2,
                       FIX = OFULL + 2, DRAIN = FIX + 2, NBAR = DRAIN + 1;
  static constexpr int MISC_OFF = BAR_OFF + 8 * NBAR;  // TMEM address, abort flag, bad-row masks
  static constexpr int BYTES = MISC_OFF + 64 + 1024;   // + alignment
  static constexpr int THREADS = Q8 ? 512 : 384;
  // registers per thread: 128 (Q8) or 168 at launch, moved to the two softmax warpgroups
  static constexpr int REGS_SOFTMAX = Q8 ? 176 : 208, REGS_OTHER = Q8 ? 80 : 88;
  static_assert(256 * REGS_SOFTMAX + (THREADS - 256) * REGS_OTHER <= THREADS * (Q8 ? 128 : 168), "register split");
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

// Two K16 steps of O += P V: P columns a, a + 8; V keys 16 further (2048 bytes) per step.
__device__ __forceinline__ void mma_pv2_elect(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\t.reg .b32 x;\n\t.reg .b64 c;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %3, 0;\n\t"
      "add.u32 x, %1, 8;\n\t"
      "add.s64 c, %2, 128;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], c, %3, q;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
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

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
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

// Four e4m3 codes -> four bf16 values, times s1 and s2 (bf16 pairs; s1 holds 2^120 times the scale as
// far as bf16 goes, s2 the rest).  The code's bits s eeee mmm become s 0000eeee mmm0000, a bf16 that is
// 2^-120 of the code's value (its subnormals are bf16 subnormals); the products are exact short of
// bf16's own underflow and overflow.
__device__ __forceinline__ uint2 expand4(uint32_t x, uint32_t s1, uint32_t s2) {
  // bytes sign-extended to 16 bits (prmt's sign mode), then moved up by 4: the sign's copies that land
  // on the exponent's upper bits are masked away
  uint32_t a, b;
  asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(a) : "r"(x));
  asm("prmt.b32 %0, %1, 0, 0xB3A2;" : "=r"(b) : "r"(x));
  a = (a << 4) & 0x87f087f0u;
  b = (b << 4) & 0x87f087f0u;
  return make_uint2(bf16x2_mul(bf16x2_mul(a, s1), s2), bf16x2_mul(bf16x2_mul(b, s1), s2));
}

template <int D, bool Q8>
__global__ void __launch_bounds__(Layout<D, Q8>::THREADS, 1)
    kv_attention_kernel(const kv::Args a, const AttnArgs g, const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_v) {
  using L = Layout<D, Q8>;
  constexpr int NH = L::NH, PANEL = L::PANEL, TB = L::TB, NS = L::NS, NR = L::NR;
  extern __shared__ uint8_t kv_smem_raw[];
  const uint32_t raw = ptx::smem_u32(kv_smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = kv_smem_raw + (sbase - raw);
  auto bar = [sbase](int i) -> uint32_t { return sbase + L::BAR_OFF + 8u * static_cast<uint32_t>(i); };
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + L::MISC_OFF + 4);
  volatile uint32_t* s_bad = reinterpret_cast<volatile uint32_t*>(smem + L::MISC_OFF + 16);  // [2][4]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tp = 2 * g.tpt;
  const int cta = static_cast<int>(blockIdx.x);

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      ptx::mbar_init(bar(L::FULL + i), Q8 ? 4 : 1);
      ptx::mbar_init(bar(L::EMPTY + i), 1);
    }
    for (int i = 0; i < NR; ++i) {
      ptx::mbar_init(bar(L::RFULL + i), 1);
      ptx::mbar_init(bar(L::REMPTY + i), 4);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(bar(L::SFULL + t), 1);
      ptx::mbar_init(bar(L::PREADY + t), 4);
      ptx::mbar_init(bar(L::QFULL + t), 1);
      ptx::mbar_init(bar(L::QEMPTY + t), 1);
      ptx::mbar_init(bar(L::OFULL + t), 1);
      ptx::mbar_init(bar(L::FIX + t), 4);
    }
    ptx::mbar_init(bar(L::DRAIN), 1);
    *s_abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(s_tmem), 512);
    ptx::tmem_relinquish();
  }
  // this CTA's share of the units (the scan's scratch lies where the key/value ring will be)
  long long* scratch = reinterpret_cast<long long*>(smem + L::KV_OFF);
  kv::Start* start = reinterpret_cast<kv::Start*>(scratch + 32);
  kv::Share share;
  const long long total = kv::locate<L::THREADS>(a, tp, scratch, start, [&](long long w) -> long long {
    share.total = w;
    share.ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), w));
    return cta < share.ctas ? share.lo(cta) : -1;
  });
  const kv::Start from = *start;
  ptx::fence_proxy_async_smem();  // the scratch is overwritten by copies
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const bool work = total > 0 && cta < share.ctas;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  kv::Walk walk(a, tp, work ? share.lo(cta) : 0, work ? share.lo(cta + 1) : 0, from.b, from.b_lo);
  kv::Seg sg;

  auto wait = [&](int i, uint32_t parity) -> bool {
    return tc_dev::wait_warp(bar(i), parity, s_abort, a.err, g.wait_cycles, g.sleep_ns);
  };

  if (warp < 4) {
    reg_dec<L::REGS_OTHER>();
    if (warp == 0) {
      // ---------------------------------------------- copies: K and V of every key tile, in that order
      const int ring = Q8 ? NR : NS;
      const int full = Q8 ? L::RFULL : L::FULL, empty = Q8 ? L::REMPTY : L::EMPTY;
      const int per_page = a.page_size / g.chunk, per_tile = TILE / g.chunk;
      int n = 0, st = 0, ph = 0;  // tiles issued; ring slot and its round's parity
      bool ok = true;
      while (ok && walk.next(sg)) {
        const int32_t* table = a.page_table + static_cast<size_t>(sg.b) * a.table_width;
        const int last = ceil_div(sg.s.len, g.chunk);  // chunks of the sequence
        int c0 = sg.t0 * per_tile;
        // page ids of chunks c0 .. c0 + 31 and the 32 after them, one per lane
        int ids = c0 + lane < last ? __ldg(table + (c0 + lane) / per_page) : 0;
        int ids2 = c0 + 32 + lane < last ? __ldg(table + (c0 + 32 + lane) / per_page) : 0;
        for (int kt = sg.t0; ok && kt < sg.t1; ++kt) {
          const int c = kt * per_tile;
          if (c - c0 >= 32) {
            c0 += 32;
            ids = ids2;
            ids2 = c0 + 32 + lane < last ? __ldg(table + (c0 + 32 + lane) / per_page) : 0;
          }
          const int have = max(0, min(per_tile, last - c));
          int page = ids;
          if (page < 0 || page >= a.num_pages) {
            if (c0 + lane < last) set_device_error(a.err, MOE_DEV_BAD_INDEX);
            page = 0;
          }
#pragma unroll 1
          for (int kind = 0; kind < 2; ++kind) {
            if (n >= ring && !wait(empty + st, ph ^ 1)) {
              ok = false;
              break;
            }
            const uint32_t f = bar(full + st);
            if (!Q8) {
              const uint32_t dst = sbase + L::KV_OFF + st * TB;
              ptx::mbar_arrive_expect_tx_elect(f, static_cast<uint32_t>(have * g.chunk * D * 2));
#pragma unroll 1
              for (int j = 0; j < have; ++j) {
                const int pg = __shfl_sync(0xffffffffu, page, c - c0 + j);
                const int row = (pg * a.heads + sg.h) * a.page_size + (c + j) % per_page * g.chunk;
#pragma unroll
                for (int hf = 0; hf < NH; ++hf)
                  ptx::tma_load_2d_elect(dst + hf * PANEL + j * g.chunk * 128, kind ? &tmap_v : &tmap_k, hf * 64, row, f);
              }
            } else {
              const uint32_t dst = sbase + L::RAW_OFF + st * L::RAW;
              const uint8_t* pool = static_cast<const uint8_t*>(kind ? a.v : a.k);
              const float* scale = kind ? a.v_scale : a.k_scale;
              ptx::mbar_arrive_expect_tx_elect(f, static_cast<uint32_t>(have * g.chunk * (D + 4)));
#pragma unroll 1
              for (int j = 0; j < have; ++j) {
                const int pg = __shfl_sync(0xffffffffu, page, c - c0 + j);
                const size_t row =
                    (static_cast<size_t>(pg) * a.heads + sg.h) * a.page_size + (c + j) % per_page * g.chunk;
                ptx::bulk_g2s_elect(dst + j * g.chunk * D, pool + row * D, g.chunk * D, f);
                ptx::bulk_g2s_elect(dst + TILE * D + j * g.chunk * 4, scale + row, g.chunk * 4, f);
              }
            }
            ++n;
            if (++st == ring) {
              st = 0;
              ph ^= 1;
            }
          }
        }
      }
      // every copy issued has landed before the CTA ends (at once unless a wait gave up)
      for (int i = n > ring ? n - ring : 0; i < n; ++i) tc_dev::wait_drain(bar(full + i % ring), (i / ring) & 1, 0);
    } else if (warp == 1) {
      // ---------------------------------------------- MMA issue, one unit behind for P V
      const uint32_t id_s = ptx::idesc_bf16_f32(TILE, TILE), id_o = idesc_pv(D);
      uint32_t p_ph[2] = {0, 0}, q_ph[2] = {0, 0};
      int kst = 0, kph = 0;  // ring slot of the current unit's K
      bool ok = true, prev = false, prev_b = false, prev_last = false, prev_first = false;
      int pst = 0;  // ring slot of the previous unit's V
      int pph = 0;
      auto pv = [&](int t) {
        const uint32_t o = tmem + TM_O + t * D, p = tmem + TM_S + t * TILE;
        const uint64_t d = desc_mn_sw128(sbase + L::KV_OFF + pst * TB, PANEL);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_pv2_elect(o, p + 16 * j, d + 256 * j, id_o, (j > 0 || !prev_first) ? 1u : 0u);
        if (prev_last) ptx::mma_commit_elect(bar(L::OFULL + t));
      };
      // O += P V of the previous unit for tile t
      auto finish = [&](int t) -> bool {
        if (t == 0 && !wait(L::FULL + pst, pph)) return false;
        if (!wait(L::PREADY + t, p_ph[t])) return false;
        p_ph[t] ^= 1;
        ptx::tc_fence_after();
        pv(t);
        return true;
      };
      while (ok && walk.next(sg)) {
        const bool has_b = sg.ntok > g.tpt;
        for (int kt = sg.t0; ok && kt < sg.t1; ++kt) {
          int vst = kst + 1, vph = kph;
          if (vst == NS) {
            vst = 0;
            vph ^= 1;
          }
          for (int t = 0; ok && t < 2; ++t) {
            if (prev && (t == 0 || prev_b)) {
              ok = finish(t);
              if (!ok) break;
            }
            if (prev && t == (prev_b ? 1 : 0)) ptx::mma_commit_elect(bar(L::EMPTY + pst));
            if (t == 0 || has_b) {
              if (kt == sg.t0) {
                ok = wait(L::QFULL + t, q_ph[t]);
                q_ph[t] ^= 1;
              }
              if (ok && t == 0) ok = wait(L::FULL + kst, kph);
              if (!ok) break;
              ptx::tc_fence_after();
              const uint64_t dq = ptx::smem_desc_sw128(sbase + L::Q_OFF + t * TB);
              const uint64_t dk = ptx::smem_desc_sw128(sbase + L::KV_OFF + kst * TB);
#pragma unroll
              for (int hf = 0; hf < NH; ++hf)
                ptx::mma_group_ss_elect(tmem + TM_S + t * TILE, dq + hf * (PANEL >> 4), dk + hf * (PANEL >> 4), id_s,
                                        hf ? 1u : 0u);
              ptx::mma_commit_elect(bar(L::SFULL + t));
              if (kt + 1 == sg.t1) ptx::mma_commit_elect(bar(L::QEMPTY + t));
              if (t == (has_b ? 1 : 0)) ptx::mma_commit_elect(bar(L::EMPTY + kst));
            }
          }
          prev = true;
          prev_b = has_b;
          prev_first = kt == sg.t0;
          prev_last = kt + 1 == sg.t1;
          pst = vst;
          pph = vph;
          kst = vst + 1;
          kph = vph;
          if (kst == NS) {
            kst = 0;
            kph ^= 1;
          }
        }
      }
      if (ok && prev) {
        ok = finish(0);
        if (ok && prev_b) finish(1);
      }
      // all MMAs are done before the tensor memory is released
      ptx::mma_commit_elect(bar(L::DRAIN));
      tc_dev::wait_drain(bar(L::DRAIN), 0, 0);
    } else {
      // ---------------------------------------------- query tile t of every item
      const int t = warp - 2;
      const uint32_t dst = sbase + L::Q_OFF + t * TB;
      uint32_t ph = 0;
      bool first = true;
      constexpr int C = D / 8;
      while (walk.next(sg)) {
        const int tok0 = t * g.tpt, ntok = min(g.tpt, sg.ntok - tok0);
        if (ntok <= 0) continue;
        if (!first) {
          if (!wait(L::QEMPTY + t, ph)) break;
          ph ^= 1;
        }
        first = false;
        const int rows = ntok * g.group;
        const uint16_t* src = g.q + static_cast<long long>(sg.s.row0 + sg.i0 + tok0) * g.q_token +
                              static_cast<long long>(sg.h) * g.group * g.q_head;
#pragma unroll 4
        for (int i = lane; i < rows * C; i += 32) {
          const int r = i / C, c = i % C;
          const int tok = r / g.group, hd = r - tok * g.group;
          ptx::cp_async_16(dst + (c >> 3) * PANEL + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                           src + tok * g.q_token + hd * g.q_head + c * 8);
        }
        ptx::cp_async_wait_all();
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(L::QFULL + t));
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------ softmax of tile t: one row per thread
    reg_inc<L::REGS_SOFTMAX>();
    const int t = (warp - 4) >> 2, w = warp & 3;
    const int r = 32 * w + lane;
    const int tok = r / g.group, hd = r - tok * g.group;
    const uint32_t lanes = static_cast<uint32_t>(32 * w) << 16;
    const uint32_t ts = tmem + lanes + TM_S + t * TILE, to = tmem + lanes + TM_O + t * D;
    uint32_t s_ph = 0, o_ph = 0;
    int n = 0;  // units before the current one
    bool ok = true;
    while (ok && walk.next(sg)) {
      const int i = t * g.tpt + tok;
      if (t == 1 && sg.ntok <= g.tpt) {
        n += sg.t1 - sg.t0;
        continue;
      }
      const bool valid = tok < g.tpt && i < sg.ntok;
      const bool active = __any_sync(0xffffffffu, valid);
      const int base = sg.s.len - sg.s.n + sg.i0;
      const int vis = base + i + 1;     // keys that this row sees: 0 .. vis - 1
      const int vis0 = base + 1;        // keys that all rows of the pair see
      float m = -INFINITY, l = 0.f;
      bool bad = false;
      for (int kt = sg.t0; kt < sg.t1; ++kt, ++n) {
        const int k0 = kt * TILE;
        ok = wait(L::SFULL + t, s_ph);
        if (!ok) break;
        s_ph ^= 1;
        ptx::tc_fence_after();
        // Values that must not reach a row through its zero weights (0 x NaN): rows of V past the
        // sequence's end, and rows that some query of the pair does not see yet and that are not
        // finite, are replaced by zeros; the latter's mask lets the rows that do see them know.
        const bool fix = k0 + TILE > min(vis0, sg.s.len);
        if (t == 0) {
          if (fix) {
            const int v = 2 * n + 1, st = v % NS;
            ok = wait(L::FULL + st, (v / NS) & 1);
            if (!ok) break;
            const uint32_t row = sbase + L::KV_OFF + st * TB + r * 128;
            const int p = k0 + r;
            uint32_t acc = 0;
            if (p >= vis0 && p < sg.s.len) {
#pragma unroll
              for (int c = 0; c < NH * 8; ++c) {
                const uint4 x = lds128(row + (c >> 3) * PANEL + (((c & 7) ^ (r & 7)) << 4));
                acc = ptx::bf16x2_fma(x.x, 0u, acc);
                acc = ptx::bf16x2_fma(x.y, 0u, acc);
                acc = ptx::bf16x2_fma(x.z, 0u, acc);
                acc = ptx::bf16x2_fma(x.w, 0u, acc);
              }
            }
            const bool nonfinite = (acc & 0x7fff7fffu) != 0;  // 0 x Inf, 0 x NaN: NaN
            if (nonfinite || p >= sg.s.len) {
#pragma unroll
              for (int c = 0; c < NH * 8; ++c)
                sts128(row + (c >> 3) * PANEL + (c << 4 & 127), make_uint4(0, 0, 0, 0));
            }
            const uint32_t mask = __ballot_sync(0xffffffffu, nonfinite);
            if (lane == 0) s_bad[(n & 1) * 4 + w] = mask;
            ptx::fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) ptx::mbar_arrive(bar(L::FIX + (n & 1)));
        }
        if (fix) {
          ok = wait(L::FIX + (n & 1), (n >> 1) & 1);
          if (!ok) break;
        }
        if (active) {
          const int lim = valid ? vis - k0 : TILE;  // columns from lim on are masked
          if (fix) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int c = valid ? lim - 32 * j : 0;
              const uint32_t sees = c >= 32 ? 0xffffffffu : c <= 0 ? 0u : (1u << c) - 1u;
              bad |= (s_bad[(n & 1) * 4 + j] & sees) != 0;
            }
          }
          uint32_t s[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) ptx::tmem_ld_32x32b_x32(ts + 32 * c, s[c]);
          ptx::tmem_wait_ld();
          if (__any_sync(0xffffffffu, lim < TILE)) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (32 * c + j >= lim) s[c][j] = 0xff800000u;
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mx[c] = -INFINITY;
#pragma unroll
            for (int j = 0; j < 32; j += 2)
              mx[c] = max3(mx[c], __uint_as_float(s[c][j]), __uint_as_float(s[c][j + 1]));
          }
          const float top = fmaxf(m, max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]));
          if (kt == sg.t0) {
            m = top;
          } else if (__any_sync(0xffffffffu, (top - m) * g.scale_log2 > 8.f)) {
            // the score MMA of this tile completed, so the P V before it has too
            const float f = top == m ? 1.f : ex2((m - top) * g.scale_log2);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              ptx::tmem_ld_32x32b_x32(to + 32 * c, o);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              ptx::tmem_st_32x32b_x32(to + 32 * c, o);
            }
            l *= f;
            m = top;
          }
          const float nm = m == -INFINITY ? 0.f : -m * g.scale_log2;
          const uint64_t nm2 = pack2(nm, nm), sl2 = pack2(g.scale_log2, g.scale_log2);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t p[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float s0 = __uint_as_float(s[2 * c + (j >> 4)][2 * j % 32]);
              const float s1 = __uint_as_float(s[2 * c + (j >> 4)][2 * j % 32 + 1]);
              const float2 x = unpack2(fma2(pack2(s0, s1), sl2, nm2));
              const float e0 = ex2(x.x), e1 = ex2(x.y);
              sum[j & 1] = add2(sum[j & 1], pack2(e0, e1));
              p[j] = pack_bf16x2(e0, e1);
            }
            ptx::tmem_st_32x32b_x32(ts + 32 * c, p);
          }
          const float2 sa = unpack2(add2(sum[0], sum[1]));
          l += sa.x + sa.y;
          ptx::tmem_wait_st();
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(L::PREADY + t));
      }
      if (!ok) break;
      // ---------------------------------------------- the item's output, or this share's part of it
      ok = wait(L::OFULL + t, o_ph);
      if (!ok) break;
      o_ph ^= 1;
      ptx::tc_fence_after();
      if (!active) continue;
      const bool whole = sg.t0 == 0 && sg.t1 == sg.nt;
      const long long row = static_cast<long long>(sg.s.row0 + sg.i0 + i) * g.q_heads + sg.h * g.group + hd;
      float* slot = g.part + (2ll * cta + (sg.t0 == 0 ? 1 : 0)) * slot_floats<D>();
      const float inv = l == 0.f ? 0.f : 1.0f / l;  // no key seen: zero
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        ptx::tmem_ld_32x32b_x32(to + 32 * c, o);
        ptx::tmem_wait_ld();
        if (bad) {
          // values that are not finite and that this row sees enter the sums as they are
          for (int p = max(vis0, sg.t0 * TILE); p < min(vis, sg.t1 * TILE); ++p) {
            const int page = kv::find_page(a, sg.b, p);
            if (page < 0) continue;
            const size_t at = (static_cast<size_t>(page) * a.heads + sg.h) * a.page_size + p % a.page_size;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              float v;
              if (Q8)
                v = kv::e4m3x2_to_float2(static_cast<const uint8_t*>(a.v)[at * D + 32 * c + j]).x * a.v_scale[at];
              else
                v = bf16_bits_to_float(static_cast<const uint16_t*>(a.v)[at * D + 32 * c + j]);
              if (!(fabsf(v) < INFINITY)) o[j] = __float_as_uint(__uint_as_float(o[j]) + v);
            }
          }
        }
        if (valid && whole) {
          uint4* dst = reinterpret_cast<uint4*>(g.out + row * D + 32 * c);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = pack_bf16x2(__uint_as_float(o[8 * j + 2 * e]) * inv, __uint_as_float(o[8 * j + 2 * e + 1]) * inv);
            dst[j] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        } else if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(slot + (t * TILE + r) * D + 32 * c);
#pragma unroll
          for (int j = 0; j < 8; ++j) dst[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
        __syncwarp();
      }
      if (valid) {
        const float ml = m == -INFINITY ? m : m * g.scale_log2;
        if (!whole) {
          slot[2 * TILE * D + t * TILE + r] = ml;
          slot[2 * TILE * (D + 1) + t * TILE + r] = l;
        } else if (g.lse) {
          g.lse[row] = l == 0.f ? -INFINITY : (ml + log2f(l)) * 0.69314718055994531f;
        }
      }
    }
  } else if (Q8) {
    // ------------------------------------------------ e4m3 -> bf16 tiles
    reg_dec<L::REGS_OTHER>();
    const int tid = threadIdx.x - 384;
    constexpr int C = D / 16;  // 16-byte chunks of a row of codes
    int n = 0;
    bool ok = true;
    while (ok && walk.next(sg)) {
      for (int x = 0; ok && x < 2 * (sg.t1 - sg.t0); ++x, ++n) {
        const int rs = n % (NR ? NR : 1), ts = n % NS;
        ok = wait(L::RFULL + rs, (n / (NR ? NR : 1)) & 1);
        if (ok && n >= NS) ok = wait(L::EMPTY + ts, (n / NS - 1) & 1);
        if (!ok) break;
        const uint32_t src = sbase + L::RAW_OFF + rs * L::RAW, dst = sbase + L::KV_OFF + ts * TB;
#pragma unroll 2
        for (int i = tid; i < TILE * C; i += 128) {
          const int r = i / C, c = i % C;
          const uint4 x4 = lds128(src + i * 16);
          uint32_t sc;
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sc) : "r"(src + TILE * D + r * 4) : "memory");
          // 2^120 times the scale as two bf16 powers of two (scale: exponent 1..247, or NaN)
          const int e = static_cast<int>(sc >> 23) + 120;
          const uint32_t lo = min(e, 254), hi = e - lo + 127;
          uint32_t s1 = lo << 7, s2 = hi << 7;
          if (sc > 0x7f800000u) s1 = 0x7fffu;
          s1 *= 0x10001u;
          s2 *= 0x10001u;
          const uint2 v0 = expand4(x4.x, s1, s2), v1 = expand4(x4.y, s1, s2);
          const uint2 v2 = expand4(x4.z, s1, s2), v3 = expand4(x4.w, s1, s2);
          const uint32_t panel = dst + (c >> 2) * PANEL + r * 128;
          const int c0 = 2 * (c & 3);
          const uint4 first = make_uint4(v0.x, v0.y, v1.x, v1.y), second = make_uint4(v2.x, v2.y, v3.x, v3.y);
          // the two panels' threads write opposite chunks at a time: no bank twice
          const bool swap = (c & 4) != 0;
          sts128(panel + (((c0 + swap) ^ (r & 7)) << 4), swap ? second : first);
          sts128(panel + (((c0 + !swap) ^ (r & 7)) << 4), swap ? first : second);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(bar(L::REMPTY + rs));
          ptx::mbar_arrive(bar(L::FULL + ts));
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the items that were cut.  Block (c, y): the item that the share of CTA c + 1 starts
// inside of, if it is the first cut of that item; the item's query rows y, y + gridDim.y, ... in turn.
// One warp adds up a row's parts (lanes over d); with few rows several warps share a row's parts and
// the first adds their sums up, in a fixed order.
constexpr int MERGE_THREADS = 512;

template <int D>
__global__ void __launch_bounds__(MERGE_THREADS) kv_merge_kernel(const kv::Args a, const AttnArgs g, int ctas) {
  constexpr int V = D / 32, W = MERGE_THREADS / 32;
  __shared__ long long scratch[40];
  __shared__ float s_acc[W][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tp = 2 * g.tpt, cut = static_cast<int>(blockIdx.x) + 1;
  kv::Start* start = reinterpret_cast<kv::Start*>(scratch + 32);
  kv::Share share;
  kv::locate<MERGE_THREADS>(a, tp, scratch, start, [&](long long w) -> long long {
    share.total = w;
    share.ctas = static_cast<int>(min(static_cast<long long>(ctas), w));
    return cut < share.ctas ? share.lo(cut) : -1;
  });
  // every block waits for the attention kernel, so that this kernel's end says that both are done
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (cut >= share.ctas) return;
  const long long u = share.lo(cut);
  kv::Walk walk(a, tp, u, share.total, start->b, start->b_lo);
  kv::Seg sg;
  if (!walk.next(sg) || sg.t0 == 0) return;
  const long long first = u - sg.t0;                // the item's first unit
  if (share.lo(cut - 1) > first) return;            // an earlier cut of the same item
  int np = 1;                                       // parts: slot 1 of CTA cut - 1, slot 0 of the CTAs after it
  while (cut + np - 1 < share.ctas && share.lo(cut + np - 1) < first + sg.nt) ++np;
  const int rows = sg.ntok * g.group;               // row = token * group + head
  int share_by = 1;                                 // warps per row
  while (share_by < W && 2 * share_by * min(rows, W) <= W && share_by < np) share_by *= 2;
  const int per_pass = W / share_by;
  const float* slot0 = g.part + (2ll * (cut - 1) + 1) * slot_floats<D>();
  const float* slot1 = g.part + 2ll * cut * slot_floats<D>();
  auto slot = [&](int p) { return p == 0 ? slot0 : slot1 + 2ll * (p - 1) * slot_floats<D>(); };
  for (int q0 = static_cast<int>(blockIdx.y) * per_pass; q0 < rows; q0 += per_pass * static_cast<int>(gridDim.y)) {
    const int q = q0 + warp % per_pass, part = warp / per_pass;
    const int tok = q / g.group, hd = q - tok * g.group;
    // the row of the slot: tokens are packed per tile
    const int r = tok < g.tpt ? q : TILE + q - g.tpt * g.group;
    float m = -INFINITY, l = 0.f, acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    if (q < rows) {
      for (int p = lane; p < np; p += 32) m = fmaxf(m, slot(p)[2 * TILE * D + r]);
#pragma unroll
      for (int x = 16; x >= 1; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
      const float m0 = m == -INFINITY ? 0.f : m;
      for (int p = lane; p < np; p += 32) l += slot(p)[2 * TILE * (D + 1) + r] * ex2(slot(p)[2 * TILE * D + r] - m0);
#pragma unroll
      for (int x = 16; x >= 1; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
#pragma unroll 4
      for (int p = part; p < np; p += share_by) {
        const float* s = slot(p);
        const float f = ex2(s[2 * TILE * D + r] - m0);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = fmaf(f, s[r * D + lane * V + j], acc[j]);
      }
    }
    if (share_by > 1) {
#pragma unroll
      for (int j = 0; j < V; ++j) s_acc[warp][lane * V + j] = acc[j];
      __syncthreads();
      if (part == 0)
        for (int x = 1; x < share_by; ++x)
#pragma unroll
          for (int j = 0; j < V; ++j) acc[j] += s_acc[warp + x * per_pass][lane * V + j];
      __syncthreads();
    }
    if (q < rows && part == 0) {
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      const long long row = static_cast<long long>(sg.s.row0 + sg.i0 + tok) * g.q_heads + sg.h * g.group + hd;
      uint32_t* dst = reinterpret_cast<uint32_t*>(g.out + row * D + lane * V);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) dst[j] = pack_bf16x2(acc[2 * j] * inv, acc[2 * j + 1] * inv);
      if (g.lse && lane == 0) g.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
  }
}

// The cache's keys or values as rows of d bf16, in 128-byte swizzled boxes of chunk x 64.
bool encode_pool(CUtensorMap* map, void* pool, long long rows, int d, int chunk) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t gdim[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows)};
  cuuint64_t gstride[1] = {static_cast<cuuint64_t>(d) * 2};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(chunk)};
  cuuint32_t estride[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, pool, gdim, gstride, box, estride,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool Q8>
cudaError_t launch(const kv::Args& a, const AttnArgs& g, const CUtensorMap& tk, const CUtensorMap& tv, int ctas,
                   cudaStream_t s) {
  using L = Layout<D, Q8>;
  cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kv_attention_kernel<D, Q8>), L::BYTES);
  if (e != cudaSuccess) return e;
  kv_attention_kernel<D, Q8><<<ctas, L::THREADS, L::BYTES, s>>>(a, g, tk, tv);
  note_launches(1);
  e = cudaGetLastError();
  // items of one key tile are never cut
  if (e != cudaSuccess || ctas == 1 || static_cast<long long>(a.table_width) * a.page_size <= TILE) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas - 1, static_cast<long long>(a.T) * g.group > 64 ? 2 : 1);
  cfg.blockDim = dim3(MERGE_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv_merge_kernel<D>, a, g, ctas);
  note_launches(1);
  return e;
}

}  // namespace

int num_sms();
unsigned long long wait_limit_ns();

size_t kv_attention_workspace_bytes(int d) {
  return 2 * static_cast<size_t>(num_sms()) * (d == 64 ? slot_floats<64>() : slot_floats<128>()) * sizeof(float);
}

cudaError_t launch_kv_attention(const kv::Args& a, bool q8, const uint16_t* q, long long q_token, long long q_head,
                                int q_heads, float scale, uint16_t* out, float* lse, void* ws, cudaStream_t s) {
  AttnArgs g;
  g.q = q;
  g.q_token = q_token;
  g.q_head = q_head;
  g.out = out;
  g.lse = lse;
  g.part = static_cast<float*>(ws);
  g.scale_log2 = scale * 1.44269504088896341f;
  g.q_heads = q_heads;
  g.group = q_heads / a.heads;
  g.tpt = TILE / g.group;
  g.chunk = a.page_size & -a.page_size;  // the largest power of two that divides the page
  if (g.chunk > TILE) g.chunk = TILE;
  const unsigned long long ns = wait_limit_ns();
  g.wait_cycles = ns > (~0ull) / 3 ? ~0ull : ns * 21 / 10;
  g.sleep_ns = ns < 20000ull ? static_cast<uint32_t>(ns > 0 ? ns : 1) : 20000u;
  CUtensorMap tk, tv;
  memset(&tk, 0, sizeof(tk));
  memset(&tv, 0, sizeof(tv));
  if (!q8) {
    const long long rows = static_cast<long long>(a.num_pages) * a.heads * a.page_size;
    if (!encode_pool(&tk, a.k, rows, a.d, g.chunk) || !encode_pool(&tv, a.v, rows, a.d, g.chunk))
      return cudaErrorInvalidValue;
  }
  const int ctas = num_sms();
  if (a.d == 64) return q8 ? launch<64, true>(a, g, tk, tv, ctas, s) : launch<64, false>(a, g, tk, tv, ctas, s);
  return q8 ? launch<128, true>(a, g, tk, tv, ctas, s) : launch<128, false>(a, g, tk, tv, ctas, s);
}

}  // namespace moe
