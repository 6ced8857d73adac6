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
// Roles (warps): 0 works out the CTA's segments and copies keys and values (TMA
// boxes of up to 128 rows of a page into 128-byte swizzled tiles), 1 issues the
// MMAs, 2 and 3 load the queries, 4-7 and 8-11 the softmax of the pair's tiles.
// Items of one tile alternate key tiles between the two halves; items of at most
// 32 rows take the form of moe_kv_thin.cuh in the same kernel.  With an e4m3
// cache warps 12-15 expand the tiles to bf16: e4m3 times a power of two is
// exact in bf16, so everything after that is the same as for a bf16 cache, to
// the bit.  Every wait is bounded (MOE_DEV_TIMEOUT).
//
// Roundings: P to bf16 (the tensor core's operand; sums are taken of the
// unrounded values), the output to bf16.  All else is FP32.
//
// What bounds it, by calls in a row from a CUDA graph (16 query heads over 2 KV
// heads of 128): 4096 tokens over 32K cached ones take 0.80 ms (0.82 to 0.84 in
// calls that go on for longer), 1.46 PFLOP/s, 0.75 of the rate of a large plain
// product; the tensor pipe is active 63 % of the time and waits for the softmax
// threads, whose tile takes them longer (the loads from TMEM, 128 exponentials
// and the conversions of a row, one after another in one thread) than its two
// products.  Six chunks of 440 to 1777 tokens over an e4m3 cache 0.32 ms.  A
// 512-token prompt takes 15 us and one token over 4K keys 11 us, nearly all of
// it a chain of latencies that no size enters: launch, plan, first page, first
// keys, scores, output, merge.  With an e4m3 cache 512 threads leave 128
// registers each, and the compiler spills a few (206 bytes stored at D = 128,
// 142 at D = 64); the bf16 kernels spill none.
#include <cuda.h>
#include <string.h>

#include <type_traits>

#include "moe_kv_attn.cuh"
#include "moe_kv_thin.cuh"
#include "moe_tmap.cuh"

namespace moe {

namespace {

using namespace kv;

// Zeros in place of the elements that are not finite of row `row` (r: its swizzle) of a bf16 tile.  A call,
// so that what hardly ever runs stays out of the loop over the key tiles.
template <int NH>
__device__ __noinline__ void keep_finite(uint32_t row, int r) {
#pragma unroll 1
  for (int c = 0; c < NH * 8; ++c) {
    const uint32_t at = row + (c >> 3) * (TILE * 128) + (((c & 7) ^ r) << 4);
    sts128(at, bf16x8_finite(lds128(at)));
  }
}

template <int D, bool Q8>
__global__ void __launch_bounds__(Layout<D, Q8>::THREADS, 1)
    kv_attention_kernel(const kv::Args a, const AttnArgs g, const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_v) {
  using L = Layout<D, Q8>;
  constexpr int NH = L::NH, PANEL = L::PANEL, TB = L::TB, NS = L::NS;
  extern __shared__ uint8_t kv_smem_raw[];
  const uint32_t raw = ptx::smem_u32(kv_smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = kv_smem_raw + (sbase - raw);
  auto bar = [sbase](int i) -> uint32_t { return sbase + L::BAR_OFF + 8u * static_cast<uint32_t>(i); };
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + L::MISC_OFF + 4);
  volatile uint32_t* s_bad = reinterpret_cast<volatile uint32_t*>(smem + L::MISC_OFF + 16);  // [2][4]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = static_cast<int>(blockIdx.x);

  if (warp == 0) {
    for (int i = lane; i < L::NBAR; i += 32) ptx::mbar_init(bar(i), L::arrivals(i));
    if (lane == 0) *s_abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(s_tmem), 512);
    ptx::tmem_relinquish();
  }
  // the kernel may start while the one before it in the stream ends: nothing is read before it has
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // this CTA's share of the units (the scan's scratch lies where the key/value ring will be)
  kv::Share share;
  kv::Start from;
  if (a.B > 32 || warp == 0)
    from = kv::locate<L::THREADS>(a, g.tokens, static_cast<int>(gridDim.x), g.merge, cta,
                                  reinterpret_cast<long long*>(smem + L::KV_OFF), share);
  Seg sg;
  kv::Walk walk(a, g.tokens, 0, 0, 0, 0, false);
  if (warp == 0) {  // works the segments out; the first while the CTA starts up
    if (cta < share.ctas)
      walk = kv::Walk(a, g.tokens, share.lo(cta), share.lo(cta + 1), from.b, from.b_lo, share.whole);
    if (!walk.next(sg)) sg.ntok = 0;  // the end
  }
  ptx::fence_proxy_async_smem();  // the scratch is overwritten by copies
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *s_tmem;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  auto wait = [&](int i, uint32_t parity) -> bool {
    return wait_warp(bar(i), parity, s_abort, a.err, g);
  };
  // the CTA's segments, in order, as warp 0 publishes them
  int segs = 0;  // taken so far
  auto next = [&](Seg& sg) -> bool {
    const int slot = segs % SEGS;
    if (!wait(L::SEGF + slot, (segs / SEGS) & 1)) return false;
    const int4* p = reinterpret_cast<const int4*>(smem + L::SEG_OFF + slot * 48);
    const int4 x = p[0], y = p[1], z = p[2];
    sg = {uniform(x.x), uniform(x.y), uniform(x.z), uniform(x.w), uniform(y.x),
          uniform(y.y), uniform(y.z), uniform(y.w), uniform(z.x), uniform(z.y)};
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar(L::SEGE + slot));
    ++segs;
    return sg.ntok > 0;
  };
  auto thin = [&](const Seg& sg) -> bool { return sg.ntok * g.group <= THIN_ROWS; };

  if (warp < 4) {
    reg_dec<L::REGS_ISSUE>();
    if (warp == 0) {
      // ---------------------------------------------- segments, and copies: K and V of every key tile
      const int per_page = g.per_page, per_tile = TILE >> g.chunk_log;
      // per ring (tile form, thin form): tiles issued, next slot, its round's parity, landing barrier
      struct Ring {
        int n, st, ph, fl;
      } tile_ring = {0, 0, 0, 0}, thin_ring = {0, 0, 0, 0};
      bool ok = true;
      int form = -1;  // the last segment's
      uint32_t tc_ph = 0;
      int4 join = make_int4(0, 0, 0, 0);
      for (;; ++segs) {
        if (segs > 0 && !walk.next(sg)) sg.ntok = 0;
        const int slot = segs % SEGS;
        if (segs >= SEGS && !wait(L::SEGE + slot, (segs / SEGS - 1) & 1)) break;
        if (lane == 0) {
          int4* p = reinterpret_cast<int4*>(smem + L::SEG_OFF + slot * 48);
          p[0] = make_int4(sg.row0, sg.len, sg.b, sg.h);
          p[1] = make_int4(sg.i0, sg.ntok, sg.base, sg.t0);
          p[2] = make_int4(sg.t1, sg.nt, 0, 0);
          ptx::mbar_arrive(bar(L::SEGF + slot));
        }
        __syncwarp();
        if (sg.ntok == 0) break;
        sg = {uniform(sg.row0), uniform(sg.len), uniform(sg.b),  uniform(sg.h),  uniform(sg.i0),
              uniform(sg.ntok), uniform(sg.base), uniform(sg.t0), uniform(sg.t1), uniform(sg.nt)};
        if (sg.t0 == 0 && sg.t1 < sg.nt)  // the rest of the item is other CTAs': this part will be joined with theirs
          join = make_int4(share.of(walk.item_end - 1) - cta + 1, sg.row0 + sg.i0, sg.ntok, sg.h);
        const int now = Q8 && thin(sg) ? 1 : 0;
        if (Q8 && form >= 0 && now != form) {
          // the rings share memory
          if (now == 1) {
            ok = wait(L::TCDONE, tc_ph);
            tc_ph ^= 1;
          } else {
            const int n = thin_ring.n;
            for (int i = max(0, n - L::NH_); ok && i < n; ++i) ok = wait(L::HEMPTY + i % L::NH_, (i / L::NH_) & 1);
          }
          if (!ok) break;
        }
        form = now;
        Ring rg = now ? thin_ring : tile_ring;
        const int slots = now ? L::NH_ : L::NL, full0 = now ? L::HFULL : L::LFULL, empty0 = now ? L::HEMPTY : L::LEMPTY;
        const uint32_t ring0 = sbase + (now ? L::H_OFF : L::L_OFF);
        const int last = (sg.len + g.chunk - 1) >> g.chunk_log;  // chunks of the sequence
        int c0 = sg.t0 * per_tile;
        // the pool's rows where chunks c0 .. c0 + 31 start, and the 32 after them, one per lane
        auto rows_of = [&](int c) -> int {
          if (c >= last) return 0;
          const int e = c / per_page;
          const int page = max(kv::page_of(a, sg.b, e), 0);  // (a bad one is recorded, and not followed)
          return (page * a.heads + sg.h) * a.page_size + ((c - e * per_page) << g.chunk_log);
        };
        int rows = rows_of(c0 + lane), rows2 = rows_of(c0 + 32 + lane);
        for (int kt = sg.t0; ok && kt < sg.t1; ++kt) {
          const int c = kt * per_tile;
          if (c - c0 >= 32) {
            c0 += 32;
            rows = rows2;
            rows2 = rows_of(c0 + 32 + lane);
          }
          const int have = max(0, min(per_tile, last - c));
#pragma unroll 1
          for (int kind = 0; kind < 2; ++kind) {
            if (rg.n >= slots && !wait(empty0 + rg.st, rg.ph ^ 1)) {
              ok = false;
              break;
            }
            const uint32_t f = bar(full0 + rg.fl), dst = ring0 + rg.st * L::LAND;
            const CUtensorMap* map = kind ? &tmap_v : &tmap_k;
            const float* scale = kind ? a.v_scale : a.k_scale;
            ptx::mbar_arrive_expect_tx_elect(f, static_cast<uint32_t>(have * g.chunk * (Q8 ? D + 4 : 2 * D)));
#pragma unroll 1
            for (int j = 0; j < have; ++j) {
              const int row = uniform(lane == c - c0 + j ? rows : 0);
              if (!Q8) {
#pragma unroll
                for (int hf = 0; hf < NH; ++hf)
                  ptx::tma_load_2d_elect(dst + hf * PANEL + j * g.chunk * 128, map, hf * 64, row, f);
              } else {
                ptx::tma_load_2d_elect(dst + j * g.chunk * D, map, 0, row, f);
                ptx::bulk_g2s_elect(sbase + L::SCALE_OFF + (rg.st * TILE + j * g.chunk) * 4, scale + row, g.chunk * 4, f);
              }
            }
            ++rg.n;
            if (++rg.fl == 2 * slots) rg.fl = 0;
            if (++rg.st == slots) {
              rg.st = 0;
              rg.ph ^= 1;
            }
          }
        }
        (now ? thin_ring : tile_ring) = rg;
        if (!ok) break;
      }
      if (lane == 0) g.joins[cta] = join;
      // every copy issued has landed before the CTA ends (at once unless a wait gave up)
      for (int i = max(0, tile_ring.n - L::NL); i < tile_ring.n; ++i)
        tc_dev::wait_drain(bar(L::LFULL + i % (2 * L::NL)), (i / (2 * L::NL)) & 1, 0);
      for (int i = max(0, thin_ring.n - L::NH_); i < thin_ring.n; ++i)
        tc_dev::wait_drain(bar(L::HFULL + i % (2 * L::NH_)), (i / (2 * L::NH_)) & 1, 0);
    } else if (warp == 1) {
      // ---------------------------------------------- MMA issue, one unit behind for P V
      // A unit's tiles: a and b (a pair), or one of them (t alternates along the keys).
      // All operands are warp-uniform, and the tiles known at compile time: an MMA whose operands have to
      // be brought to the uniform registers lane by lane takes longer to issue than to run.
      const uint32_t id_s = ptx::idesc_bf16_f32(TILE, TILE), id_o = idesc_pv(D);
      const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
      const uint64_t q_desc = ptx::smem_desc_sw128(sbase + L::Q_OFF), k_desc = ptx::smem_desc_sw128(sbase + L::KV_OFF);
      const uint64_t v_desc = desc_mn_sw128(sbase + L::KV_OFF, PANEL);
      uint32_t pa_ph = 0, pb_ph = 0, qb_ph = 0;
      // the current unit's K: slot of the bf16 ring, its barrier (twice as many for bf16), the round's parity
      constexpr int BARS = Q8 ? NS : 2 * NS, FULL0 = Q8 ? L::FULL : L::LFULL, EMPTY0 = Q8 ? L::EMPTY : L::LEMPTY;
      int st = 0, fl = 0, ph = 0;
      auto advance = [&](int by) {
        st += by;
        while (st >= NS) st -= NS;
        fl += by;
        while (fl >= BARS) {
          fl -= BARS;
          ph ^= 1;
        }
      };
      // the previous unit: tiles whose P V is still to do, V's slot, barrier and parity, first and last of
      // the item's run for its tiles
      int todo = 0, v_st = 0, v_fl = 0, v_ph = 0;
      bool v_first = false, v_last = false;
      // releases a ring tile once the MMAs issued so far are done with it
      auto release = [&](int slot) {
        if (!Q8 && lane == 0) mbar_arrive_n(bar(EMPTY0 + slot), 7);
        ptx::mma_commit_elect(bar(EMPTY0 + slot));
      };
      // O += P V of the previous unit for tile t
      auto finish = [&](auto tile) -> bool {
        constexpr int t = decltype(tile)::value;
        if (!(todo & (1 << t))) return true;
        uint32_t& p_ph = t == 0 ? pa_ph : pb_ph;
        if (!wait(FULL0 + v_fl, v_ph) || !wait(L::PREADY + t, p_ph)) return false;
        p_ph ^= 1;
        ptx::tc_fence_after();
        mma_pv_elect(tm + TM_O + t * D, tm + TM_S + t * TILE, v_desc + static_cast<uint32_t>(v_st * (TB >> 4)), id_o,
                     v_first ? 0u : 1u);
        if (v_last) ptx::mma_commit_elect(bar(L::OFULL + t));
        todo &= ~(1 << t);
        if (todo == 0) release(v_st);
        return true;
      };
      // S = Q K^T of the current unit into tile t's scores, from query tile q
      auto scores = [&](auto tile, auto query, bool last) {
        constexpr int t = decltype(tile)::value, q = decltype(query)::value;
        ptx::tc_fence_after();
        const uint64_t dk = k_desc + static_cast<uint32_t>(st * (TB >> 4));
        if (NH == 2)
          mma_qk2_elect(tm + TM_S + t * TILE, q_desc + q * (TB >> 4), dk, id_s);
        else
          ptx::mma_group_ss_elect(tm + TM_S + t * TILE, q_desc + q * (TB >> 4), dk, id_s, 0u);
        ptx::mma_commit_elect(bar(L::SFULL + t));
        if (last) {
          if (q == 1 && lane == 0) mbar_arrive_n(bar(L::QEMPTY + 1), 7);
          ptx::mma_commit_elect(bar(L::QEMPTY + q));
        }
      };
      const std::integral_constant<int, 0> A;
      const std::integral_constant<int, 1> B;
      // the current unit becomes the previous one
      auto pass = [&](int tiles, bool first, bool last) {
        advance(1);
        todo = tiles;
        v_st = st;
        v_fl = fl;
        v_ph = ph;
        v_first = first;
        v_last = last;
        advance(1);
      };
      bool ok = true, tiles_before = false;  // tiles_before: the last segment was of the tile form
      while (ok && next(sg)) {
        const uint32_t seg_ph = (segs - 1) & 1;
        const int run = sg.t1 - sg.t0;
        if (thin(sg)) {
          // the softmax warps' own; its tiles pass by, and what is pending must not wait for it
          ok = finish(A) && finish(B) && wait(L::QFULL, seg_ph);
          if (ok && lane == 0) ptx::mbar_arrive(bar(L::QEMPTY));
          if (Q8 && tiles_before) ptx::mma_commit_elect(bar(L::TCDONE));
          tiles_before = false;
          if (!Q8) advance(2 * run % BARS), ph ^= 2 * run / BARS & 1;
          continue;
        }
        tiles_before = true;
        if (sg.ntok > g.tpt) {
          for (int j = 0; j < run; ++j) {
            const bool last = j + 1 == run;
            if (!(ok = (j > 0 || wait(L::QFULL, seg_ph)) && wait(FULL0 + fl, ph) && finish(A))) break;
            scores(A, A, last);
            if (!(ok = finish(B) && (j > 0 || wait(L::QFULL + 1, qb_ph)))) break;
            if (j == 0) qb_ph ^= 1;
            scores(B, B, last);
            release(st);
            pass(3, j == 0, last);
          }
        } else {
          // the scores of the next unit come before the previous unit's P V, which has the other buffer
          for (int j = 0; j < run; ++j) {
            const bool last = j + 1 == run;
            if (j & 1) {
              if (!(ok = finish(B) && wait(FULL0 + fl, ph))) break;
              scores(B, A, last);
              release(st);
              if (!(ok = finish(A))) break;
            } else {
              if (!(ok = finish(A) && (j > 0 || wait(L::QFULL, seg_ph)) && wait(FULL0 + fl, ph))) break;
              scores(A, A, last);
              release(st);
              if (!(ok = finish(B))) break;
            }
            pass(1 << (j & 1), j < 2, j + 2 >= run);
          }
        }
      }
      if (ok) ok = finish(A) && finish(B);
      // all MMAs are done before the tensor memory is released
      ptx::mma_commit_elect(bar(L::DRAIN));
      tc_dev::wait_drain(bar(L::DRAIN), 0, 0);
    } else {
      // ---------------------------------------------- queries: tile t of a pair, or half of a lone tile's rows
      const int t = warp - 2;
      constexpr int C = D / 8, R = 32 / C;  // a row's pieces of 8 values, a lane each; rows at a time
      const long long by_token = g.q_token - g.group * g.q_head;
      uint32_t ph = 1, phb = 1;  // of QEMPTY: the first use waits for nothing
      while (next(sg)) {
        const bool pair = sg.ntok > g.tpt;
        if (!wait(L::QEMPTY, ph)) break;
        ph ^= 1;
        if (t == 1) {
          // tile a's barrier waits for this warp too: the thin form uses both tiles' memory
          if (pair || thin(sg)) {
            if (!wait(L::QEMPTY + 1, phb)) break;
            phb ^= 1;
          }
          if (pair && lane == 0) ptx::mbar_arrive(bar(L::QFULL));
        }
        const int tile = pair ? t : 0, tok0 = tile * g.tpt, rows = min(g.tpt, sg.ntok - tok0) * g.group;
        // rows in the order token, head: from r every `step` rows, that is `dt` tokens and `dh` heads on
        const int step = pair ? R : 2 * R, dt = step / g.group, dh = step - dt * g.group;
        int r = (pair ? 0 : t * R) + lane / C;
        const int tok = r / g.group;
        int hd = r - tok * g.group;
        const uint16_t* src = g.q + (sg.row0 + sg.i0 + tok0 + tok) * g.q_token +
                              (static_cast<long long>(sg.h) * g.group + hd) * g.q_head + lane % C * 8;
        const long long jump = dt * g.q_token + dh * g.q_head;
        const uint32_t col = sbase + L::Q_OFF + tile * TB + (lane % C >> 3) * PANEL;
#pragma unroll 8
        for (; r < rows; r += step) {
          ptx::cp_async_16(col + r * 128 + (((lane & 7) ^ (r & 7)) << 4), src);
          hd += dh;
          const bool over = hd >= g.group;
          hd -= over ? g.group : 0;
          src += jump + (over ? by_token : 0);
        }
        ptx::cp_async_wait_all();
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(L::QFULL + tile));
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
    float* s_ml = reinterpret_cast<float*>(smem + L::ML_OFF);
    uint32_t s_ph = 0, o_ph[2] = {0, 0}, x_ph = 0;
    int all = 0, n = 0;  // units before the current segment: in all, and of the tile form
    uint32_t team_ph = 0;
    bool ok = true, lent = false;  // lent: O b (and its rows' sums) are being read by tile a's threads
    while (ok && next(sg)) {
      const int run = sg.t1 - sg.t0;
      ok = wait(L::QFULL, (segs - 1) & 1);
      if (!ok) break;
      if (thin(sg)) {
        if (lent) {
          ok = wait(L::OBFREE, t == 1 ? x_ph : x_ph ^ 1);
          if (!ok) break;
          if (t == 1) x_ph ^= 1;
          lent = false;
        }
        const ThinCtx ctx = {sbase, smem, s_abort, warp - 4, lane};
        ok = sg.ntok * g.group <= 8 ? thin_segment<D, Q8, true>(a, g, sg, ctx, cta, Q8 ? all - n : all, team_ph)
                                    : thin_segment<D, Q8, false>(a, g, sg, ctx, cta, Q8 ? all - n : all, team_ph);
        all += run;
        continue;
      }
      if (lane == 0) ptx::mbar_arrive(bar(L::QEMPTY));  // the queries are the MMA warp's
      const int ring0 = Q8 ? 2 * n : 2 * all;           // bf16 tiles before the segment
      const int n0 = n;
      all += run;
      n += run;
      const bool pair = sg.ntok > g.tpt;
      const bool two = pair || run > 1;  // tile b has work
      if (t == 1 && !two) continue;
      const int i = (pair ? t * g.tpt : 0) + tok;
      const bool valid = tok < g.tpt && i < sg.ntok;
      const bool active = __any_sync(0xffffffffu, valid);
      const int vis = sg.base + i + 1;  // keys that this row sees: 0 .. vis - 1
      const int vis0 = sg.base + 1;     // keys that all rows of the pair see
      const int first = sg.t0 + (pair ? 0 : t), step = pair ? 1 : 2;
      float m = -INFINITY, l = 0.f;
      bool bad = false;
      if (t == 1 && lent) {
        ok = wait(L::OBFREE, x_ph);
        if (!ok) break;
        x_ph ^= 1;
        lent = false;
      }
      for (int kt = first; kt < sg.t1; kt += step) {
        const int k0 = kt * TILE, un = n0 + kt - sg.t0;
        ok = wait(L::SFULL + t, s_ph);
        if (!ok) break;
        s_ph ^= 1;
        ptx::tc_fence_after();
        // Values that must not reach a row through its zero weights (0 x NaN): rows of V past the
        // sequence's end, and the elements that are not finite of rows that some query of the pair does
        // not see yet, are replaced by zeros; the mask of the latter's rows lets those that do see them
        // know.
        const bool fix = k0 + TILE > min(vis0, sg.len);
        if (t == 0 || !pair) {
          if (fix) {
            const int v = ring0 + 2 * (kt - sg.t0) + 1, st = v % NS;
            ok = Q8 ? wait(L::FULL + st, (v / NS) & 1) : wait(L::LFULL + v % (2 * NS), (v / (2 * NS)) & 1);
            if (!ok) break;
            const uint32_t row = sbase + L::KV_OFF + st * TB + r * 128;
            const int p = k0 + r;
            uint32_t acc = 0;
            if (p >= vis0 && p < sg.len) {
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
            if (p >= sg.len) {
#pragma unroll
              for (int c = 0; c < NH * 8; ++c)
                sts128(row + (c >> 3) * PANEL + (((c & 7) ^ (r & 7)) << 4), make_uint4(0, 0, 0, 0));
            }
            const uint32_t mask = __ballot_sync(0xffffffffu, nonfinite);
            if (lane == 0) s_bad[(un & 1) * 4 + w] = mask;
            if (nonfinite) keep_finite<NH>(row, r & 7);
            ptx::fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) ptx::mbar_arrive(bar(L::FIX + (un & 1)));
        }
        if (fix) {
          ok = wait(L::FIX + (un & 1), (un >> 1) & 1);
          if (!ok) break;
        }
        if (active) {
          const int lim = valid ? vis - k0 : TILE;  // columns from lim on are masked
          if (fix) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int c = valid ? lim - 32 * j : 0;
              const uint32_t sees = c >= 32 ? 0xffffffffu : c <= 0 ? 0u : (1u << c) - 1u;
              bad |= (s_bad[(un & 1) * 4 + j] & sees) != 0;
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
          if (kt == first) {
            m = top;
          } else if (__any_sync(0xffffffffu, valid && (top - m) * g.scale_log2 > 8.f)) {
            // (rows of no query hold leftovers and have no say)
            // this tile's scores are complete, so the P V that was issued before them is too
            const float f = top == m ? 1.f : ex2((m - top) * g.scale_log2);
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld_x16(to + 16 * c, o);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st_x16(to + 16 * c, o);
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
      float ml = m == -INFINITY ? m : m * g.scale_log2;
      if (t == 1 && !pair) {
        // tile a's threads join both halves of the keys
        s_ml[r] = ml;
        s_ml[TILE + r] = l;
        smem[L::ML_OFF + 8 * TILE + r] = bad;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(L::ML));
        o_ph[1] ^= 1;
        lent = true;
        continue;
      }
      ok = wait(L::OFULL + t, o_ph[t]);
      if (!ok) break;
      o_ph[t] ^= 1;
      float fa = 1.f, fb = 0.f;
      const bool join = !pair && two;
      if (t == 0 && two) {
        if (join) {
          ok = wait(L::OFULL + 1, o_ph[1]) && wait(L::ML, x_ph);
          if (!ok) break;
          x_ph ^= 1;
          const float mb = s_ml[r], top = fmaxf(ml, mb), top0 = top == -INFINITY ? 0.f : top;
          fa = ex2(ml - top0);
          fb = ex2(mb - top0);
          l = l * fa + s_ml[TILE + r] * fb;
          ml = top;
          bad |= smem[L::ML_OFF + 8 * TILE + r] != 0;
        }
        o_ph[1] ^= 1;
      }
      ptx::tc_fence_after();
      if (active) {
        const bool whole = sg.t0 == 0 && sg.t1 == sg.nt;
        const long long row = static_cast<long long>(sg.row0 + sg.i0 + i) * g.q_heads + sg.h * g.group + hd;
        float* slot = g.part + (2ll * cta + (sg.t0 == 0 ? 1 : 0)) * slot_floats<D>();
        const float inv = l == 0.f ? 0.f : 1.0f / l;  // no key seen: zero
        const int q = (pair ? t : 0) * TILE + r;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          ptx::tmem_ld_32x32b_x32(to + 32 * c, o);
          if (join) {
            uint32_t ob[32];
            ptx::tmem_ld_32x32b_x32(to + D + 32 * c, ob);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              o[j] = __float_as_uint(__uint_as_float(o[j]) * fa + __uint_as_float(ob[j]) * fb);
          } else {
            ptx::tmem_wait_ld();
          }
          if (bad) {
            // elements that are not finite and that this row sees enter the sums as they are
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
            uint4* dst = reinterpret_cast<uint4*>(slot + q * D + 32 * c);
#pragma unroll
            for (int j = 0; j < 8; ++j) dst[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
          __syncwarp();
        }
        if (valid) {
          if (!whole) {
            slot[2 * TILE * D + q] = ml;
            slot[2 * TILE * (D + 1) + q] = l;
          } else if (g.lse) {
            g.lse[row] = l == 0.f ? -INFINITY : (ml + log2f(l)) * 0.69314718055994531f;
          }
        }
      }
      lent = join;
      if (join) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(L::OBFREE));
      }
    }
  } else if (Q8) {
    // ------------------------------------------------ e4m3 -> bf16 tiles
    reg_dec<L::REGS_EXPAND>();
    const int tid = threadIdx.x - 384;
    constexpr int C = D / 16;  // 16-byte chunks of a row of codes
    int n = 0;                 // tiles so far
    bool ok = true;
    while (ok && next(sg)) {
      if (thin(sg)) continue;
      for (int x = 0; ok && x < 2 * (sg.t1 - sg.t0); ++x, ++n) {
        const int rs = n % L::NL, ts = n % NS;
        ok = wait(L::LFULL + n % (2 * L::NL), (n / (2 * L::NL)) & 1);
        if (!ok) break;
        // one row per thread; the swizzles keep eight neighbouring threads' loads and stores in
        // different banks
        const uint32_t src = sbase + L::L_OFF + rs * L::LAND + tid * D, dst = sbase + L::KV_OFF + ts * TB + tid * 128;
        uint4 codes[C];
#pragma unroll
        for (int c = 0; c < C; ++c) codes[c] = lds128(src + ((c ^ (D == 128 ? tid & 7 : (tid >> 1) & 3)) << 4));
        float sc;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(sc) : "r"(sbase + L::SCALE_OFF + (rs * TILE + tid) * 4) : "memory");
        uint32_t s1, s2;
        scale_pairs(sc, &s1, &s2);
        const bool twice = __any_sync(0xffffffffu, s2 != 0x3f803f80u);
        if (n >= NS) {
          ok = wait(L::EMPTY + ts, (n / NS - 1) & 1);
          if (!ok) break;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          uint2 v[4] = {expand4(codes[c].x, s1), expand4(codes[c].y, s1), expand4(codes[c].z, s1),
                        expand4(codes[c].w, s1)};
          if (twice) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = make_uint2(bf16x2_mul(v[j].x, s2), bf16x2_mul(v[j].y, s2));
          }
          const uint32_t panel = dst + (c >> 2) * PANEL;
          const int c0 = 2 * (c & 3);
          sts128(panel + ((c0 ^ (tid & 7)) << 4), make_uint4(v[0].x, v[0].y, v[1].x, v[1].y));
          sts128(panel + (((c0 + 1) ^ (tid & 7)) << 4), make_uint4(v[2].x, v[2].y, v[3].x, v[3].y));
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(bar(L::LEMPTY + rs));
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

// Joins the parts of the items that were cut.  Blocks (c, y): the item whose first part is CTA c's, if
// there is one, and every gridDim.y-th of its rows.  A row's parts go to 1, 2, 4 or 8 warps (at four parts
// per warp's round the loads of a round are in flight together), lanes over d, each with a running
// maximum; the warps' sums are added in a fixed order.
// Sixteen blocks per item: with 8, six drafted tokens of 8 sequences take 23.4 us, not 20.6; with 32, 8 e4m3
// sequences of one token 30.1, not 29.5.
constexpr int MERGE_WARPS = 8, MERGE_Y = 16;

template <int D>
__global__ void __launch_bounds__(32 * MERGE_WARPS) kv_merge_kernel(const AttnArgs g) {
  constexpr int V = D / 32;
  __shared__ float s_m[MERGE_WARPS], s_l[MERGE_WARPS], s_acc[MERGE_WARPS][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = static_cast<int>(blockIdx.x);
  // every block waits for the attention kernel, so that this kernel's end says that both are done
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 join = g.joins[cta];
  const int np = join.x, rows = join.z * g.group;  // parts: slot 1 of this CTA, slot 0 of those after it
  if (np == 0) return;
  const int per_row = np <= 4 ? 1 : np <= 8 ? 2 : np <= 16 ? 4 : 8, per_pass = MERGE_WARPS / per_row;
  const int sub = warp % per_row;
  const float* slot0 = g.part + (2ll * cta + 1) * slot_floats<D>();
  const float* slot1 = g.part + 2ll * (cta + 1) * slot_floats<D>();
  auto slot = [&](int p) { return p == 0 ? slot0 : slot1 + 2ll * (p - 1) * slot_floats<D>(); };
  for (int q0 = static_cast<int>(blockIdx.y) * per_pass; q0 < rows; q0 += per_pass * static_cast<int>(gridDim.y)) {
    const int q = min(q0 + warp / per_row, rows - 1);
    // the row of a slot: tokens are packed per tile
    const int r = q < g.tpt * g.group ? q : TILE + q - g.tpt * g.group;
    float m = -INFINITY, l = 0.f, acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    for (int p0 = sub; p0 < np; p0 += 4 * per_row) {
      float pm[4], pl[4], po[4][V];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = p0 + i * per_row;
        const float* s = slot(min(p, np - 1));
        pm[i] = s[2 * TILE * D + r];
        pl[i] = s[2 * TILE * (D + 1) + r];
        if (V == 4) {
          const float4 x = *reinterpret_cast<const float4*>(s + r * D + lane * 4);
          po[i][0] = x.x, po[i][1] = x.y, po[i][V - 2] = x.z, po[i][V - 1] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(s + r * D + lane * 2);
          po[i][0] = x.x, po[i][1] = x.y;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (p0 + i * per_row >= np) pm[i] = -INFINITY, pl[i] = 0.f;
      const float top = fmaxf(m, fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])));
      const float t0 = top == -INFINITY ? 0.f : top, f = ex2(m - t0);
      l *= f;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] *= f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (p0 + i * per_row < np) {
          const float w = ex2(pm[i] - t0);
          l = fmaf(pl[i], w, l);
#pragma unroll
          for (int j = 0; j < V; ++j) acc[j] = fmaf(po[i][j], w, acc[j]);
        }
      m = top;
    }
    if (per_row > 1) {
      if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
      for (int j = 0; j < V; ++j) s_acc[warp][lane * V + j] = acc[j];
      __syncthreads();
      if (sub == 0) {
        for (int w = warp; w < warp + per_row; ++w) m = fmaxf(m, s_m[w]);
        const float t0 = m == -INFINITY ? 0.f : m;
        l = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = 0.f;
        for (int w = warp; w < warp + per_row; ++w) {
          const float f = ex2(s_m[w] - t0);
          l = fmaf(s_l[w], f, l);
#pragma unroll
          for (int j = 0; j < V; ++j) acc[j] = fmaf(s_acc[w][lane * V + j], f, acc[j]);
        }
      }
      __syncthreads();
    }
    if (sub == 0 && q0 + warp / per_row < rows) {
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      const int tok = q / g.group, hd = q - tok * g.group;
      const long long row = static_cast<long long>(join.y + tok) * g.q_heads + join.w * g.group + hd;
      uint32_t* dst = reinterpret_cast<uint32_t*>(g.out + row * D + lane * V);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) dst[j] = pack_bf16x2(acc[2 * j] * inv, acc[2 * j + 1] * inv);
      if (g.lse && lane == 0) g.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
  }
}

// The cache's keys or values as rows of d, in boxes of `chunk` rows: bf16 64 wide with 128-byte swizzle,
// e4m3 whole rows with a swizzle of their length.
bool encode_pool(CUtensorMap* map, void* pool, long long rows, int d, int chunk, bool q8) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t gdim[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows)};
  cuuint64_t gstride[1] = {static_cast<cuuint64_t>(d) * (q8 ? 1 : 2)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(q8 ? d : 64), static_cast<cuuint32_t>(chunk)};
  cuuint32_t estride[2] = {1, 1};
  return enc(map, q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, pool, gdim, gstride, box,
             estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
             q8 && d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool Q8>
cudaError_t launch(const kv::Args& a, const AttnArgs& g, const CUtensorMap& tk, const CUtensorMap& tv, int ctas,
                   cudaStream_t s) {
  using L = Layout<D, Q8>;
  cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kv_attention_kernel<D, Q8>), L::BYTES);
  if (e != cudaSuccess) return e;
  // each kernel may start while the one before it in the stream ends, and waits for its results itself
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(L::THREADS);
  cfg.dynamicSmemBytes = L::BYTES;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv_attention_kernel<D, Q8>, a, g, tk, tv);
  note_launches(1);
  // items of up to that many key tiles are never cut
  if (e != cudaSuccess || a.most <= g.merge * TILE) return e;
  cfg.gridDim = dim3(ctas - 1, min(static_cast<long long>(a.T) * g.group, static_cast<long long>(MERGE_Y)));
  cfg.blockDim = dim3(32 * MERGE_WARPS);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, kv_merge_kernel<D>, g);
  note_launches(1);
  return e;
}

}  // namespace

int num_sms();
unsigned long long wait_limit_ns();

cudaError_t launch_kv_expand(const kv::Args& a, uint16_t* k, uint16_t* v, int tile, int tiles, cudaStream_t s);

// Bytes of keys (or values) when an e4m3 cache is to be expanded to bf16 before an attention, else 0.  The
// attention of a pair of query tiles expands its keys and values on chip, every pair the same ones: from two
// pairs per sequence on, on average, one pass over the cache before it costs less (six chunks of 440 to 1777
// tokens over 1K to 10K: 457 us on chip, 335 us expanded first).  What the sequences' tables have room for is
// reserved, up to 8 GiB.  Going by the average has a price where one long chunk comes with single tokens over
// long caches, which are expanded too (4096 tokens and 15 single ones over 32K: 336 us, in two calls 190).
size_t kv_expanded_bytes(const kv::Args& a, bool q8, int q_heads) {
  if (!q8 || a.B > 65535 || static_cast<long long>(a.T) * (q_heads / a.heads) < 4ll * TILE * a.B) return 0;
  const long long rows = static_cast<long long>(a.B) * ((a.most + TILE - 1) / TILE) * TILE * a.heads;
  return rows < (1ll << 31) && rows * a.d <= (1ll << 31) ? rows * a.d * 2 : 0;
}

size_t kv_attention_workspace_bytes(const kv::Args& a, bool q8, int q_heads) {
  const size_t slot = (a.d == 64 ? slot_floats<64>() : slot_floats<128>()) * sizeof(float);
  return num_sms() * (sizeof(int4) + 2 * slot) + 2 * kv_expanded_bytes(a, q8, q_heads);
}

cudaError_t launch_kv_attention(const kv::Args& args, bool q8, const uint16_t* q, long long q_token, long long q_head,
                                int q_heads, float scale, uint16_t* out, float* lse, void* ws, cudaStream_t s) {
  kv::Args a = args;
  const size_t wide = kv_expanded_bytes(a, q8, q_heads);
  if (wide) {
    // the expanded cache: pages of TILE tokens in order
    uint16_t* k = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + kv_attention_workspace_bytes(a, false, q_heads));
    uint16_t* v = k + wide / 2;
    const int tiles = (a.most + TILE - 1) / TILE;
    const cudaError_t e = launch_kv_expand(a, k, v, TILE, tiles, s);
    if (e != cudaSuccess) return e;
    a.k = k;
    a.v = v;
    a.page_size = TILE;
    a.table_width = tiles;
    a.num_pages = a.B * tiles;
    a.in_order = true;
    q8 = false;
  }
  AttnArgs g;
  g.q = q;
  g.q_token = q_token;
  g.q_head = q_head;
  g.out = out;
  g.lse = lse;
  const int ctas = num_sms();
  g.joins = static_cast<int4*>(ws);
  g.part = reinterpret_cast<float*>(g.joins + ctas);
  g.scale_log2 = scale * 1.44269504088896341f;
  g.q_heads = q_heads;
  g.group = q_heads / a.heads;
  g.tpt = TILE / g.group;
  // pairs of tiles; but with so few of them that half of the SMs would have none, single tiles (a 512-token
  // prompt 20.5 -> 18.0 us, over 8000 cached tokens 64 -> 57 us, a 2048-token one 50 us as pairs, 58 single)
  const long long pairs = (a.T + 2ll * g.tpt - 1) / (2 * g.tpt) * a.heads;
  g.tokens = pairs <= num_sms() / 2 ? g.tpt : 2 * g.tpt;
  // cutting costs a tile's rows written, read and joined: with 16 in place of 10 (single tiles) and 6 (pairs)
  // 2048 tokens 49.8 -> 43.3 us, four chunks of 300 over 3000 39.7 -> 36.4 us, six e4m3 chunks 335 -> 328 us; the
  // few rows of decoding cost little (1, 3 and 6 measure alike)
  g.merge = static_cast<long long>(a.T) * g.group <= static_cast<long long>(THIN_ROWS) * a.B ? 3 : 16;
  g.chunk = a.page_size & -a.page_size;  // the largest power of two that divides the page
  if (g.chunk > TILE) g.chunk = TILE;
  g.chunk_log = __builtin_ctz(static_cast<unsigned>(g.chunk));
  g.per_page = a.page_size / g.chunk;
  const unsigned long long ns = wait_limit_ns();
  g.wait_cycles = ns > (~0ull) / 3 ? ~0ull : ns * 21 / 10;
  g.poll = ns < 20000ull;
  CUtensorMap tk, tv;
  memset(&tk, 0, sizeof(tk));
  memset(&tv, 0, sizeof(tv));
  const long long rows = static_cast<long long>(a.num_pages) * a.heads * a.page_size;
  if (!encode_pool(&tk, a.k, rows, a.d, g.chunk, q8) || !encode_pool(&tv, a.v, rows, a.d, g.chunk, q8))
    return cudaErrorInvalidValue;
  if (a.d == 64) return q8 ? launch<64, true>(a, g, tk, tv, ctas, s) : launch<64, false>(a, g, tk, tv, ctas, s);
  return q8 ? launch<128, true>(a, g, tk, tv, ctas, s) : launch<128, false>(a, g, tk, tv, ctas, s);
}

}  // namespace moe
