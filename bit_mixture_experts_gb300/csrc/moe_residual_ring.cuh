// The residual addition over many rows: a ring of rows in shared memory.
//
// Persistent blocks: one warp issues bulk copies some rows ahead, so that
// memory is busy while the others take a row's two sums; the gains stay in their
// registers from row to row.  A stage is all that a token needs (its row of x,
// its row or rows of y, its row of the gate); where two such stages do not fit, a
// stage is one row (ROWS).  Rows that do not start on 16 bytes are copied with
// what is around them in the same 16 bytes, and read from there and written
// element by element.
//
// What bounds it: memory.  16384 rows of 8192 channels, float32 stream, a gate
// per element: 279 us, 0.99 of the copy rate; the combine of 16384 tokens, nine
// rows of 2048 each: 138 us, 1.0 of it; 4096 rows of 2048: 15 us where the copy
// rate allows 9.9 (ramp and tail of a short call).  Rows that are not aligned:
// the elements' loads and stores, 50000 rows of 1999 205 us, 0.57 of the rate (by
// way of shared memory, in whole pieces, the outputs took two barriers more:
// 253 us).
#pragma once
#include "moe_launch.cuh"
#include "moe_ptx.cuh"
#include "moe_residual_dev.cuh"

namespace moe {

int num_sms();
unsigned long long wait_limit_ns();

namespace residual {

struct Ring {
  int stages, stage_bytes;
  int x_bytes, row_bytes;  // room for a row of x, for one of y or of the gate
  unsigned long long wait_cycles;
  bool poll;  // the limit is too short for waits inside an instruction
};

constexpr int RING_MAX_STAGES = 8, RING_MAX_ROWS = 16;  // stages of a token, of a row
constexpr int RING_BYTES = 216 * 1024;  // of an SM's shared memory
// Bytes per SM on their way ahead of use where as much is written as read: enough to cover the latency, and no more,
// or reads and writes come in bursts of their own (4096 rows of 2048 channels 15.4 us with two stages per block,
// 17.6 with six; 8192 rows of 16384 199 and 261).
constexpr int RING_AHEAD = 64 * 1024;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// A row of `len` bytes as the 16-byte pieces that hold it: returns their bytes.
__device__ __forceinline__ uint32_t pieces(const uint8_t* row, uint32_t len, const uint8_t** from) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(row), lo = at & ~static_cast<uintptr_t>(15);
  *from = reinterpret_cast<const uint8_t*>(lo);
  return static_cast<uint32_t>(((at + len + 15) & ~static_cast<uintptr_t>(15)) - lo);
}

__device__ __forceinline__ uint32_t skip_of(const void* row) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u); }

// A row's sum of squares from its consumer warps' parts; s: 16 floats, zeros behind the last warp's.
__device__ __forceinline__ float ring_sum(float v, float* s, int warps) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  ptx::named_bar_sync(1, 32 * warps);
  float4 x = *reinterpret_cast<const float4*>(s);
  v = (x.x + x.y) + (x.z + x.w);
#pragma unroll 1
  for (int w = 4; w < warps; w += 4) {
    x = *reinterpret_cast<const float4*>(s + w);
    v += (x.x + x.y) + (x.z + x.w);
  }
  return v;
}

// Blocks per SM that registers have to leave room for.
__host__ __device__ constexpr int ring_blocks(int ch, int threads) {
  return threads <= 160 ? 4 : threads > 288 ? 1 : ch == 1 ? 3 : 2;
}

// Consumer warps, and behind them one that issues the copies.  NT: threads at most.
template <bool VEC, bool X32, bool COMBINE, int CH, int NT, bool ROWS>
__global__ void __launch_bounds__(NT, ring_blocks(CH, NT))
    ring_kernel(const __grid_constant__ ResidualArgs p, const Ring g) {
  constexpr bool KEEP = CH <= 2;  // the gains in registers; else those are for y and its gains, then for x and its
  constexpr int XS = X32 ? 4 : 2, MOST = ROWS ? RING_MAX_ROWS : RING_MAX_STAGES;
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ __align__(8) uint64_t s_full[MOST], s_empty[MOST];
  __shared__ __align__(16) float s_sum[2][2][16];
  __shared__ float s_w[ROWS ? 1 : MOST][32], s_one[MOST];  // weights; a row's weight or gate
  __shared__ uint32_t s_bad[MOST];
  const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x - 32, warps = threads >> 5;
  const int H = p.H, A = p.T * p.k, step = static_cast<int>(gridDim.x);
  const bool gate_rows = gate_is_rows(p), gate_values = p.gate && !p.gate_channel && p.gate_token != 0;
  const int gs = p.gate_f32 ? 4 : 2;
  auto full = [&](int st) -> uint32_t { return ptx::smem_u32(&s_full[st]); };
  auto empty = [&](int st) -> uint32_t { return ptx::smem_u32(&s_empty[st]); };
  auto gate_row = [&](int t) { return static_cast<const uint8_t*>(p.gate) + t * p.gate_token * gs; };
  // bounded wait of a whole warp; false when it gave up (recorded)
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, g.poll ? ptx::mbar_test_wait(bar, parity) : ptx::mbar_try_wait(bar, parity))) return true;
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, g.poll ? ptx::mbar_test_wait(bar, parity) : ptx::mbar_try_wait(bar, parity))) {
      if (__any_sync(0xffffffffu, static_cast<unsigned long long>(clock64() - t0) > g.wait_cycles)) {
        set_device_error(p.err, MOE_DEV_TIMEOUT);
        return false;
      }
    }
    return true;
  };
  // the stages in turn
  struct Turn {
    int st, ph;
    __device__ __forceinline__ void next(int stages) {
      if (++st == stages) {
        st = 0;
        ph ^= 1;
      }
    }
  } turn = {0, 0};

  if (tid == 0) {
    for (int i = 0; i < g.stages; ++i) {
      ptx::mbar_init(full(i), 1);
      ptx::mbar_init(empty(i), warps);
    }
    ptx::fence_mbar_init();
  }
  if (tid < 64) s_sum[tid >> 5][tid >> 4 & 1][tid & 15] = 0.f;
  __syncthreads();
  wait_for_earlier();

  if (tid >= threads) {
    // ------------------------------------------------ copies, a lane per row of a token's y
    auto load_index = [&](int t, int* idx, float* w) {
      *idx = 0;
      *w = 0.f;
      if (COMBINE && lane < p.k && t < p.T) {
        *idx = __ldg(p.inv_perm + static_cast<size_t>(t) * p.k + lane);
        *w = __ldg(p.topk_w + static_cast<size_t>(t) * p.k + lane);
      }
    };
    auto expect = [&](uint32_t bytes) {
      __syncwarp();  // every lane's weight is written before the stage is announced by one (reductions do not order memory)
      if (lane == 0)
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full(turn.st)), "r"(bytes) : "memory");
      __syncwarp();
    };
    int idx, issued = 0;
    float w;
    bool ok = true;
    load_index(blockIdx.x, &idx, &w);
    for (int t = blockIdx.x; ok && t < p.T; t += step) {
      int next_idx;
      float next_w;
      load_index(t + step, &next_idx, &next_w);
      const bool bad = COMBINE && lane < p.k && (idx < 0 || idx >= A);
      if (bad) set_device_error(p.err, MOE_DEV_BAD_INDEX);
      const uint32_t mask = __ballot_sync(0xffffffffu, bad);
      if (ROWS) {
        // in the order in which they are used: y's rows, the gate's, x's
        const int ys = COMBINE ? p.k + 1 : p.y ? 1 : 0, rows = ys + (gate_rows ? 1 : 0) + 1;
        // (several at a time where there are stages enough, a lane each: one after the other they took 860 cycles a row)
        const int each = max(1, min(4, g.stages / 4));
        for (int r0 = 0; ok && r0 < rows; r0 += each) {
          const int n = min(each, rows - r0), r = r0 + lane;
          Turn mine = turn;
          for (int q = 0; ok && q < n; ++q) {
            ok = issued + q < g.stages || wait(empty(turn.st), turn.ph ^ 1);
            turn.next(g.stages);
            if (q < lane) mine = turn;
          }
          if (!ok) break;
          const int at = __shfl_sync(0xffffffffu, idx, r & 31);
          const float its = __shfl_sync(0xffffffffu, w, r & 31);
          if (lane < n) {
            const uint8_t* src = nullptr;
            uint32_t len = 0;
            float one = 1.f;
            if (r < ys) {
              if (COMBINE && r < p.k) one = its;
              if (!(COMBINE && r < p.k && mask >> r & 1))
                len = pieces(row_of<2>(p.y, COMBINE ? r < p.k ? at : A + t : t, p.y_stride), H * 2, &src);
            } else if (r + 1 < rows) {
              len = pieces(gate_row(t), H * gs, &src);
            } else {
              len = pieces(row_of<XS>(static_cast<const uint8_t*>(p.x), t, p.x_stride), H * XS, &src);
              one = token_gate(p, t);
            }
            s_one[mine.st] = one;
            s_bad[mine.st] = len == 0;
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full(mine.st)), "r"(len) : "memory");
            if (len) bulk_load(ptx::smem_u32(ring_smem) + mine.st * g.stage_bytes, src, len, full(mine.st));
          }
          __syncwarp();
          issued += n;
        }
      } else {
        const float one = token_gate(p, t);
        ok = issued < g.stages || wait(empty(turn.st), turn.ph ^ 1);
        if (!ok) break;
        const uint32_t base = ptx::smem_u32(ring_smem) + turn.st * g.stage_bytes;
        uint32_t len[3] = {0, 0, 0}, ylen = 0;
        const uint8_t *src[3] = {nullptr, nullptr, nullptr}, *ysrc = nullptr;
        if (lane == 0) {
          len[0] = pieces(row_of<XS>(static_cast<const uint8_t*>(p.x), t, p.x_stride), H * XS, &src[0]);
          if (gate_rows) len[1] = pieces(gate_row(t), H * gs, &src[1]);
          // the shared row, or the only one
          if (COMBINE || p.y) len[2] = pieces(row_of<2>(p.y, COMBINE ? A + t : t, p.y_stride), H * 2, &src[2]);
          s_one[turn.st] = one;
          s_bad[turn.st] = mask;
        }
        if (COMBINE) {
          s_w[ROWS ? 0 : turn.st][lane] = w;
          if (lane < p.k && !bad) ylen = pieces(row_of<2>(p.y, idx, p.y_stride), H * 2, &ysrc);
        }
        expect(__reduce_add_sync(0xffffffffu, len[0] + len[1] + len[2] + ylen));
        const uint32_t dst[3] = {base, base + g.x_bytes, base + g.stage_bytes - g.row_bytes};
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (len[i]) bulk_load(dst[i], src[i], len[i], full(turn.st));
        if (COMBINE && ylen) bulk_load(base + g.stage_bytes - (p.k + 1 - lane) * g.row_bytes, ysrc, ylen, full(turn.st));
        __syncwarp();
        turn.next(g.stages);
        ++issued;
      }
      idx = next_idx;
      w = next_w;
    }
    // no copy outlives the block, whatever the consumers did (at once unless a wait gave up)
    if (lane == 0)
      for (int i = max(0, issued - g.stages); i < issued; ++i) {
        const long long t0 = clock64();
        while (!ptx::mbar_try_wait_sleep(full(i % g.stages), (i / g.stages) & 1, 20000u) && clock64() - t0 < 20000000ll) {
        }
      }
    return;
  }

  // -------------------------------------------------- a row at a time
  float ga[KEEP ? CH : 1][8], gb[KEEP ? CH : 1][8];
  if (KEEP) {
#pragma unroll
    for (int c = 0; c < (KEEP ? CH : 1); ++c) {
      gains_y<VEC>(p, c, tid, threads, ga[c]);
      gains<VEC>(p.w_pre, p, c, tid, threads, gb[c]);
    }
  }
  const bool add = COMBINE || p.y;
  const float inv_h = 1.0f / static_cast<float>(H);
  bool dead = false;
  auto take = [&]() -> const uint8_t* {
    // A warp whose wait gave up goes on without waiting or writing, so that none is left at a barrier; and without
    // releasing stages, so that none is filled again before its last copies have landed.
    if (!dead) dead = !wait(full(turn.st), turn.ph);
    return ring_smem + turn.st * g.stage_bytes;
  };
  auto give = [&]() {
    __syncwarp();
    if (lane == 0 && !dead) ptx::mbar_arrive(empty(turn.st));
    turn.next(g.stages);
  };
  for (int i = 0, t = blockIdx.x; t < p.T; ++i, t += step) {
    float x[CH][8], y[CH][8];
    float one = 1.f;  // the token's gate
    const uint8_t* stage = nullptr;
    const uint8_t* x_at = row_of<XS>(static_cast<const uint8_t*>(p.x), t, p.x_stride);
    if (!ROWS) {
      stage = take();
      one = gate_values ? s_one[turn.st] : 1.f;
      if (KEEP) {
#pragma unroll
        for (int c = 0; c < CH; ++c) load8<VEC, X32>(stage + (VEC ? 0 : skip_of(x_at)), c, tid, threads, H, x[c]);
      }
    }
    if (COMBINE) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) y[c][j] = 0.f;
      const uint32_t bad = ROWS ? 0 : s_bad[turn.st];
      const uint8_t* row = ROWS ? nullptr : stage + g.stage_bytes - (p.k + 1) * g.row_bytes;
#pragma unroll 1
      for (int j = 0; j <= p.k; ++j) {
        if (ROWS) row = take();
        if (ROWS ? s_bad[turn.st] == 0 : !(j < p.k && bad >> j & 1)) {
          const float f = ROWS ? s_one[turn.st] : j < p.k ? s_w[ROWS ? 0 : turn.st][j] : 1.f;
          uint32_t s = 0;
          if (!VEC) s = skip_of(row_of<2>(p.y, j < p.k ? __ldg(p.inv_perm + static_cast<size_t>(t) * p.k + j) : A + t, p.y_stride));
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            float v[8];
            load8<VEC, false>(row + s, c, tid, threads, H, v);
            fma8(y[c], f, v, y[c]);
          }
        }
        if (ROWS)
          give();
        else
          row += g.row_bytes;
      }
    } else if (p.y) {
      const uint8_t* row = ROWS ? take() : stage + g.stage_bytes - g.row_bytes;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        load8<VEC, false>(row + (VEC ? 0 : skip_of(row_of<2>(p.y, t, p.y_stride))), c, tid, threads, H, y[c]);
      if (ROWS) give();
    }
    if (!ROWS && KEEP && !gate_rows) give();
    float f = 1.f;
    if (p.post) {
      float sq[8] = {};
#pragma unroll
      for (int c = 0; c < CH; ++c) fma8(sq, y[c], y[c], sq);
      f = rsqrtf(fmaf(ring_sum(sum8(sq), s_sum[i & 1][0], warps), inv_h, p.eps));
    }
    if (add) {
      f *= one;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float a[8];
        if (!KEEP) gains_y<VEC>(p, c, tid, threads, a);
        mul8(y[c], f, y[c]);
        mul8(y[c], KEEP ? ga[KEEP ? c : 0] : a, y[c]);
      }
      if (gate_rows) {
        const uint8_t* row = (ROWS ? take() : stage + g.x_bytes) + (VEC ? 0 : skip_of(gate_row(t)));
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          float v[8];
          if (p.gate_f32)
            load8<VEC, true>(row, c, tid, threads, H, v);
          else
            load8<VEC, false>(row, c, tid, threads, H, v);
          mul8(y[c], v, y[c]);
        }
        if (ROWS || KEEP) give();
      }
    }
    if (ROWS || !KEEP) {
      const uint8_t* row = ROWS ? take() : stage;
      if (ROWS && gate_values && add) one = s_one[turn.st];
#pragma unroll
      for (int c = 0; c < CH; ++c) load8<VEC, X32>(row + (VEC ? 0 : skip_of(x_at)), c, tid, threads, H, x[c]);
      give();
    }
    float sq[8] = {};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      mul8(x[c], p.scale, x[c]);
      if (add) {
        if (ROWS && gate_values)
          fma8(x[c], one, y[c], x[c]);
        else
#pragma unroll
          for (int j = 0; j < 8; ++j) x[c][j] += y[c][j];
      }
      fma8(sq, x[c], x[c], sq);
    }
    uint8_t* r_at = p.r ? row_of<XS>(static_cast<uint8_t*>(p.r), t, p.r_stride) : nullptr;
    uint8_t* n_at = p.n ? row_of<2>(p.n, t, p.n_stride) : nullptr;
    if (p.r && !dead) {
#pragma unroll
      for (int c = 0; c < CH; ++c) store8<VEC, X32>(r_at, c, tid, threads, H, x[c]);
    }
    if (p.n) {
      f = rsqrtf(fmaf(ring_sum(sum8(sq), s_sum[i & 1][1], warps), inv_h, p.eps));
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float b[8];
        if (!KEEP) gains<VEC>(p.w_pre, p, c, tid, threads, b);
        mul8(x[c], f, x[c]);
        mul8(x[c], KEEP ? gb[KEEP ? c : 0] : b, x[c]);
        if (!dead) store8<VEC, false>(n_at, c, tid, threads, H, x[c]);
      }
    }
  }
}

template <bool VEC, bool X32, bool COMBINE, int CH, int NT, bool ROWS>
cudaError_t launch_ring(const ResidualArgs& p, Ring g, int threads, cudaStream_t s) {
  const auto kernel = ring_kernel<VEC, X32, COMBINE, CH, NT, ROWS>;
  // as many blocks per SM as registers allow and leave two stages to each
  const int blocks = max(1, min(ring_blocks(CH, NT), RING_BYTES / (2 * g.stage_bytes)));
  g.stages = min(ROWS ? RING_MAX_ROWS : RING_MAX_STAGES, RING_BYTES / blocks / g.stage_bytes);
  if (!COMBINE) g.stages = min(g.stages, max(2, RING_AHEAD / blocks / g.stage_bytes));
  const size_t smem = static_cast<size_t>(g.stages) * g.stage_bytes;
  cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), smem);
  int per_sm = 0;
  if (e == cudaSuccess) e = cached_occupancy(reinterpret_cast<const void*>(kernel), threads + 32, smem, &per_sm);
  if (e != cudaSuccess) return e;
  if (per_sm < 1) return cudaErrorInvalidValue;
  note_launches(1);
  return launch_early(kernel, min(p.T, num_sms() * per_sm), threads + 32, smem, s, p, g);
}

// Runs the ring if it holds two stages; *ran tells.
template <bool VEC, bool X32, bool COMBINE>
cudaError_t try_ring(const ResidualArgs& p, cudaStream_t s, bool* ran) {
  Ring g;
  auto room = [](int bytes) { return (bytes + 15) / 16 * 16 + (VEC ? 0 : 16); };
  const bool gate_rows = p.gate && p.gate_channel && p.gate_token != 0;
  const int gate_bytes = gate_rows ? room(p.H * (p.gate_f32 ? 4 : 2)) : 0;
  g.x_bytes = room(p.H * (X32 ? 4 : 2));
  g.row_bytes = room(p.H * 2);
  g.stage_bytes = (g.x_bytes + gate_bytes + (COMBINE ? p.k + 1 : p.y ? 1 : 0) * g.row_bytes + 127) / 128 * 128;
  const bool rows = 2 * g.stage_bytes > RING_BYTES;
  if (rows) g.stage_bytes = (max(max(g.x_bytes, gate_bytes), g.row_bytes) + 127) / 128 * 128;
  *ran = 2 * g.stage_bytes <= RING_BYTES;
  if (!*ran) return cudaSuccess;
  const unsigned long long ns = wait_limit_ns();
  g.wait_cycles = ns > (~0ull) / 3 ? ~0ull : ns * 21 / 10;
  g.poll = ns < 20000ull;
  const int chunks = ceil_div(p.H, 8);
  const int one = ceil_div(chunks, 32) * 32, two = ceil_div(chunks, 64) * 32, four = ceil_div(chunks, 128) * 32;
  if (rows) {
    if (chunks <= 512) return launch_ring<VEC, X32, COMBINE, 1, 544, true>(p, g, one, s);
    if (chunks <= 1024) return launch_ring<VEC, X32, COMBINE, 2, 544, true>(p, g, two, s);
    return launch_ring<VEC, X32, COMBINE, 4, 544, true>(p, g, four, s);
  }
  if (chunks <= 128) return launch_ring<VEC, X32, COMBINE, 1, 160, false>(p, g, one, s);
  // a thread's work: with one chunk more warps share what a token's k + 1 rows or unaligned pieces take (4096
  // tokens of 2048 channels, nine rows: 34.6 us, two chunks 41), with two the sums of plain rows cost less
  // (12.2 us, one chunk 13.1)
  if constexpr (COMBINE || !VEC) {
    if (chunks <= 256) return launch_ring<VEC, X32, COMBINE, 1, 288, false>(p, g, one, s);
    if (chunks <= 512) return launch_ring<VEC, X32, COMBINE, 1, 544, false>(p, g, one, s);
  } else {
    if (chunks <= 256) return launch_ring<VEC, X32, COMBINE, 2, 160, false>(p, g, two, s);
    if (chunks <= 512) return launch_ring<VEC, X32, COMBINE, 2, 288, false>(p, g, two, s);
  }
  if (chunks <= 1024) return launch_ring<VEC, X32, COMBINE, 2, 544, false>(p, g, two, s);
  return launch_ring<VEC, X32, COMBINE, 4, 544, false>(p, g, four, s);
}

}  // namespace residual
}  // namespace moe
