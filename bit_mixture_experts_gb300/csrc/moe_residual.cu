// A block's residual addition between the norm of what the block gave and the
// norm of what the next one takes:
//
//   z = y / rms(y) * (w_post + offset)      (or y itself)
//   r = scale x + gate z                    (the residual stream)
//   n = r / rms(r) * (w_pre + offset)       rms(v) = sqrt(mean v^2 + eps)
//
// where y is a dense tensor, or each token's weighted sum of its expert rows and
// its shared expert's row (moe_combine's sum, not rounded in between).
//
// One pass: a row's values stay in its threads' registers between the two
// sums, so every input is read and every output written once.  All sums and
// products in FP32, r and n rounded once.
#include "moe_ptx.cuh"
#include "moe_residual.cuh"

namespace moe {

int num_sms();
unsigned long long wait_limit_ns();

namespace {

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = __uint_as_float(u[q] << 16);
    f[2 * q + 1] = __uint_as_float(u[q] & 0xffff0000u);
  }
}

// Which eight channels of a row a thread's chunk c has: VEC eight in a row, else every `threads`-th.
template <bool VEC>
__device__ __forceinline__ int channel(int c, int j, int tid, int threads) {
  return VEC ? (c * threads + tid) * 8 + j : (c * 8 + j) * threads + tid;
}

// Eight values of a row of bf16 or float; those past H are 0.
template <bool VEC, bool F32>
__device__ __forceinline__ void load8(const void* row, int c, int tid, int threads, int H, float (&f)[8]) {
  if (VEC) {
    const int i = channel<true>(c, 0, tid, threads);
    if (i >= H) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = 0.f;
    } else if (F32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(row) + i);
      const float4 a = p[0], b = p[1];
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
      unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + i), f);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = channel<false>(c, j, tid, threads);
      f[j] = i >= H ? 0.f : F32 ? static_cast<const float*>(row)[i] : bf16_bits_to_float(static_cast<const uint16_t*>(row)[i]);
    }
  }
}

template <bool VEC, bool F32>
__device__ __forceinline__ void store8(void* row, int c, int tid, int threads, int H, const float (&f)[8]) {
  if (VEC) {
    const int i = channel<true>(c, 0, tid, threads);
    if (i >= H) return;
    if (F32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + i);
      p[0] = make_float4(f[0], f[1], f[2], f[3]);
      p[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + i) =
          make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = channel<false>(c, j, tid, threads);
      if (i >= H) continue;
      if (F32)
        static_cast<float*>(row)[i] = f[j];
      else
        static_cast<uint16_t*>(row)[i] = float_to_bf16_bits(f[j]);
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void load8_any(const void* row, bool f32, int c, int tid, int threads, int H, float (&f)[8]) {
  if (f32)
    load8<VEC, true>(row, c, tid, threads, H, f);
  else
    load8<VEC, false>(row, c, tid, threads, H, f);
}

// A norm's gains for a chunk.
template <bool VEC>
__device__ __forceinline__ void gains(const void* w, const ResidualArgs& p, int c, int tid, int threads, float (&f)[8]) {
  if (w) load8_any<VEC>(w, p.param_f32, c, tid, threads, p.H, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = w ? f[j] + p.offset : 1.f;
}

// Sum of v over the threads of the row; s: a float per warp of them.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* s, int warps) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  if (WARP) return v;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < warps; ++w) v += s[w];
  return v;
}

// WARP: a row per warp, else a row per block.  CH chunks of eight channels per thread.
template <bool VEC, bool X32, bool COMBINE, bool WARP, int CH>
__global__ void __launch_bounds__(WARP ? 256 : 1024) residual_kernel(const __grid_constant__ ResidualArgs p) {
  __shared__ float s_a[32], s_b[32];
  const int threads = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int t = WARP ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (t >= p.T) return;
  const int H = p.H, warps = threads >> 5;
  const size_t xs = static_cast<size_t>(t) * p.x_stride * (X32 ? 4 : 2);
  float y[CH][8], x[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) load8<VEC, X32>(static_cast<const uint8_t*>(p.x) + xs, c, tid, threads, H, x[c]);
  if (COMBINE) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) y[c][j] = 0.f;
    const int A = p.T * p.k;
    for (int j = 0; j <= p.k; ++j) {
      int row = A + t;
      float w = 1.f;
      if (j < p.k) {
        row = __ldg(p.inv_perm + static_cast<size_t>(t) * p.k + j);
        w = __ldg(p.topk_w + static_cast<size_t>(t) * p.k + j);
        if (row < 0 || row >= A) {
          set_device_error(p.err, MOE_DEV_BAD_INDEX);
          continue;
        }
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float v[8];
        load8<VEC, false>(p.y + row * p.y_stride, c, tid, threads, H, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[c][i] = fmaf(w, v[i], y[c][i]);
      }
    }
  } else if (p.y) {
#pragma unroll
    for (int c = 0; c < CH; ++c) load8<VEC, false>(p.y + t * p.y_stride, c, tid, threads, H, y[c]);
  }
  if (p.post) {
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(y[c][j], y[c][j], ss);
    ss = row_sum<WARP>(ss, s_a, warps);
    const float f = 1.0f / sqrtf(ss / static_cast<float>(H) + p.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float w[8];
      gains<VEC>(p.w_post, p, c, tid, threads, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[c][j] *= f * w[j];
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (p.gate) {
      const uint8_t* row = static_cast<const uint8_t*>(p.gate) + t * p.gate_token * (p.gate_f32 ? 4 : 2);
      float g[8];
      if (p.gate_channel) {
        load8_any<VEC>(row, p.gate_f32, c, tid, threads, H, g);
      } else {
        const float one = p.gate_f32 ? *reinterpret_cast<const float*>(row)
                                     : bf16_bits_to_float(*reinterpret_cast<const uint16_t*>(row));
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = one;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) y[c][j] *= g[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[c][j] = COMBINE || p.y ? fmaf(p.scale, x[c][j], y[c][j]) : p.scale * x[c][j];
      ss = fmaf(x[c][j], x[c][j], ss);
    }
  }
  if (p.r) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      store8<VEC, X32>(static_cast<uint8_t*>(p.r) + static_cast<size_t>(t) * p.r_stride * (X32 ? 4 : 2), c, tid, threads, H, x[c]);
  }
  if (!p.n) return;
  ss = row_sum<WARP>(ss, s_b, warps);
  const float f = 1.0f / sqrtf(ss / static_cast<float>(H) + p.eps);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float w[8];
    gains<VEC>(p.w_pre, p, c, tid, threads, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= x[c][j] * f;
    store8<VEC, false>(p.n + t * p.n_stride, c, tid, threads, H, w);
  }
}

// ---------------------------------------------------------------- many rows: a ring of rows in shared memory
// Persistent blocks; a stage is what a token needs (its row of x, its row or rows of y, its row of the gate),
// copied by bulk copies some tokens ahead, so that memory is busy while a row's two sums are taken.  Rows
// that do not start on 16 bytes are copied with what is around them in the same 16 bytes.  The gains stay in
// registers from row to row.

struct Ring {
  int stages, stage_bytes;
  int x_bytes, row_bytes;  // of a stage: room for a row of x, for one of y or of the gate
  unsigned long long wait_cycles;
  bool poll;  // the limit is too short for waits inside an instruction
};

constexpr int RING_MAX_STAGES = 8;
constexpr int RING_BYTES = 216 * 1024;  // of an SM's shared memory

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// A row of `len` bytes as the 16-byte pieces that hold it: returns their bytes.
__device__ __forceinline__ uint32_t pieces(const uint8_t* row, uint32_t len, const uint8_t** from) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(row), lo = at & ~static_cast<uintptr_t>(15);
  *from = reinterpret_cast<const uint8_t*>(lo);
  return static_cast<uint32_t>((at + len + 15 & ~static_cast<uintptr_t>(15)) - lo);
}

// Eight values of a row that lies `skip` bytes into a stage's piece `s`.
template <bool VEC, bool F32>
__device__ __forceinline__ void stage8(const uint8_t* s, uint32_t skip, int c, int tid, int threads, int H, float (&f)[8]) {
  load8<VEC, F32>(s + (VEC ? 0 : skip), c, tid, threads, H, f);
}

template <bool VEC, bool X32, bool COMBINE, int CH>
__global__ void __launch_bounds__(CH == 1 ? 256 : 512, CH == 1 ? 3 : 1)
    ring_kernel(const __grid_constant__ ResidualArgs p, const Ring g) {
  constexpr bool KEEP = CH <= 2;  // the gains in registers
  constexpr int XS = X32 ? 4 : 2;
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ __align__(8) uint64_t s_full[RING_MAX_STAGES];
  __shared__ float s_sum[2][2][32];
  __shared__ float s_w[RING_MAX_STAGES][32], s_gate[RING_MAX_STAGES];
  __shared__ uint32_t s_bad[RING_MAX_STAGES];
  const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x, warps = threads >> 5;
  const int H = p.H, A = p.T * p.k;
  const bool gate_rows = p.gate && p.gate_channel && p.gate_token != 0;
  const bool gate_values = p.gate && !gate_rows && p.gate_token != 0;  // one per token
  const int gs = p.gate_f32 ? 4 : 2;
  auto bar = [&](int st) -> uint32_t { return ptx::smem_u32(&s_full[st]); };
  auto row_at = [](const void* base, long long row, long long stride, int size) {
    return static_cast<const uint8_t*>(base) + row * stride * size;
  };

  if (tid == 0) {
    for (int i = 0; i < g.stages; ++i) ptx::mbar_init(bar(i), 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();

  // warp 0: token t's rows on their way into stage st; idx, w: lane j < k's row of y and its weight
  auto issue = [&](int st, int t, int idx, float w) {
    const uint32_t base = ptx::smem_u32(ring_smem) + st * g.stage_bytes;
    uint32_t mine = 0, len[3] = {0, 0, 0}, dst[3];
    const uint8_t* src[3];
    if (lane == 0) {
      dst[0] = base;
      len[0] = pieces(row_at(p.x, t, p.x_stride, XS), H * XS, &src[0]);
      if (gate_rows) {
        dst[1] = base + g.x_bytes;
        len[1] = pieces(row_at(p.gate, t, p.gate_token, gs), H * gs, &src[1]);
      }
      if (COMBINE || p.y) {
        dst[2] = base + g.stage_bytes - g.row_bytes;  // the shared row, or the only one
        len[2] = pieces(row_at(p.y, COMBINE ? A + t : t, p.y_stride, 2), H * 2, &src[2]);
      }
      mine = len[0] + len[1] + len[2];
    }
    uint32_t ylen = 0;
    const uint8_t* ysrc = nullptr;
    if (COMBINE) {
      const bool bad = lane < p.k && (idx < 0 || idx >= A);
      if (bad) set_device_error(p.err, MOE_DEV_BAD_INDEX);
      const uint32_t mask = __ballot_sync(0xffffffffu, bad);
      if (lane == 0) s_bad[st] = mask;
      s_w[st][lane] = w;
      if (lane < p.k && !bad) ylen = pieces(row_at(p.y, idx, p.y_stride, 2), H * 2, &ysrc);
      mine += ylen;
    }
    if (gate_values && lane == 0)
      s_gate[st] = p.gate_f32 ? static_cast<const float*>(p.gate)[t * p.gate_token]
                              : bf16_bits_to_float(static_cast<const uint16_t*>(p.gate)[t * p.gate_token]);
    const uint32_t bytes = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0)
      asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar(st)), "r"(bytes) : "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (len[i]) bulk_load(dst[i], src[i], len[i], bar(st));
    if (COMBINE && ylen) bulk_load(base + g.stage_bytes - (p.k + 1 - lane) * g.row_bytes, ysrc, ylen, bar(st));
  };
  auto load_index = [&](int t, int* idx, float* w) {
    *idx = 0;
    *w = 0.f;
    if (COMBINE && lane < p.k && t < p.T) {
      *idx = __ldg(p.inv_perm + static_cast<size_t>(t) * p.k + lane);
      *w = __ldg(p.topk_w + static_cast<size_t>(t) * p.k + lane);
    }
  };
  const int step = static_cast<int>(gridDim.x);
  int issued = 0;
  if (tid < 32) {
    for (; issued < g.stages; ++issued) {
      const int t = blockIdx.x + issued * step;
      if (t >= p.T) break;
      int idx;
      float w;
      load_index(t, &idx, &w);
      issue(issued, t, idx, w);
    }
  }
  // the gains: of y, with a gate that all tokens share, and of r
  const bool shared_gate = p.gate && p.gate_token == 0;
  auto gain_y = [&](int c, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 1.f;
    if (p.post) gains<VEC>(p.w_post, p, c, tid, threads, f);
    if (shared_gate && p.gate_channel) {
      float x[8];
      load8_any<VEC>(p.gate, p.gate_f32, c, tid, threads, H, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= x[j];
    } else if (shared_gate) {
      const float x = p.gate_f32 ? *static_cast<const float*>(p.gate) : bf16_bits_to_float(*static_cast<const uint16_t*>(p.gate));
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= x;
    }
  };
  float ga[KEEP ? CH : 1][8], gb[KEEP ? CH : 1][8];
  if (KEEP) {
#pragma unroll
    for (int c = 0; c < (KEEP ? CH : 1); ++c) {
      gain_y(c, ga[c]);
      gains<VEC>(p.w_pre, p, c, tid, threads, gb[c]);
    }
  }
  __syncthreads();  // the first stages' weights and gates

  bool dead = false;
  int st = 0, ph = 0;
  for (int i = 0, t = blockIdx.x; t < p.T; ++i, t += step) {
    int idx = 0;
    float w = 0.f;
    const int ahead = t + g.stages * step;
    if (tid < 32 && !dead) load_index(ahead, &idx, &w);
    if (!dead && !__all_sync(0xffffffffu, g.poll ? ptx::mbar_test_wait(bar(st), ph) : ptx::mbar_try_wait(bar(st), ph))) {
      const long long t0 = clock64();
      while (!__all_sync(0xffffffffu, g.poll ? ptx::mbar_test_wait(bar(st), ph) : ptx::mbar_try_wait(bar(st), ph))) {
        if (__any_sync(0xffffffffu, static_cast<unsigned long long>(clock64() - t0) > g.wait_cycles)) {
          set_device_error(p.err, MOE_DEV_TIMEOUT);
          dead = true;
          break;
        }
      }
    }
    const uint8_t* stage = ring_smem + st * g.stage_bytes;
    auto skip = [&](const void* base, long long row, long long stride, int size) {
      return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row_at(base, row, stride, size)) & 15u);
    };
    float x[CH][8], y[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) stage8<VEC, X32>(stage, skip(p.x, t, p.x_stride, XS), c, tid, threads, H, x[c]);
    if (COMBINE) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) y[c][j] = 0.f;
      const uint32_t bad = s_bad[st];
      const uint8_t* row = stage + g.stage_bytes - (p.k + 1) * g.row_bytes;
      for (int j = 0; j <= p.k; ++j, row += g.row_bytes) {
        float f = 1.f;
        uint32_t s = 0;
        if (j < p.k) {
          if (bad >> j & 1) continue;
          f = s_w[st][j];
          if (!VEC) s = skip(p.y, __ldg(p.inv_perm + static_cast<size_t>(t) * p.k + j), p.y_stride, 2);
        } else if (!VEC) {
          s = skip(p.y, A + t, p.y_stride, 2);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          float v[8];
          stage8<VEC, false>(row, s, c, tid, threads, H, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[c][e] = fmaf(f, v[e], y[c][e]);
        }
      }
    } else if (p.y) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        stage8<VEC, false>(stage + g.stage_bytes - g.row_bytes, skip(p.y, t, p.y_stride, 2), c, tid, threads, H, y[c]);
    }
    // The stage is free once every thread has read it: behind the first barrier, or where the gate's row is
    // read after that, behind the second.
    bool freed = false;
    auto refill = [&]() {
      freed = true;
      if (tid < 32 && !dead && ahead < p.T) {
        issue(st, ahead, idx, w);
        ++issued;
      }
    };
    float f = 1.f;
    if (p.post) {
      float ss = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(y[c][j], y[c][j], ss);
      ss = row_sum<false>(ss, s_sum[i & 1][0], warps);
      f = 1.0f / sqrtf(ss / static_cast<float>(H) + p.eps);
      if (!gate_rows && !gate_values) refill();
    }
    if (gate_values) f *= s_gate[st];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (COMBINE || p.y) {
        float a[8];
        if (!KEEP) gain_y(c, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[c][j] *= f * (KEEP ? ga[KEEP ? c : 0][j] : a[j]);
        if (gate_rows) {
          float v[8];
          const uint32_t s = skip(p.gate, t, p.gate_token, gs);
          if (p.gate_f32)
            stage8<VEC, true>(stage + g.x_bytes, s, c, tid, threads, H, v);
          else
            stage8<VEC, false>(stage + g.x_bytes, s, c, tid, threads, H, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[c][j] *= v[j];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[c][j] = COMBINE || p.y ? fmaf(p.scale, x[c][j], y[c][j]) : p.scale * x[c][j];
        ss = fmaf(x[c][j], x[c][j], ss);
      }
    }
    if (p.r && !dead) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        store8<VEC, X32>(static_cast<uint8_t*>(p.r) + t * p.r_stride * XS, c, tid, threads, H, x[c]);
    }
    if (p.n) {
      ss = row_sum<false>(ss, s_sum[i & 1][1], warps);
      if (!freed) refill();
      f = 1.0f / sqrtf(ss / static_cast<float>(H) + p.eps);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float b[8];
        if (!KEEP) gains<VEC>(p.w_pre, p, c, tid, threads, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = x[c][j] * f * (KEEP ? gb[KEEP ? c : 0][j] : b[j]);
        if (!dead) store8<VEC, false>(p.n + t * p.n_stride, c, tid, threads, H, b);
      }
    } else if (!freed) {
      __syncthreads();
      refill();
    }
    if (++st == g.stages) {
      st = 0;
      ph ^= 1;
    }
  }
  // after a wait that gave up: no copy outlives the block
  if (tid == 0 && dead)
    for (int i = max(0, issued - g.stages); i < issued; ++i) {
      const long long t0 = clock64();
      while (!ptx::mbar_try_wait_sleep(bar(i % g.stages), (i / g.stages) & 1, 20000u) && clock64() - t0 < 20000000ll) {
      }
    }
}

template <bool VEC, bool X32, bool COMBINE, int CH>
cudaError_t launch_ring(const ResidualArgs& p, Ring g, int threads, cudaStream_t s) {
  const void* kernel = reinterpret_cast<const void*>(ring_kernel<VEC, X32, COMBINE, CH>);
  // as many blocks per SM as leave two stages to each
  const int room = RING_BYTES / (CH == 1 ? max(1, min(3, RING_BYTES / (2 * g.stage_bytes))) : 1);
  g.stages = min(RING_MAX_STAGES, room / g.stage_bytes);
  const size_t smem = static_cast<size_t>(g.stages) * g.stage_bytes;
  cudaError_t e = ensure_dyn_smem(kernel, smem);
  int per_sm = 0;
  if (e == cudaSuccess) e = cached_occupancy(kernel, threads, smem, &per_sm);
  if (e != cudaSuccess) return e;
  if (per_sm < 1) return cudaErrorInvalidValue;
  ring_kernel<VEC, X32, COMBINE, CH><<<min(p.T, num_sms() * per_sm), threads, smem, s>>>(p, g);
  note_launches(1);
  return cudaGetLastError();
}

template <bool VEC, bool X32, bool COMBINE>
cudaError_t launch_any_ring(const ResidualArgs& p, const Ring& g, cudaStream_t s) {
  const int chunks = ceil_div(p.H, 8);
  if (chunks <= 256) return launch_ring<VEC, X32, COMBINE, 1>(p, g, ceil_div(chunks, 32) * 32, s);
  if (chunks <= 1024) return launch_ring<VEC, X32, COMBINE, 2>(p, g, ceil_div(chunks, 64) * 32, s);
  return launch_ring<VEC, X32, COMBINE, 4>(p, g, ceil_div(chunks, 128) * 32, s);
}

constexpr int RING_MIN_CHUNKS = 64, RING_MAX_CHUNKS = 2048, RING_MIN_ROWS = 2;

template <bool VEC, bool X32, bool COMBINE>
cudaError_t launch(const ResidualArgs& p, cudaStream_t s) {
  const int chunks = ceil_div(p.H, 8);
  // a ring where it holds two tokens and there are tokens enough to keep it full
  Ring g;
  g.x_bytes = (p.H * (X32 ? 4 : 2) + 15) / 16 * 16 + (VEC ? 0 : 16);
  const bool gate_rows = p.gate && p.gate_channel && p.gate_token != 0;
  const int gate_bytes = gate_rows ? (p.H * (p.gate_f32 ? 4 : 2) + 15) / 16 * 16 + (VEC ? 0 : 16) : 0;
  g.row_bytes = (p.H * 2 + 15) / 16 * 16 + (VEC ? 0 : 16);
  g.stage_bytes = (g.x_bytes + gate_bytes + (COMBINE ? p.k + 1 : p.y ? 1 : 0) * g.row_bytes + 127) / 128 * 128;
  g.stages = 0;
  if (2 * g.stage_bytes <= RING_BYTES && chunks > RING_MIN_CHUNKS && chunks <= RING_MAX_CHUNKS &&
      p.T > RING_MIN_ROWS * num_sms()) {
    const unsigned long long ns = wait_limit_ns();
    g.wait_cycles = ns > (~0ull) / 3 ? ~0ull : ns * 21 / 10;
    g.poll = ns < 20000ull;
    return launch_any_ring<VEC, X32, COMBINE>(p, g, s);
  }
  if (chunks <= 64) {
    const int rows = 8;
    if (chunks <= 32)
      residual_kernel<VEC, X32, COMBINE, true, 1><<<ceil_div(p.T, rows), 32 * rows, 0, s>>>(p);
    else
      residual_kernel<VEC, X32, COMBINE, true, 2><<<ceil_div(p.T, rows), 32 * rows, 0, s>>>(p);
  } else if (chunks <= 1024) {
    residual_kernel<VEC, X32, COMBINE, false, 1><<<p.T, ceil_div(chunks, 32) * 32, 0, s>>>(p);
  } else if (chunks <= 2048) {
    residual_kernel<VEC, X32, COMBINE, false, 2><<<p.T, ceil_div(chunks, 64) * 32, 0, s>>>(p);
  } else {
    residual_kernel<VEC, X32, COMBINE, false, 4><<<p.T, ceil_div(chunks, 128) * 32, 0, s>>>(p);
  }
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace

constexpr int RESIDUAL_MAX_H = 32768;

int residual_max_h() { return RESIDUAL_MAX_H; }

cudaError_t launch_residual(const ResidualArgs& p, bool combine, bool x32, cudaStream_t s) {
  // rows in pieces of eight values, if every row of every tensor starts on 16 bytes
  auto ok = [](const void* ptr, long long stride, int size) {
    return (reinterpret_cast<uintptr_t>(ptr) | static_cast<uintptr_t>(stride * size)) % 16 == 0;
  };
  const int xs = x32 ? 4 : 2, ps = p.param_f32 ? 4 : 2;
  const bool vec = p.H % 8 == 0 && ok(p.x, p.x_stride, xs) && ok(p.y, p.y_stride, 2) && ok(p.r, p.r_stride, xs) &&
                   ok(p.n, p.n_stride, 2) && ok(p.w_pre, 0, ps) && ok(p.w_post, 0, ps) &&
                   (!p.gate_channel || ok(p.gate, p.gate_token, p.gate_f32 ? 4 : 2));
  if (vec) {
    if (combine) return x32 ? launch<true, true, true>(p, s) : launch<true, false, true>(p, s);
    return x32 ? launch<true, true, false>(p, s) : launch<true, false, false>(p, s);
  }
  if (combine) return x32 ? launch<false, true, true>(p, s) : launch<false, false, true>(p, s);
  return x32 ? launch<false, true, false>(p, s) : launch<false, false, false>(p, s);
}

}  // namespace moe
