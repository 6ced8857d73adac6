// The residual addition over few or short rows, and which kernel a call takes.
#pragma once
#include "moe_residual_ring.cuh"

namespace moe {
namespace residual {

// ---------------------------------------------------------------- a row per block
// For few rows (one token: the chain of latencies of a launch, a load and two sums) and for rows that no ring
// holds.
template <bool VEC, bool X32, bool COMBINE, int CH>
__global__ void __launch_bounds__(1024) row_kernel(const __grid_constant__ ResidualArgs p) {
  __shared__ float s_sum[2][32];
  constexpr int XS = X32 ? 4 : 2;
  const int tid = threadIdx.x, threads = blockDim.x, warps = threads >> 5, t = blockIdx.x, H = p.H;
  const bool add = COMBINE || p.y;
  wait_for_earlier();
  auto row_sum = [&](float v, float* s) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if ((tid & 31) == 0) s[tid >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < warps; ++w) v += s[w];
    return v;
  };
  constexpr bool EARLY = CH == 1;  // all loads before the first sum; else registers are for y, then for x
  float y[CH][8], x[CH][8], a[8];
  auto load_x = [&]() {
    const uint8_t* x_at = row_of<XS>(static_cast<const uint8_t*>(p.x), t, p.x_stride);
#pragma unroll
    for (int c = 0; c < CH; ++c) load8<VEC, X32>(x_at, c, tid, threads, H, x[c]);
  };
  auto load_a = [&](int c) {
    gains_y<VEC>(p, c, tid, threads, a);
    if (gate_is_rows(p)) {
      float v[8];
      load8_any<VEC>(static_cast<const uint8_t*>(p.gate) + t * p.gate_token * (p.gate_f32 ? 4 : 2), p.gate_f32, c, tid,
                     threads, H, v);
      mul8(a, v, a);
    }
  };
  if (EARLY) load_x();
  if (COMBINE) {
    combine_rows<VEC, CH, CH == 1 && VEC ? 9 : 4>(p, t, tid, threads, y);
  } else if (p.y) {
#pragma unroll
    for (int c = 0; c < CH; ++c) load8<VEC, false>(row_of<2>(p.y, t, p.y_stride), c, tid, threads, H, y[c]);
  }
  float f = 1.f;
  if (add) {
    if (EARLY) load_a(0);
    f = token_gate(p, t);
  }
  if (p.post) {
    float sq[8] = {};
#pragma unroll
    for (int c = 0; c < CH; ++c) fma8(sq, y[c], y[c], sq);
    f *= rsqrtf(row_sum(sum8(sq), s_sum[0]) / static_cast<float>(H) + p.eps);
  }
  if (!EARLY && add) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      load_a(c);
      mul8(y[c], a, y[c]);
    }
  }
  if (!EARLY) load_x();
  float sq[8] = {};
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    mul8(x[c], p.scale, x[c]);
    if (add) {
      if (EARLY) mul8(y[c], a, y[c]);
      fma8(x[c], f, y[c], x[c]);
    }
    fma8(sq, x[c], x[c], sq);
  }
  if (EARLY && p.n) gains<VEC>(p.w_pre, p, 0, tid, threads, a);
  if (p.r) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      store8<VEC, X32>(row_of<XS>(static_cast<uint8_t*>(p.r), t, p.r_stride), c, tid, threads, H, x[c]);
  }
  if (!p.n) return;
  f = rsqrtf(row_sum(sum8(sq), s_sum[1]) / static_cast<float>(H) + p.eps);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (!EARLY) gains<VEC>(p.w_pre, p, c, tid, threads, a);
    mul8(x[c], f, x[c]);
    mul8(x[c], a, x[c]);
    store8<VEC, false>(row_of<2>(p.n, t, p.n_stride), c, tid, threads, H, x[c]);
  }
}

// ---------------------------------------------------------------- short rows: LANES lanes of a warp per row
// Persistent warps, the gains in registers; LANES x CH chunks hold a row.
template <bool VEC, bool X32, bool COMBINE, int LANES, int CH>
__global__ void __launch_bounds__(256, COMBINE ? 2 : 4) short_kernel(const __grid_constant__ ResidualArgs p) {
  constexpr int XS = X32 ? 4 : 2, ROWS = 32 / LANES;
  const int lane = threadIdx.x & 31, tid = lane % LANES, H = p.H;
  const bool add = COMBINE || p.y;
  const float inv_h = 1.0f / static_cast<float>(H);
  constexpr bool KEEP = CH == 1;  // the gains in registers
  wait_for_earlier();
  float ga[8], gb[8];
  if (KEEP) {
    gains_y<VEC>(p, 0, tid, LANES, ga);
    gains<VEC>(p.w_pre, p, 0, tid, LANES, gb);
  }
  auto row_sum = [&](float v) {
#pragma unroll
    for (int m = LANES / 2; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
  };
  const int step = static_cast<int>(gridDim.x) * 8 * ROWS;
  for (int t0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * ROWS; t0 < p.T; t0 += step) {
    const bool here = t0 + lane / LANES < p.T;  // (lanes of no row repeat the last one's)
    const int t = min(t0 + lane / LANES, p.T - 1);
    float x[CH][8], y[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c)
      load8<VEC, X32>(row_of<XS>(static_cast<const uint8_t*>(p.x), t, p.x_stride), c, tid, LANES, H, x[c]);
    if (COMBINE) {
      combine_rows<VEC, CH, CH == 1 ? 9 : 5>(p, t, tid, LANES, y);
    } else if (p.y) {
#pragma unroll
      for (int c = 0; c < CH; ++c) load8<VEC, false>(row_of<2>(p.y, t, p.y_stride), c, tid, LANES, H, y[c]);
    }
    float f = add ? token_gate(p, t) : 1.f;
    if (p.post) {
      float sq[8] = {};
#pragma unroll
      for (int c = 0; c < CH; ++c) fma8(sq, y[c], y[c], sq);
      f *= rsqrtf(fmaf(row_sum(sum8(sq)), inv_h, p.eps));
    }
    float sq[8] = {};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      mul8(x[c], p.scale, x[c]);
      if (add) {
        float a[8];
        if (!KEEP) gains_y<VEC>(p, c, tid, LANES, ga);
        mul8(a, f, ga);
        if (gate_is_rows(p)) {
          float v[8];
          load8_any<VEC>(static_cast<const uint8_t*>(p.gate) + t * p.gate_token * (p.gate_f32 ? 4 : 2), p.gate_f32, c, tid,
                         LANES, H, v);
          mul8(a, v, a);
        }
        fma8(x[c], a, y[c], x[c]);
      }
      fma8(sq, x[c], x[c], sq);
    }
    __syncwarp();  // an output may take an input's place: lanes that repeat a row have read it
    if (p.r && here) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        store8<VEC, X32>(row_of<XS>(static_cast<uint8_t*>(p.r), t, p.r_stride), c, tid, LANES, H, x[c]);
    }
    if (!p.n) continue;
    f = rsqrtf(fmaf(row_sum(sum8(sq)), inv_h, p.eps));
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (!KEEP) gains<VEC>(p.w_pre, p, c, tid, LANES, gb);
      mul8(x[c], f, x[c]);
      mul8(x[c], gb, x[c]);
      if (here) store8<VEC, false>(row_of<2>(p.n, t, p.n_stride), c, tid, LANES, H, x[c]);
    }
  }
}

template <bool VEC, bool X32, bool COMBINE, int LANES, int CH>
cudaError_t launch_short(const ResidualArgs& p, cudaStream_t s) {
  const auto kernel = short_kernel<VEC, X32, COMBINE, LANES, CH>;
  int per_sm = 0;
  const cudaError_t e = cached_occupancy(reinterpret_cast<const void*>(kernel), 256, 0, &per_sm);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return launch_early(kernel, min(ceil_div(p.T, 8 * 32 / LANES), num_sms() * per_sm), 256, 0, s, p);
}

// Rows of up to 512 channels: lanes of a warp (131072 rows of 384 88 us, in the ring 108).  More: a block each as long
// as all of them run at once, else the ring (760 rows of 2048 channels 3.95 us in blocks, 4.85 in the ring; 912 5.4 and
// 4.8; 456 combined 5.8 and 6.7, 912 9.5 and 8.9; 152 of 8192 4.3 and 4.3, 200 7.3 and 5.7).
constexpr int SHORT_CHUNKS = 64, RING_MAX_CHUNKS = 2048;

template <bool VEC, bool X32, bool COMBINE>
cudaError_t launch(const ResidualArgs& p, cudaStream_t s) {
  const int chunks = ceil_div(p.H, 8);
  if (chunks <= SHORT_CHUNKS) {
    if (chunks <= 4) return launch_short<VEC, X32, COMBINE, 4, 1>(p, s);
    if (chunks <= 8) return launch_short<VEC, X32, COMBINE, 8, 1>(p, s);
    if (chunks <= 16) return launch_short<VEC, X32, COMBINE, 16, 1>(p, s);
    if (chunks <= 32) return launch_short<VEC, X32, COMBINE, 32, 1>(p, s);
    return launch_short<VEC, X32, COMBINE, 32, 2>(p, s);
  }
  const int ch = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : 4, threads = ceil_div(chunks, 32 * ch) * 32;
  const auto kernel = ch == 1   ? row_kernel<VEC, X32, COMBINE, 1>
                      : ch == 2 ? row_kernel<VEC, X32, COMBINE, 2>
                                : row_kernel<VEC, X32, COMBINE, 4>;
  if (chunks <= RING_MAX_CHUNKS) {
    int per_sm = 0;
    cudaError_t e = cached_occupancy(reinterpret_cast<const void*>(kernel), threads, 0, &per_sm);
    if (e != cudaSuccess) return e;
    if (p.T > num_sms() * per_sm) {
      bool ran;
      e = try_ring<VEC, X32, COMBINE>(p, s, &ran);
      if (e != cudaSuccess || ran) return e;
    }
  }
  note_launches(1);
  return launch_early(kernel, p.T, threads, 0, s, p);
}

}  // namespace residual
}  // namespace moe
