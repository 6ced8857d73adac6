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
#include "moe_residual.cuh"

namespace moe {

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

template <bool VEC, bool X32, bool COMBINE>
cudaError_t launch(const ResidualArgs& p, cudaStream_t s) {
  const int chunks = ceil_div(p.H, 8);
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
