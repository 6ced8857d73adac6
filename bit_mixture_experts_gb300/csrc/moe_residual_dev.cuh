// Device helpers of the residual addition's kernels: rows in pieces of eight
// values, arithmetic on two floats at a time.
#pragma once
#include <type_traits>

#include "moe_residual.cuh"

namespace moe {
namespace residual {

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

// Two floats at a time.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ void unpack2(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}

// d = a b + c and d = a b, eight values each.
__device__ __forceinline__ void fma8(float (&d)[8], const float (&a)[8], const float (&b)[8], const float (&c)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(pack2(a[j], a[j + 1])), "l"(pack2(b[j], b[j + 1])), "l"(pack2(c[j], c[j + 1])));
    unpack2(r, d[j], d[j + 1]);
  }
}

__device__ __forceinline__ void fma8(float (&d)[8], float a, const float (&b)[8], const float (&c)[8]) {
  const float x[8] = {a, a, a, a, a, a, a, a};
  fma8(d, x, b, c);
}

__device__ __forceinline__ void mul8(float (&d)[8], const float (&a)[8], const float (&b)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a[j], a[j + 1])), "l"(pack2(b[j], b[j + 1])));
    unpack2(r, d[j], d[j + 1]);
  }
}

__device__ __forceinline__ void mul8(float (&d)[8], float a, const float (&b)[8]) {
  const float x[8] = {a, a, a, a, a, a, a, a};
  mul8(d, x, b);
}

__device__ __forceinline__ float sum8(const float (&f)[8]) {
  return ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
}

// The gains of y: its norm's (if it has one), times a gate that all tokens share.
template <bool VEC>
__device__ __forceinline__ void gains_y(const ResidualArgs& p, int c, int tid, int threads, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = 1.f;
  if (p.post) gains<VEC>(p.w_post, p, c, tid, threads, f);
  if (p.gate && p.gate_token == 0) {
    if (p.gate_channel) {
      float x[8];
      load8_any<VEC>(p.gate, p.gate_f32, c, tid, threads, p.H, x);
      mul8(f, f, x);
    } else {
      mul8(f, p.gate_f32 ? *static_cast<const float*>(p.gate) : bf16_bits_to_float(*static_cast<const uint16_t*>(p.gate)), f);
    }
  }
}

// A gate of token t's own: its one value, or 1.
__device__ __forceinline__ float token_gate(const ResidualArgs& p, int t) {
  if (!p.gate || p.gate_channel || p.gate_token == 0) return 1.f;
  return p.gate_f32 ? static_cast<const float*>(p.gate)[t * p.gate_token]
                    : bf16_bits_to_float(static_cast<const uint16_t*>(p.gate)[t * p.gate_token]);
}

__device__ __forceinline__ bool gate_is_rows(const ResidualArgs& p) { return p.gate && p.gate_channel && p.gate_token != 0; }

template <int SIZE, typename T>
__device__ __forceinline__ auto* row_of(T* base, long long row, long long stride) {
  using B = std::conditional_t<std::is_const_v<T>, const uint8_t, uint8_t>;
  return reinterpret_cast<B*>(base) + row * stride * SIZE;
}

// y += the k + 1 rows of token t, weighted, RB of them in flight together.
template <bool VEC, int CH, int RB>
__device__ __forceinline__ void combine_rows(const ResidualArgs& p, int t, int tid, int threads, float (&y)[CH][8]) {
  const int A = p.T * p.k;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) y[c][j] = 0.f;
  for (int j0 = 0; j0 <= p.k; j0 += RB) {
    long long row[RB];
    float w[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int j = j0 + b;
      row[b] = j == p.k ? A + t : -1;
      w[b] = 1.f;
      if (j < p.k) {
        row[b] = __ldg(p.inv_perm + static_cast<size_t>(t) * p.k + j);
        w[b] = __ldg(p.topk_w + static_cast<size_t>(t) * p.k + j);
        if (row[b] < 0 || row[b] >= A) {
          set_device_error(p.err, MOE_DEV_BAD_INDEX);
          row[b] = -1;
        }
      }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (VEC) {
        const int i = channel<true>(c, 0, tid, threads);
        uint4 v[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b)
          if (row[b] >= 0 && i < p.H) v[b] = __ldg(reinterpret_cast<const uint4*>(p.y + row[b] * p.y_stride + i));
#pragma unroll
        for (int b = 0; b < RB; ++b)
          if (row[b] >= 0 && i < p.H) {
            float f[8];
            unpack8(v[b], f);
            fma8(y[c], w[b], f, y[c]);
          }
      } else {
#pragma unroll
        for (int b = 0; b < RB; ++b)
          if (row[b] >= 0) {
            float f[8];
            load8<false, false>(p.y + row[b] * p.y_stride, c, tid, threads, p.H, f);
            fma8(y[c], w[b], f, y[c]);
          }
      }
    }
  }
}

}  // namespace residual
}  // namespace moe
