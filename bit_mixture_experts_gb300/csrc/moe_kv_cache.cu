// Writing new tokens' keys and values into the paged cache and reading them
// back: bf16 as it is, or e4m3 with one power-of-two scale per token and head.
//
// e4m3 row of d values x: a = max|x|, scale 2^e with e the least integer (at
// least -126) such that a <= 448 * 2^e, stored value e4m3(x * 2^-e).  The scale
// is a power of two because it then costs no accuracy (the format is a float:
// its relative step is the same whatever the scale, short of the subnormals,
// which start 2^-14 below the largest value) and no rounding: x * 2^-e is
// exact, so each value is rounded once, and e4m3 * 2^e is exact in bf16, so
// reading back rounds nothing and an attention over the cache sees the same
// bits as one over the bf16 values it stands for.
//
// Both kernels move every byte once and compute next to nothing: a thread per
// eight values (one 16-byte load or store of bf16), d/8 threads per row.
#include "moe_kv_dev.cuh"

namespace moe {

namespace {

constexpr int KV_THREADS = 256;

struct NewRows {
  const uint16_t* k;
  const uint16_t* v;
  long long k_token, k_head, v_token, v_head;
};

// Scale of a row from the largest magnitude among its bf16 bits (as an integer: the order of
// magnitudes is that of their bits).  Returns the float32 bits of 2^e; *inv gets those of 2^-e.
__device__ __forceinline__ uint32_t row_scale_bits(uint32_t amax, uint32_t* inv) {
  if (amax >= 0x7f80u) {  // an infinity or NaN in the row
    *inv = 0x7fffffffu;
    return 0x7fffffffu;
  }
  int e = 0;
  if (amax) {
    // a = 2^(E - 127) (1 + m / 128); 448 = 1.75 * 2^8.  Subnormals fall under the limit of -126.
    const int E = static_cast<int>(amax >> 7), m = static_cast<int>(amax & 0x7fu);
    e = max(E - 127 - 8 + (m > 96 ? 1 : 0), -126);
  }
  *inv = static_cast<uint32_t>(127 - e) << 23;
  return static_cast<uint32_t>(127 + e) << 23;
}

// One thread: eight values of one row.  Item i: chunk i % (D/8) of row i / (D/8); rows in the order
// token, key before value, head.
template <int D, bool Q8>
__global__ void __launch_bounds__(KV_THREADS) kv_append_kernel(const kv::Args a, const NewRows in) {
  constexpr int C = D / 8;
  const long long items = static_cast<long long>(a.T) * 2 * a.heads * C;
  const long long i = static_cast<long long>(blockIdx.x) * KV_THREADS + threadIdx.x;
  const bool live = i < items;
  const long long row = live ? i / C : 0;
  const int c = static_cast<int>(i % C);
  const int t = static_cast<int>(row / (2 * a.heads)), r = static_cast<int>(row % (2 * a.heads));
  const bool is_v = r >= a.heads;
  const int h = is_v ? r - a.heads : r;
  uint4 x = make_uint4(0, 0, 0, 0);
  size_t at = 0;  // row of the pool
  bool write = false;
  if (live) {
    const uint16_t* src = is_v ? in.v + t * in.v_token + h * in.v_head : in.k + t * in.k_token + h * in.k_head;
    x = __ldg(reinterpret_cast<const uint4*>(src) + c);
    const int b = kv::find_seq(a, t);
    if (b >= 0) {
      const kv::Seq s = kv::load_seq(a, b);
      const int p = s.len - s.n + t - s.row0;
      const int page = p >= 0 && p < s.len ? kv::find_page(a, b, p) : -1;
      write = page >= 0;
      at = (static_cast<size_t>(max(page, 0)) * a.heads + h) * a.page_size + max(p, 0) % a.page_size;
    }
  }
  if (!Q8) {
    if (write) reinterpret_cast<uint4*>(is_v ? a.v : a.k)[at * C + c] = x;
    return;
  }
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) amax = max(amax, max(u[j] & 0x7fffu, (u[j] >> 16) & 0x7fffu));
#pragma unroll
  for (int m = C / 2; m >= 1; m >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  uint32_t inv_bits;
  const uint32_t scale = row_scale_bits(amax, &inv_bits);
  const float inv = __uint_as_float(inv_bits);
  uint32_t o[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint16_t lo, hi;
    const uint32_t p = u[2 * j], q = u[2 * j + 1];
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(lo)
        : "f"(__uint_as_float(p & 0xffff0000u) * inv), "f"(__uint_as_float(p << 16) * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(hi)
        : "f"(__uint_as_float(q & 0xffff0000u) * inv), "f"(__uint_as_float(q << 16) * inv));
    o[j] = static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
  }
  if (write) {
    reinterpret_cast<uint2*>(is_v ? a.v : a.k)[at * C + c] = make_uint2(o[0], o[1]);
    if (c == 0) (is_v ? a.v_scale : a.k_scale)[at] = __uint_as_float(scale);
  }
}

template <int D, bool Q8>
__global__ void __launch_bounds__(KV_THREADS) kv_read_kernel(const kv::Args a, uint16_t* __restrict__ k_out,
                                                             uint16_t* __restrict__ v_out) {
  constexpr int C = D / 8;
  const long long items = static_cast<long long>(a.T) * 2 * a.heads * C;
  const long long i = static_cast<long long>(blockIdx.x) * KV_THREADS + threadIdx.x;
  if (i >= items) return;
  const long long row = i / C;
  const int c = static_cast<int>(i % C);
  const int t = static_cast<int>(row / (2 * a.heads)), r = static_cast<int>(row % (2 * a.heads));
  const bool is_v = r >= a.heads;
  const int h = is_v ? r - a.heads : r;
  const int b = kv::find_seq(a, t);
  if (b < 0) return;
  const kv::Seq s = kv::load_seq(a, b);
  const int p = s.len - s.n + t - s.row0;
  const int page = p >= 0 && p < s.len ? kv::find_page(a, b, p) : -1;
  uint4 o = make_uint4(0, 0, 0, 0);
  if (page >= 0) {
    const size_t at = (static_cast<size_t>(page) * a.heads + h) * a.page_size + p % a.page_size;
    if (!Q8) {
      o = reinterpret_cast<const uint4*>(is_v ? a.v : a.k)[at * C + c];
    } else {
      const uint2 x = reinterpret_cast<const uint2*>(is_v ? a.v : a.k)[at * C + c];
      const float sc = (is_v ? a.v_scale : a.k_scale)[at];
      const float2 f0 = kv::e4m3x2_to_float2(x.x & 0xffffu), f1 = kv::e4m3x2_to_float2(x.x >> 16);
      const float2 f2 = kv::e4m3x2_to_float2(x.y & 0xffffu), f3 = kv::e4m3x2_to_float2(x.y >> 16);
      o = make_uint4(pack_bf16x2(f0.x * sc, f0.y * sc), pack_bf16x2(f1.x * sc, f1.y * sc),
                     pack_bf16x2(f2.x * sc, f2.y * sc), pack_bf16x2(f3.x * sc, f3.y * sc));
    }
  }
  reinterpret_cast<uint4*>(is_v ? v_out : k_out)[(static_cast<size_t>(t) * a.heads + h) * C + c] = o;
}

unsigned blocks_for(const kv::Args& a) {
  const long long items = static_cast<long long>(a.T) * 2 * a.heads * (a.d / 8);
  return static_cast<unsigned>((items + KV_THREADS - 1) / KV_THREADS);
}

}  // namespace

cudaError_t launch_kv_append(const kv::Args& a, bool q8, const uint16_t* k, long long k_token, long long k_head,
                             const uint16_t* v, long long v_token, long long v_head, cudaStream_t s) {
  const NewRows in = {k, v, k_token, k_head, v_token, v_head};
  const unsigned grid = blocks_for(a);
  if (a.d == 64)
    q8 ? kv_append_kernel<64, true><<<grid, KV_THREADS, 0, s>>>(a, in)
       : kv_append_kernel<64, false><<<grid, KV_THREADS, 0, s>>>(a, in);
  else
    q8 ? kv_append_kernel<128, true><<<grid, KV_THREADS, 0, s>>>(a, in)
       : kv_append_kernel<128, false><<<grid, KV_THREADS, 0, s>>>(a, in);
  note_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const kv::Args& a, bool q8, uint16_t* k, uint16_t* v, cudaStream_t s) {
  const unsigned grid = blocks_for(a);
  if (a.d == 64)
    q8 ? kv_read_kernel<64, true><<<grid, KV_THREADS, 0, s>>>(a, k, v)
       : kv_read_kernel<64, false><<<grid, KV_THREADS, 0, s>>>(a, k, v);
  else
    q8 ? kv_read_kernel<128, true><<<grid, KV_THREADS, 0, s>>>(a, k, v)
       : kv_read_kernel<128, false><<<grid, KV_THREADS, 0, s>>>(a, k, v);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace moe
