// Shared by the kernels of the paged key/value cache (moe_kv_cache.cu,
// moe_kv_attn.cu): the batch description and the lookup of tokens and pages.
#pragma once
#include "moe_common.cuh"

namespace moe {
namespace kv {

// The cache and a step's batch as the kernels take them.
struct Args {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  const int32_t* page_table;
  const int32_t* cu_q;
  const int32_t* kv_len;
  int* err;
  int num_pages, page_size, heads, d;
  int B, table_width, T;
  int most;       // tokens of a sequence that its table has pages for
  bool in_order;  // no table: sequence b's pages are b * table_width and on
};

// One sequence: its first row in the dense tensors, its new tokens, its tokens in all.
struct Seq {
  int row0, n, len;
};

__device__ __forceinline__ Seq load_seq(const Args& a, int b) {
  Seq s;
  int lo = __ldg(a.cu_q + b), hi = __ldg(a.cu_q + b + 1), len = __ldg(a.kv_len + b);
  if (lo < 0 || hi < lo || hi > a.T || len < 0 || len > a.most) {
    set_device_error(a.err, MOE_DEV_BAD_INDEX);
    lo = min(max(lo, 0), a.T);
    hi = min(max(hi, lo), a.T);
    len = min(max(len, 0), a.most);
  }
  s.row0 = lo;
  s.n = hi - lo;
  s.len = len;
  return s;
}

// The sequence whose rows hold t, or -1.
__device__ __forceinline__ int find_seq(const Args& a, int t) {
  int lo = 0, hi = a.B;  // the first b in [lo, hi] with cu_q[b] > t, less one
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.cu_q + mid) > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  const int b = lo - 1;
  return b >= 0 && t < __ldg(a.cu_q + b + 1) ? b : -1;
}

// Page e of sequence b, or -1 (recorded) where the table holds none.
__device__ __forceinline__ int page_of(const Args& a, int b, int e) {
  if (a.in_order) return b * a.table_width + e;
  const int page = __ldg(a.page_table + static_cast<size_t>(b) * a.table_width + e);
  if (page < 0 || page >= a.num_pages) {
    set_device_error(a.err, MOE_DEV_BAD_INDEX);
    return -1;
  }
  return page;
}

__device__ __forceinline__ int find_page(const Args& a, int b, int p) { return page_of(a, b, p / a.page_size); }

// Two e4m3 bytes (low 16 bits of x, the first in the low byte) -> floats, exact.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t x) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(x)));
  float2 f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// A bf16 pair with zeros in place of infinities and NaN.
__device__ __forceinline__ uint32_t bf16x2_finite(uint32_t x) {
  return x & (((x & 0x7f80u) != 0x7f80u ? 0xffffu : 0u) | ((x & 0x7f800000u) != 0x7f800000u ? 0xffff0000u : 0u));
}

__device__ __forceinline__ uint4 bf16x8_finite(uint4 x) {
  return make_uint4(bf16x2_finite(x.x), bf16x2_finite(x.y), bf16x2_finite(x.z), bf16x2_finite(x.w));
}

// Four e4m3 codes -> four bf16 values times s (a bf16 pair).  The code's bits s eeee mmm become
// s 0000eeee mmm0000, a bf16 that is 2^-120 of the code's value (its subnormals are bf16 subnormals);
// s holds 2^120 times the scale as far as bf16 goes.  The product is exact short of bf16's own
// underflow.
__device__ __forceinline__ uint2 expand4(uint32_t x, uint32_t s) {
  // bytes sign-extended to 16 bits (prmt's sign mode), then moved up by 4: the sign's copies that land
  // on the exponent's upper bits are masked away
  uint32_t a, b;
  asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(a) : "r"(x));
  asm("prmt.b32 %0, %1, 0, 0xB3A2;" : "=r"(b) : "r"(x));
  return make_uint2(bf16x2_mul((a << 4) & 0x87f087f0u, s), bf16x2_mul((b << 4) & 0x87f087f0u, s));
}

// 2^120 times a scale (a power of two; NaN stays NaN) as two bf16 pairs whose product it is: *s2 is 1 but
// for scales of 2^8 and more, which 2^120 times is beyond bf16.
__device__ __forceinline__ void scale_pairs(float scale, uint32_t* s1, uint32_t* s2) {
  const uint32_t sc = __float_as_uint(scale);
  const int e = static_cast<int>(sc >> 23) + 120;
  const uint32_t lo = min(e, 254), hi = e - lo + 127;
  *s1 = (sc > 0x7f800000u ? 0x7fffu : lo << 7) * 0x10001u;
  *s2 = (hi << 7) * 0x10001u;
}

}  // namespace kv
}  // namespace moe
