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
};

// One sequence: its first row in the dense tensors, its new tokens, its tokens in all.
struct Seq {
  int row0, n, len;
};

__device__ __forceinline__ Seq load_seq(const Args& a, int b) {
  Seq s;
  int lo = __ldg(a.cu_q + b), hi = __ldg(a.cu_q + b + 1), len = __ldg(a.kv_len + b);
  const int most = a.table_width * a.page_size;
  if (lo < 0 || hi < lo || hi > a.T || len < 0 || len > most) {
    set_device_error(a.err, MOE_DEV_BAD_INDEX);
    lo = min(max(lo, 0), a.T);
    hi = min(max(hi, lo), a.T);
    len = min(max(len, 0), most);
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

// Page of position p of sequence b, or -1 (recorded) where the table holds none.
__device__ __forceinline__ int find_page(const Args& a, int b, int p) {
  const int page = __ldg(a.page_table + static_cast<size_t>(b) * a.table_width + p / a.page_size);
  if (page < 0 || page >= a.num_pages) {
    set_device_error(a.err, MOE_DEV_BAD_INDEX);
    return -1;
  }
  return page;
}

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

}  // namespace kv
}  // namespace moe
