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
// Both kernels move every byte once and compute next to nothing.  A warp takes
// 1, 4 or 16 consecutive tokens: its lanes look up one token's sequence, page
// and row each, then move the tokens' rows (keys then values, by head), a row
// per d/8 lanes (d/16 where a row is read from e4m3: 16 codes a lane).  The
// lookups cost as much as moving several rows, so they are not done per row:
// with one thread per eight values looking up its own token the kernels ran at
// the instruction rate, not the memory's (append and read of 46K bf16 tokens
// 180 us).  Four rows per lane are in flight.  Measured, calls in a row from a
// CUDA graph: 46K bf16 tokens of 8 KV heads of 128 appended and read 121 us
// (766 MB, 6.3 TB/s), 131071 e4m3 tokens of 2 heads read 37 us (5.5 TB/s: 256
// bytes written for 132 read); small calls are bound by two launches (5 us).
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

// A token's place: the pool's row of its head 0 (head h: h * page_size further), or -1 where it has none
// (rows of no sequence: -2).
__device__ __forceinline__ int find_place(const kv::Args& a, int t) {
  if (t >= a.T) return -2;
  const int b = kv::find_seq(a, t);
  if (b < 0) return -2;
  const kv::Seq s = kv::load_seq(a, b);
  const int p = s.len - s.n + t - s.row0;
  if (p < 0 || p >= s.len) return -1;
  const int e = p / a.page_size, page = kv::find_page(a, b, p);
  return page < 0 ? -1 : page * a.heads * a.page_size + p - e * a.page_size;
}

// Sixteen codes as bf16 values, 32 bytes.
__device__ __forceinline__ void store_expanded(uint4* dst, uint4 x, float scale) {
  uint32_t s1, s2;
  kv::scale_pairs(scale, &s1, &s2);
  const uint2 v0 = kv::expand4(x.x, s1), v1 = kv::expand4(x.y, s1);
  const uint2 v2 = kv::expand4(x.z, s1), v3 = kv::expand4(x.w, s1);
  dst[0] = make_uint4(kv::bf16x2_mul(v0.x, s2), kv::bf16x2_mul(v0.y, s2), kv::bf16x2_mul(v1.x, s2),
                      kv::bf16x2_mul(v1.y, s2));
  dst[1] = make_uint4(kv::bf16x2_mul(v2.x, s2), kv::bf16x2_mul(v2.y, s2), kv::bf16x2_mul(v3.x, s2),
                      kv::bf16x2_mul(v3.y, s2));
}

constexpr int FLIGHT = 4;  // row loads of a lane in flight

// Walks a warp's (token, group of RPW rows) pairs in order, FLIGHT at a time.
struct Step {
  int i, r0;  // token of the warp, first row
  __device__ __forceinline__ void next(int rows, int rpw) {
    r0 += rpw;
    if (r0 >= rows) {
      r0 = 0;
      ++i;
    }
  }
};

template <int D, bool Q8>
__global__ void __launch_bounds__(KV_THREADS) kv_append_kernel(const kv::Args a, const NewRows in, int tokens) {
  constexpr int C = D / 8, RPW = 32 / C;  // lanes of a row, rows at a time
  const int warp = (blockIdx.x * KV_THREADS + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  const int t0 = warp * tokens, c = lane % C, rows = 2 * a.heads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (t0 >= a.T) return;
  const int mine = lane < tokens ? find_place(a, t0 + lane) : -2;
  Step s = {0, 0};
  while (s.i < tokens) {
    uint4 x[FLIGHT];
    int place[FLIGHT], row[FLIGHT];  // place: of the token, -1 for none; row: of the token's rows
#pragma unroll
    for (int u = 0; u < FLIGHT; ++u) {
      const int r = s.r0 + lane / C, t = t0 + s.i;
      place[u] = __shfl_sync(0xffffffffu, mine, s.i & 31);
      if (s.i >= tokens || r >= rows) place[u] = -1;
      row[u] = r;
      x[u] = make_uint4(0, 0, 0, 0);
      if (place[u] >= 0) {
        const uint16_t* src =
            r >= a.heads ? in.v + t * in.v_token + (r - a.heads) * in.v_head : in.k + t * in.k_token + r * in.k_head;
        x[u] = __ldg(reinterpret_cast<const uint4*>(src) + c);
      }
      s.next(rows, RPW);
    }
#pragma unroll
    for (int u = 0; u < FLIGHT; ++u) {
      const bool live = place[u] >= 0, is_v = row[u] >= a.heads;
      const size_t at = static_cast<size_t>(max(place[u], 0)) + (is_v ? row[u] - a.heads : row[u]) * a.page_size;
      if (!Q8) {
        if (live) reinterpret_cast<uint4*>(is_v ? a.v : a.k)[at * C + c] = x[u];
        continue;
      }
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      uint32_t amax = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) amax = max(amax, max(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
#pragma unroll
      for (int m = C / 2; m >= 1; m >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, m));
      uint32_t inv_bits;
      const uint32_t scale = row_scale_bits(amax, &inv_bits);
      const float inv = __uint_as_float(inv_bits);
      uint32_t o[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint16_t lo, hi;
        const uint32_t p = w[2 * j], q = w[2 * j + 1];
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
            : "=h"(lo)
            : "f"(__uint_as_float(p & 0xffff0000u) * inv), "f"(__uint_as_float(p << 16) * inv));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
            : "=h"(hi)
            : "f"(__uint_as_float(q & 0xffff0000u) * inv), "f"(__uint_as_float(q << 16) * inv));
        o[j] = static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
      }
      if (live) {
        reinterpret_cast<uint2*>(is_v ? a.v : a.k)[at * C + c] = make_uint2(o[0], o[1]);
        if (c == 0) (is_v ? a.v_scale : a.k_scale)[at] = __uint_as_float(scale);
      }
    }
  }
}

template <int D, bool Q8>
__global__ void __launch_bounds__(KV_THREADS) kv_read_kernel(const kv::Args a, uint16_t* __restrict__ k_out,
                                                             uint16_t* __restrict__ v_out, int tokens) {
  constexpr int C = Q8 ? D / 16 : D / 8, RPW = 32 / C;  // 16-byte pieces of a stored row
  const int warp = (blockIdx.x * KV_THREADS + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  const int t0 = warp * tokens, c = lane % C, rows = 2 * a.heads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (t0 >= a.T) return;
  const int mine = lane < tokens ? find_place(a, t0 + lane) : -2;
  Step s = {0, 0};
  while (s.i < tokens) {
    uint4 x[FLIGHT];
    float scale[FLIGHT];
    int token[FLIGHT], row[FLIGHT];  // token -1: nothing to do
#pragma unroll
    for (int u = 0; u < FLIGHT; ++u) {
      const int r = s.r0 + lane / C, place = __shfl_sync(0xffffffffu, mine, s.i & 31);
      const bool is_v = r >= a.heads;
      token[u] = s.i < tokens && r < rows && place != -2 ? t0 + s.i : -1;
      row[u] = r;
      x[u] = make_uint4(0, 0, 0, 0);
      scale[u] = 1.f;
      if (token[u] >= 0 && place >= 0) {
        const size_t at = static_cast<size_t>(place) + (is_v ? r - a.heads : r) * a.page_size;
        x[u] = __ldg(reinterpret_cast<const uint4*>(is_v ? a.v : a.k) + at * C + c);
        if (Q8) scale[u] = __ldg((is_v ? a.v_scale : a.k_scale) + at);
      }
      s.next(rows, RPW);
    }
#pragma unroll
    for (int u = 0; u < FLIGHT; ++u) {
      if (token[u] < 0) continue;
      const bool is_v = row[u] >= a.heads;
      uint4* dst = reinterpret_cast<uint4*>(is_v ? v_out : k_out) +
                   (static_cast<size_t>(token[u]) * a.heads + (is_v ? row[u] - a.heads : row[u])) * (D / 8) + (Q8 ? 2 * c : c);
      if (!Q8) {
        *dst = x[u];
        continue;
      }
      store_expanded(dst, x[u], scale[u]);
    }
  }
}

// Expands what the sequences with new tokens have cached to bf16 pages of TILE tokens in order: block
// (tile, b), a warp per 16 tokens.  For an attention of many query rows, each tile of which would expand
// the same codes again.
template <int D>
__global__ void __launch_bounds__(KV_THREADS) kv_expand_kernel(const kv::Args a, uint16_t* __restrict__ k_out,
                                                               uint16_t* __restrict__ v_out, int tile) {
  constexpr int C = D / 16, RPW = 32 / C, TOKENS = 16;
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = lane % C, rows = 2 * a.heads, t0 = warp * TOKENS;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const kv::Seq q = kv::load_seq(a, b);
  const int p0 = blockIdx.x * tile + t0;
  if (q.n == 0 || p0 >= q.len) return;
  int mine = -2;
  if (lane < TOKENS && p0 + lane < q.len) {
    const int p = p0 + lane, e = p / a.page_size, page = kv::page_of(a, b, e);
    mine = page < 0 ? -1 : page * a.heads * a.page_size + p - e * a.page_size;
  }
  const size_t out0 = (static_cast<size_t>(b) * gridDim.x + blockIdx.x) * a.heads * tile + t0;
  Step s = {0, 0};
  while (s.i < TOKENS) {
    uint4 x[FLIGHT];
    float scale[FLIGHT];
    int token[FLIGHT], row[FLIGHT];
#pragma unroll
    for (int u = 0; u < FLIGHT; ++u) {
      const int r = s.r0 + lane / C, place = __shfl_sync(0xffffffffu, mine, s.i & 31);
      const bool is_v = r >= a.heads;
      token[u] = s.i < TOKENS && r < rows && place != -2 ? s.i : -1;
      row[u] = r;
      x[u] = make_uint4(0, 0, 0, 0);
      scale[u] = 1.f;
      if (token[u] >= 0 && place >= 0) {
        const size_t at = static_cast<size_t>(place) + (is_v ? r - a.heads : r) * a.page_size;
        x[u] = __ldg(reinterpret_cast<const uint4*>(is_v ? a.v : a.k) + at * C + c);
        scale[u] = __ldg((is_v ? a.v_scale : a.k_scale) + at);
      }
      s.next(rows, RPW);
    }
#pragma unroll
    for (int u = 0; u < FLIGHT; ++u) {
      if (token[u] < 0) continue;
      const bool is_v = row[u] >= a.heads;
      const size_t at = out0 + static_cast<size_t>(is_v ? row[u] - a.heads : row[u]) * tile + token[u];
      store_expanded(reinterpret_cast<uint4*>(is_v ? v_out : k_out) + at * (D / 8) + 2 * c, x[u], scale[u]);
    }
  }
}

// Tokens per warp: 1 to 16, as many as leave 16384 warps or more (about 100 per SM: with half as many the
// read of 131071 e4m3 tokens takes 41 us, not 36).
int tokens_per_warp(int T) {
  int n = 1;
  while (n < 16 && T / (2 * n) >= 16384) n *= 2;
  return n;
}

// A grid that is started while the kernel before it in the stream ends (the kernels wait for its results
// themselves).
template <typename... P, typename... Q>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, cudaStream_t s, Q... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(KV_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  note_launches(1);
  return e;
}

// One warp per `tokens` tokens.
dim3 warps_for(int T, int tokens) { return dim3(ceil_div(ceil_div(T, tokens), KV_THREADS / 32)); }

}  // namespace

cudaError_t launch_kv_append(const kv::Args& a, bool q8, const uint16_t* k, long long k_token, long long k_head,
                             const uint16_t* v, long long v_token, long long v_head, cudaStream_t s) {
  const NewRows in = {k, v, k_token, k_head, v_token, v_head};
  const int n = tokens_per_warp(a.T);
  const dim3 grid = warps_for(a.T, n);
  if (a.d == 64)
    return q8 ? launch_early(kv_append_kernel<64, true>, grid, s, a, in, n)
              : launch_early(kv_append_kernel<64, false>, grid, s, a, in, n);
  return q8 ? launch_early(kv_append_kernel<128, true>, grid, s, a, in, n)
            : launch_early(kv_append_kernel<128, false>, grid, s, a, in, n);
}

cudaError_t launch_kv_read(const kv::Args& a, bool q8, uint16_t* k, uint16_t* v, cudaStream_t s) {
  const int n = tokens_per_warp(a.T);
  const dim3 grid = warps_for(a.T, n);
  if (a.d == 64)
    return q8 ? launch_early(kv_read_kernel<64, true>, grid, s, a, k, v, n)
              : launch_early(kv_read_kernel<64, false>, grid, s, a, k, v, n);
  return q8 ? launch_early(kv_read_kernel<128, true>, grid, s, a, k, v, n)
            : launch_early(kv_read_kernel<128, false>, grid, s, a, k, v, n);
}

// Pages of `tile` = 128 tokens, `tiles` per sequence.
cudaError_t launch_kv_expand(const kv::Args& a, uint16_t* k, uint16_t* v, int tile, int tiles, cudaStream_t s) {
  const dim3 grid(tiles, a.B);
  return a.d == 64 ? launch_early(kv_expand_kernel<64>, grid, s, a, k, v, tile)
                   : launch_early(kv_expand_kernel<128>, grid, s, a, k, v, tile);
}

}  // namespace moe
