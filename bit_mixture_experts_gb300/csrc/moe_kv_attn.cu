// Causal attention of new tokens over a paged key/value cache, GQA, online
// softmax: o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m), s_j = scale q.k_j.
//
// One warp per (token, query head): each lane holds d/32 values of q and of the
// running output; one key at a time, the dot product summed over the warp.
#include "moe_kv_dev.cuh"

namespace moe {

namespace {

constexpr int AT_THREADS = 128;

struct AttnArgs {
  const uint16_t* q;
  long long q_token, q_head;
  uint16_t* out;
  float* lse;
  float scale;
  int q_heads;
};

template <int D, bool Q8>
__device__ __forceinline__ void load_row(const void* pool, const float* scale, size_t at, int lane, float (&x)[D / 32]) {
  constexpr int N = D / 32;
  if (!Q8) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(pool) + (at * D + lane * N) / 2;
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const uint32_t u = p[j];
      x[2 * j] = __uint_as_float(u << 16);
      x[2 * j + 1] = __uint_as_float(u & 0xffff0000u);
    }
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(pool) + (at * D + lane * N) / 2;
    const float sc = scale[at];
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const float2 f = kv::e4m3x2_to_float2(p[j]);
      x[2 * j] = f.x * sc;
      x[2 * j + 1] = f.y * sc;
    }
  }
}

template <int D, bool Q8>
__global__ void __launch_bounds__(AT_THREADS) kv_attention_kernel(const kv::Args a, const AttnArgs g) {
  constexpr int N = D / 32;
  const long long row = (static_cast<long long>(blockIdx.x) * AT_THREADS + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<long long>(a.T) * g.q_heads) return;
  const int t = static_cast<int>(row / g.q_heads), hq = static_cast<int>(row % g.q_heads);
  const int h = hq / (g.q_heads / a.heads);
  const int b = kv::find_seq(a, t);
  if (b < 0) return;
  const kv::Seq s = kv::load_seq(a, b);
  const int seen = s.len - s.n + t - s.row0 + 1;
  float q[N], o[N];
  const uint16_t* qp = g.q + t * g.q_token + hq * g.q_head + lane * N;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    q[j] = bf16_bits_to_float(qp[j]) * g.scale;
    o[j] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int p = 0; p < seen; ++p) {
    const int page = kv::find_page(a, b, p);
    if (page < 0) continue;
    const size_t at = (static_cast<size_t>(page) * a.heads + h) * a.page_size + p % a.page_size;
    float k[N], v[N];
    load_row<D, Q8>(a.k, a.k_scale, at, lane, k);
    load_row<D, Q8>(a.v, a.v_scale, at, lane, v);
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) dot = fmaf(q[j], k[j], dot);
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, w);
    const float m1 = fmaxf(m, dot);
    const float m0 = m1 == -INFINITY ? 0.f : m1;
    const float f = expf(m - m0), w = expf(dot - m0);
    l = fmaf(l, f, w);
    m = m1;
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = fmaf(o[j], f, w * v[j]);
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;  // no key seen: 0
  uint16_t* op = g.out + row * D + lane * N;
#pragma unroll
  for (int j = 0; j < N; ++j) op[j] = float_to_bf16_bits(o[j] * inv);
  if (g.lse && lane == 0) g.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t kv_attention_workspace_bytes(int d) { return 0 * static_cast<size_t>(d); }

cudaError_t launch_kv_attention(const kv::Args& a, bool q8, const uint16_t* q, long long q_token, long long q_head,
                                int q_heads, float scale, uint16_t* out, float* lse, void* ws,
                                cudaStream_t s) {
  (void)ws;
  const AttnArgs g = {q, q_token, q_head, out, lse, scale, q_heads};
  const long long rows = static_cast<long long>(a.T) * q_heads;
  const unsigned grid = static_cast<unsigned>((rows * 32 + AT_THREADS - 1) / AT_THREADS);
  if (a.d == 64)
    q8 ? kv_attention_kernel<64, true><<<grid, AT_THREADS, 0, s>>>(a, g)
       : kv_attention_kernel<64, false><<<grid, AT_THREADS, 0, s>>>(a, g);
  else
    q8 ? kv_attention_kernel<128, true><<<grid, AT_THREADS, 0, s>>>(a, g)
       : kv_attention_kernel<128, false><<<grid, AT_THREADS, 0, s>>>(a, g);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace moe
