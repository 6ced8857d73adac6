// extern "C" entry points of libmoe_w4.so: argument checks, the device error
// word, and the launch sequence of the layer.  Every compute step runs in the
// kernels of moe_route.cu, moe_gemm_tc.cu, moe_gemm_gemv.cu, moe_decode.cu,
// moe_combine.cu, moe_gate.cu, moe_residual.cu, moe_kv_cache.cu and
// moe_kv_attn.cu; nothing here touches tensor data on the host.
#include <float.h>

#include <atomic>
#include <mutex>

#include "moe_common.cuh"
#include "moe_kv_dev.cuh"
#include "moe_residual.cuh"
#ifdef MOE_TRACE
#include "moe_tc_dev.cuh"  // the trace words' layout (TRACE_ERR_INTS, TRACE_CTAS, trace_wait)
#endif

namespace moe {

#ifdef MOE_TRACE
// The trace build keeps the wait statistics of the tensor-core kernels right after the error word
// (TRACE_ERR_INTS ints, then TRACE_CTAS x 32 warps x 4 words; see trace_wait).
using tc_dev::TRACE_ERR_INTS;
constexpr size_t TRACE_WORDS = static_cast<size_t>(tc_dev::TRACE_CTAS) * 32 * 4;
struct TraceBlock {
  int err[TRACE_ERR_INTS];
  unsigned long long words[TRACE_WORDS];
};
__device__ TraceBlock g_trace_block;
#define MOE_ERROR_SYMBOL g_trace_block  // the error word is its first int
#else
__device__ int g_device_error = 0;
#define MOE_ERROR_SYMBOL g_device_error
#endif

// Per-device address of the device error word, looked up once per device.
int* device_error_ptr() {
  static std::mutex mu;
  static int* ptrs[64] = {nullptr};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!ptrs[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, MOE_ERROR_SYMBOL) != cudaSuccess) return nullptr;
    ptrs[dev] = static_cast<int*>(p);
  }
  return ptrs[dev];
}

static std::atomic<uint64_t> g_launches{0};

void note_launches(int n) { g_launches.fetch_add(static_cast<uint64_t>(n), std::memory_order_relaxed); }

int num_sms() {
  static int cached[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return 148;
  if (!cached[dev]) {
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    cached[dev] = n > 0 ? n : 148;
  }
  return cached[dev];
}

// defined in the kernel files
size_t route_workspace_bytes(int T, int E, int k);
cudaError_t launch_route(const float* logits, int T, int E, int k, int bn, int32_t* ids, float* w, int32_t* counts,
                         int32_t* offsets, int32_t* perm, int32_t* inv_perm, int32_t* bm, int32_t* nb, void* ws,
                         size_t ws_bytes, cudaStream_t s, int ids_given);
cudaError_t launch_rms_norm(const uint16_t* x, uint16_t* out, int T, int H, float eps, int num_sms, cudaStream_t s);
int norm_router_max_tokens();
cudaError_t launch_norm_router(const uint16_t* x, const uint16_t* wr, uint16_t* xn, float* logits, int T, int H,
                               int E, float eps, cudaStream_t s);
cudaError_t launch_router(const uint16_t* x, const uint16_t* w_router, int T, int H, int E, int k, float* logits,
                          int32_t* ids, float* w, cudaStream_t s);
cudaError_t launch_combine(const uint16_t* y, const int32_t* inv_perm, const float* topk_w, uint16_t* out, int T,
                           int H, int k, int num_sms, cudaStream_t s);
size_t repacked_bytes(int n_mat, int rows, int K);
cudaError_t launch_repack(const uint32_t* packed, const uint16_t* scale, const uint16_t* bias, int n_mat, int rows,
                          int K, int gate_up, void* out, cudaStream_t s);
cudaError_t launch_gemm_gemv(int mode, const uint16_t* act, int T, int H, int F, int E, int k, const void* w,
                             const int32_t* perm, const float* topk_w, const int32_t* block_map,
                             const int32_t* num_blocks, int bn, int cap, void* out, int num_sms, cudaStream_t s);
int gemv_max_rows();
int decode_max_tokens();
size_t decode_workspace_bytes(int T, int H);
cudaError_t launch_ffn_tc(const uint16_t* x, int T, int H, int F, int E, int k, const void* w13, const void* w2,
                          const int32_t* perm, const int32_t* block_map, const int32_t* num_blocks, int bn, int cap,
                          uint16_t* y, int num_sms, cudaStream_t s);
cudaError_t launch_decode(const uint16_t* x, const float* logits, const void* w13, const void* w2, int T, int H, int F,
                          int E, int k, int bn, int32_t* topk_ids, float* topk_w, int32_t* counts, int32_t* offsets,
                          int32_t* perm, int32_t* inv_perm, int32_t* block_map, int32_t* num_blocks, uint16_t* h,
                          uint16_t* y, uint16_t* out, void* ws, unsigned long long wait_ns, int num_sms,
                          cudaStream_t s);
unsigned long long wait_limit_ns();
cudaError_t launch_gemm_tc(int mode, const uint16_t* act, int T, int H, int F, int E, int k, const void* w,
                           const int32_t* perm, const float* topk_w, const int32_t* block_map,
                           const int32_t* num_blocks, int bn, int cap, void* out, int num_sms, cudaStream_t s,
                           bool raw, uint16_t* cmb_out, const int32_t* inv_perm, int* cmb_cnt);
size_t expanded_bytes(int n_mat, int rows, int K);
cudaError_t launch_expand(const void* w4, int n_mat, int rows, int K, void* out, cudaStream_t s);
cudaError_t launch_gemm_pair(int mode, const uint16_t* act, int T, int H, int F, int E, int k, const void* w,
                             const int32_t* perm, const int32_t* block_map, const int32_t* num_blocks, int bn, int cap,
                             void* out, cudaStream_t s);
void set_wait_limit_ns(unsigned long long ns);
cudaError_t launch_kv_append(const kv::Args& a, bool q8, const uint16_t* k, long long k_token, long long k_head,
                             const uint16_t* v, long long v_token, long long v_head, cudaStream_t s);
cudaError_t launch_kv_read(const kv::Args& a, bool q8, uint16_t* k, uint16_t* v, cudaStream_t s);
cudaError_t launch_kv_attention(const kv::Args& a, bool q8, const uint16_t* q, long long q_token, long long q_head,
                                int q_heads, float scale, uint16_t* out, float* lse, void* ws, cudaStream_t s);
size_t kv_attention_workspace_bytes(const kv::Args& a, bool q8, int q_heads);
cudaError_t launch_gate(const float* logits, int T, const moe_gate_t* p, int E, int k, int32_t* ids, float* w,
                        cudaStream_t s);
int residual_max_h();
cudaError_t launch_residual(const ResidualArgs& p, bool combine, bool x32, cudaStream_t s);

namespace {

int check_gate(const moe_gate_t* g, int E, int k) {
  if (!g) return MOE_ERR_NULL;
  if ((g->score != MOE_SCORE_SOFTMAX && g->score != MOE_SCORE_SIGMOID) ||
      (g->group_score != MOE_GROUP_MAX && g->group_score != MOE_GROUP_TOP2))
    return MOE_ERR_MODE;
  if (g->groups < 1 || g->groups > 32 || E % g->groups != 0) return MOE_ERR_SHAPE;
  if (g->top_groups < 1 || g->top_groups > g->groups || g->top_groups * (E / g->groups) < k) return MOE_ERR_SHAPE;
  if (!(g->scale >= -FLT_MAX && g->scale <= FLT_MAX)) return MOE_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(g->bias) & 3u) return MOE_ERR_ALIGN;
  return MOE_OK;
}

// Rows of a tensor in bytes: first row, distance of rows, length and number of rows.
struct Rows {
  uintptr_t at;
  unsigned long long stride, len;
  long long n;
  uintptr_t end() const { return at + (n - 1) * stride + len; }
};

Rows rows_of(const void* p, long long stride, long long cols, int size, long long n) {
  return {reinterpret_cast<uintptr_t>(p), n > 1 ? static_cast<unsigned long long>(stride) * size : 0ull,
          static_cast<unsigned long long>(cols) * size, p ? n : 0};
}

// Whether two sets of rows have a byte in common.
bool overlap(const Rows& a, const Rows& b) {
  if (a.n == 0 || b.n == 0 || a.end() <= b.at || b.end() <= a.at) return false;
  if (a.stride != b.stride || a.stride == 0) return true;
  // columns of one wider tensor
  const unsigned long long d = b.at >= a.at ? (b.at - a.at) % a.stride : (a.stride - (a.at - b.at) % a.stride) % a.stride;
  return d < a.len || d + b.len > a.stride;
}

// A gate's choice must lie apart from what it is made of: other tokens' logits are read while it is written.
int check_gate_overlap(const float* logits, int T, int E, int k, const moe_gate_t* g, const int32_t* ids, const float* w) {
  const Rows out[2] = {rows_of(ids, 0, static_cast<long long>(T) * k, 4, 1), rows_of(w, 0, static_cast<long long>(T) * k, 4, 1)};
  const Rows in[2] = {rows_of(logits, 0, static_cast<long long>(T) * E, 4, 1), rows_of(g->bias, 0, E, 4, 1)};
  if (overlap(out[0], out[1])) return MOE_ERR_OVERLAP;
  for (const Rows& o : out)
    for (const Rows& i : in)
      if (overlap(o, i)) return MOE_ERR_OVERLAP;
  return MOE_OK;
}

bool same(const Rows& a, const Rows& b) { return a.at == b.at && a.stride == b.stride && a.len == b.len && a.n == b.n; }

bool aligned(const void* p, int size) { return reinterpret_cast<uintptr_t>(p) % size == 0; }

// Checks a residual addition of T rows of H channels and fills the kernels' description of it; y: the
// block's output, `y_rows` rows of it (each read by its own row of x, or all by any).
int residual_args(const uint16_t* y, long long y_stride, long long y_rows, bool combine, int T, int H,
                  const moe_residual_t* p, ResidualArgs* a) {
  if (!p) return MOE_ERR_NULL;
  if (T < 0 || T > (1 << 20) || H < 1 || H > residual_max_h()) return MOE_ERR_SHAPE;
  if (!(p->eps >= 0.0f) || !(p->eps <= FLT_MAX) || !(p->scale >= -FLT_MAX && p->scale <= FLT_MAX) ||
      !(p->offset >= -FLT_MAX && p->offset <= FLT_MAX))
    return MOE_ERR_SHAPE;
  const long long most = 1ll << 40;
  for (long long s : {static_cast<long long>(p->x_stride), y_stride, static_cast<long long>(p->gate_token_stride)})
    if (s < 0 || s >= most) return MOE_ERR_SHAPE;
  if (T > 1 && ((p->r && (p->r_stride < H || p->r_stride >= most)) || (p->n && (p->n_stride < H || p->n_stride >= most))))
    return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (!p->x || (!p->r && !p->n)) return MOE_ERR_NULL;
  const int xs = p->stream_f32 ? 4 : 2, ps = p->param_f32 ? 4 : 2, gs = p->gate_f32 ? 4 : 2;
  if (!aligned(p->x, xs) || !aligned(p->r, xs) || !aligned(p->n, 2) || !aligned(y, 2) || !aligned(p->w_pre, ps) ||
      !aligned(p->w_post, ps) || !aligned(p->gate, gs))
    return MOE_ERR_ALIGN;
  const Rows r = rows_of(p->r, p->r_stride, H, xs, T), n = rows_of(p->n, p->n_stride, H, 2, T);
  const Rows in[5] = {rows_of(p->x, p->x_stride, H, xs, T), rows_of(y, y_stride, H, 2, y_rows),
                      rows_of(p->gate, p->gate_token_stride, p->gate_per_channel ? H : 1, gs, T),
                      rows_of(p->w_pre, 0, H, ps, 1), rows_of(p->w_post, 0, H, ps, 1)};
  // Inputs whose place an output may take: each value is read before it is written, by the same thread.  (Not those of
  // all tokens, although with one token their rows are as the output's.)
  const bool place[5] = {true, !combine, (p->gate_per_channel || H == 1) && p->gate_token_stride != 0, false, false};
  if (overlap(r, n)) return MOE_ERR_OVERLAP;
  for (int i = 0; i < 5; ++i)
    for (const Rows& o : {r, n})
      if (overlap(in[i], o) && !(place[i] && same(in[i], o))) return MOE_ERR_OVERLAP;
  a->y = y;
  a->y_stride = y_stride;
  a->inv_perm = nullptr;
  a->topk_w = nullptr;
  a->k = 0;
  a->T = T;
  a->H = H;
  a->x = p->x;
  a->x_stride = p->x_stride;
  a->r = p->r;
  a->r_stride = p->r_stride;
  a->n = p->n;
  a->n_stride = p->n_stride;
  a->w_pre = p->w_pre;
  a->w_post = p->w_post;
  a->gate = y ? p->gate : nullptr;
  a->gate_token = p->gate_token_stride;
  a->gate_channel = p->gate_per_channel != 0;
  a->offset = p->offset;
  a->scale = p->scale;
  a->eps = p->eps;
  a->post = y && p->post;
  a->param_f32 = p->param_f32 != 0;
  a->gate_f32 = p->gate_f32 != 0;
  return MOE_OK;
}

// The outputs lie apart from the combine's places and weights.
int check_places_overlap(const int32_t* inv_perm, const float* topk_w, int T, int H, int k, const moe_residual_t* p) {
  const Rows r = rows_of(p->r, p->r_stride, H, p->stream_f32 ? 4 : 2, T), n = rows_of(p->n, p->n_stride, H, 2, T);
  for (const void* i : {static_cast<const void*>(inv_perm), static_cast<const void*>(topk_w)}) {
    const Rows in = rows_of(i, 0, static_cast<long long>(T) * k, 4, 1);
    if (overlap(in, r) || overlap(in, n)) return MOE_ERR_OVERLAP;
  }
  return MOE_OK;
}

// Checks a cache and a batch and fills the kernels' description of them.  Sizes before pointers, as
// elsewhere.  T = 0 passes (the entry points then return before they look at the dense tensors).
int kv_args(const moe_kv_cache_t* c, const moe_kv_batch_t* b, kv::Args* a) {
  if (!c || !b) return MOE_ERR_NULL;
  if (c->format != MOE_KV_BF16 && c->format != MOE_KV_E4M3) return MOE_ERR_MODE;
  if (c->d != 64 && c->d != 128) return MOE_ERR_SHAPE;
  if (c->page_size < 16 || c->page_size > 1024 || c->page_size % 16 != 0) return MOE_ERR_SHAPE;
  if (c->heads < 1 || c->heads > 1024 || c->num_pages < 1) return MOE_ERR_SHAPE;
  if (static_cast<long long>(c->num_pages) * c->heads * c->page_size >= (1ll << 31)) return MOE_ERR_SHAPE;
  if (b->T < 0 || b->T > (1 << 20) || b->B < 1 || b->B > 65536 || b->table_width < 1) return MOE_ERR_SHAPE;
  if (static_cast<long long>(b->table_width) * c->page_size > (1ll << 30)) return MOE_ERR_SHAPE;
  const bool q8 = c->format == MOE_KV_E4M3;
  int rc = check_ptrs(c->k, c->v);
  if (!rc && q8) rc = check_ptrs(c->k_scale, c->v_scale);
  if (rc) return rc;
  const void* idx[3] = {b->page_table, b->cu_q, b->kv_len};
  for (const void* p : idx)
    if (!p) return MOE_ERR_NULL;
  for (const void* p : idx)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return MOE_ERR_ALIGN;
  a->k = c->k;
  a->v = c->v;
  a->k_scale = q8 ? c->k_scale : nullptr;
  a->v_scale = q8 ? c->v_scale : nullptr;
  a->page_table = b->page_table;
  a->cu_q = b->cu_q;
  a->kv_len = b->kv_len;
  a->num_pages = c->num_pages;
  a->page_size = c->page_size;
  a->heads = c->heads;
  a->d = c->d;
  a->B = b->B;
  a->table_width = b->table_width;
  a->T = b->T;
  a->most = b->table_width * c->page_size;
  a->in_order = false;
  return MOE_OK;
}

// Strides of a [T, heads, d] tensor whose rows of d are contiguous: rows must start on 16 bytes.  The
// stride of a dimension of one element says nothing and is not looked at.
bool kv_strides_ok(long long token, long long head, int T, int heads) {
  const long long most = 1ll << 40;
  if (T <= 1) token = 0;
  if (heads <= 1) head = 0;
  return token % 8 == 0 && head % 8 == 0 && token >= 0 && head >= 0 && token < most && head < most;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_version(void) { return 0x000100; }

uint64_t moe_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

int moe_block_map_capacity(int T, int E, int k, int block_n) {
  if (T < 1 || E < 1 || k < 1 || block_n < 1) return 0;
  const long long A = static_cast<long long>(T) * k;
  return static_cast<int>((A + block_n - 1) / block_n + E + (T + block_n - 1) / block_n);
}

size_t moe_route_workspace_size(int T, int E, int k, int block_n) {
  (void)block_n;
  if (T < 1 || E < 1 || k < 1) return 0;
  return route_workspace_bytes(T, E, k);
}

int moe_route(const float* logits, int T, int E, int k, int block_n, int32_t* topk_ids, float* topk_w,
              int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv_perm, int32_t* block_map,
              int32_t* num_blocks, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  int rc = check_route_shape(T, E, k, block_n);
  if (rc) return rc;
  rc = check_ptrs(logits, topk_ids, topk_w, counts, offsets, perm, inv_perm, block_map, num_blocks);
  if (rc) return rc;
  const size_t need = route_workspace_bytes(T, E, k);
  if (need > 0) {
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
    rc = check_ptrs(workspace);
    if (rc) return rc;
  }
  if (!device_error_ptr()) return MOE_ERR_CUDA;
  return cuda_status(launch_route(logits, T, E, k, block_n, topk_ids, topk_w, counts, offsets, perm, inv_perm,
                                  block_map, num_blocks, workspace, workspace_bytes,
                                  reinterpret_cast<cudaStream_t>(stream), 0));
}

int moe_rms_norm(const uint16_t* x, uint16_t* out, int T, int H, float eps, moe_stream_t stream) {
  if (T < 1 || T > (1 << 20) || H < 8 || H % 8 != 0 || !(eps >= 0.0f)) return MOE_ERR_SHAPE;
  int rc = check_ptrs(x, out);
  if (rc) return rc;
  return cuda_status(launch_rms_norm(x, out, T, H, eps, num_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

int moe_norm_router(const uint16_t* x, const uint16_t* w_router, int T, int H, int E, float eps, uint16_t* x_norm,
                    float* logits, moe_stream_t stream) {
  if (T < 1 || T > norm_router_max_tokens() || H < 8 || H % 8 != 0 || E < 1 || E > 1024 || !(eps >= 0.0f))
    return MOE_ERR_SHAPE;
  int rc = check_ptrs(x, w_router, x_norm, logits);
  if (rc) return rc;
  return cuda_status(
      launch_norm_router(x, w_router, x_norm, logits, T, H, E, eps, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_router(const uint16_t* x, const uint16_t* w_router, int T, int H, int E, int k, float* logits,
               int32_t* topk_ids, float* topk_w, moe_stream_t stream) {
  int rc = check_route_shape(T, E, k, 1);
  if (rc) return rc;
  if (H < 64 || H % 64 != 0 || E % 64 != 0 || E > 512) return MOE_ERR_SHAPE;
  rc = check_ptrs(x, w_router, logits, topk_ids, topk_w);
  if (rc) return rc;
  if (!device_error_ptr()) return MOE_ERR_CUDA;
  return cuda_status(launch_router(x, w_router, T, H, E, k, logits, topk_ids, topk_w,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

int moe_gate(const float* logits, int T, int E, int k, const moe_gate_t* gate, int32_t* topk_ids, float* topk_w,
             moe_stream_t stream) {
  int rc = check_route_shape(T == 0 ? 1 : T, E, k, 1);
  if (rc || (rc = check_gate(gate, E, k))) return rc;
  if (T == 0) return MOE_OK;
  rc = check_ptrs(logits, topk_ids, topk_w);
  if (rc || (rc = check_gate_overlap(logits, T, E, k, gate, topk_ids, topk_w))) return rc;
  return cuda_status(launch_gate(logits, T, gate, E, k, topk_ids, topk_w, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_route_gated(const float* logits, int T, int E, int k, const moe_gate_t* gate, int block_n, int32_t* topk_ids,
                    float* topk_w, int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv_perm,
                    int32_t* block_map, int32_t* num_blocks, void* workspace, size_t workspace_bytes,
                    moe_stream_t stream) {
  int rc = check_route_shape(T, E, k, block_n);
  if (rc || (logits && (rc = check_gate(gate, E, k)))) return rc;
  rc = check_ptrs(topk_ids, topk_w, counts, offsets, perm, inv_perm, block_map, num_blocks);
  if (rc) return rc;
  if (!aligned16(logits)) return MOE_ERR_ALIGN;
  const size_t need = route_workspace_bytes(T, E, k);
  if (need > 0) {
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
    rc = check_ptrs(workspace);
    if (rc) return rc;
  }
  if (logits && (rc = check_gate_overlap(logits, T, E, k, gate, topk_ids, topk_w))) return rc;
  if (!device_error_ptr()) return MOE_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (logits && (rc = cuda_status(launch_gate(logits, T, gate, E, k, topk_ids, topk_w, s)))) return rc;
  return cuda_status(launch_route(logits, T, E, k, block_n, topk_ids, topk_w, counts, offsets, perm, inv_perm,
                                  block_map, num_blocks, workspace, workspace_bytes, s, 1));
}

int moe_residual_norm(const uint16_t* y, int64_t y_stride, int T, int H, const moe_residual_t* p, moe_stream_t stream) {
  ResidualArgs a;
  int rc = residual_args(y, y ? y_stride : 0, T, false, T, H, p, &a);
  if (rc || T == 0) return rc;
  if (!(a.err = device_error_ptr())) return MOE_ERR_CUDA;
  return cuda_status(launch_residual(a, false, p->stream_f32 != 0, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_combine_residual_norm(const uint16_t* y, const int32_t* inv_perm, const float* topk_w, int T, int H, int k,
                              const moe_residual_t* p, moe_stream_t stream) {
  if (k < 1 || k > 32) return MOE_ERR_SHAPE;
  ResidualArgs a;
  int rc = residual_args(y, H, (k + 1ll) * T, true, T, H, p, &a);
  if (rc || T == 0) return rc;
  rc = check_ptrs(y, inv_perm, topk_w);
  if (rc) return rc;
  if ((rc = check_places_overlap(inv_perm, topk_w, T, H, k, p))) return rc;
  a.inv_perm = inv_perm;
  a.topk_w = topk_w;
  a.k = k;
  if (!(a.err = device_error_ptr())) return MOE_ERR_CUDA;
  return cuda_status(launch_residual(a, true, p->stream_f32 != 0, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_route_x(const uint16_t* x, const uint16_t* w_router, int T, int H, int E, int k, int block_n, float* logits,
                int32_t* topk_ids, float* topk_w, int32_t* counts, int32_t* offsets, int32_t* perm,
                int32_t* inv_perm, int32_t* block_map, int32_t* num_blocks, void* workspace,
                size_t workspace_bytes, moe_stream_t stream) {
  int rc = check_route_shape(T, E, k, block_n);
  if (rc) return rc;
  if (H < 64 || H % 64 != 0 || E % 64 != 0 || E > 512) return MOE_ERR_SHAPE;
  rc = check_ptrs(x, w_router, logits, topk_ids, topk_w, counts, offsets, perm, inv_perm, block_map, num_blocks);
  if (rc) return rc;
  const size_t need = route_workspace_bytes(T, E, k);
  if (need > 0) {
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
    rc = check_ptrs(workspace);
    if (rc) return rc;
  }
  if (!device_error_ptr()) return MOE_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  rc = cuda_status(launch_router(x, w_router, T, H, E, k, logits, topk_ids, topk_w, s));
  if (rc) return rc;
  return cuda_status(launch_route(logits, T, E, k, block_n, topk_ids, topk_w, counts, offsets, perm, inv_perm,
                                  block_map, num_blocks, workspace, workspace_bytes, s, 1));
}

int moe_expert_gemm_w4(int mode, int impl, const uint16_t* act, int T, int H, int F, int E, int k,
                       const void* w_packed, const int32_t* perm, const float* topk_w, const int32_t* block_map,
                       const int32_t* num_blocks, int block_n, void* out, moe_stream_t stream) {
  int rc = check_shape(T, H, F, E, k, block_n);
  if (rc) return rc;
  if (mode != MOE_GATE_UP_SWIGLU && mode != MOE_DOWN) return MOE_ERR_MODE;
  rc = check_ptrs(act, w_packed, perm, topk_w, block_map, num_blocks, out);
  if (rc) return rc;
  if (impl == MOE_IMPL_AUTO) impl = block_n <= gemv_max_rows() ? MOE_IMPL_GEMV : MOE_IMPL_TC;
  if (impl != MOE_IMPL_GEMV && impl != MOE_IMPL_TC && impl != MOE_IMPL_TC2 && impl != MOE_IMPL_TC_BF16)
    return MOE_ERR_MODE;
  // the kernels step K and M by 128; the GEMV takes tiles of at most 8 rows, the tensor-core kernels
  // 128, the CTA-pair kernel 256
  if (H % 128 != 0 || F % 128 != 0) return MOE_ERR_SHAPE;
  if (block_n > (impl == MOE_IMPL_GEMV ? gemv_max_rows() : impl == MOE_IMPL_TC2 ? 256 : 128)) return MOE_ERR_SHAPE;
  if (!device_error_ptr()) return MOE_ERR_CUDA;
  const int cap = moe_block_map_capacity(T, E, k, block_n);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (impl == MOE_IMPL_GEMV)
    return cuda_status(launch_gemm_gemv(mode, act, T, H, F, E, k, w_packed, perm, topk_w, block_map, num_blocks,
                                        block_n, cap, out, num_sms(), s));
  if (impl == MOE_IMPL_TC2)
    return cuda_status(launch_gemm_pair(mode, act, T, H, F, E, k, w_packed, perm, block_map, num_blocks, block_n,
                                        cap, out, s));
  return cuda_status(launch_gemm_tc(mode, act, T, H, F, E, k, w_packed, perm, topk_w, block_map, num_blocks,
                                    block_n, cap, out, num_sms(), s, impl == MOE_IMPL_TC_BF16, nullptr, nullptr,
                                    nullptr));
}

int moe_expert_ffn_w4(const uint16_t* x, int T, int H, int F, int E, int k, const void* w13, const void* w2,
                      const int32_t* perm, const int32_t* block_map, const int32_t* num_blocks, int block_n,
                      uint16_t* y, moe_stream_t stream) {
  int rc = check_shape(T, H, F, E, k, block_n);
  if (rc) return rc;
  if (H % 128 != 0 || F % 256 != 0 || block_n > 64) return MOE_ERR_SHAPE;
  rc = check_ptrs(x, w13, w2, perm, block_map, num_blocks, y);
  if (rc) return rc;
  if (!device_error_ptr()) return MOE_ERR_CUDA;
  const int cap = moe_block_map_capacity(T, E, k, block_n);
  return cuda_status(launch_ffn_tc(x, T, H, F, E, k, w13, w2, perm, block_map, num_blocks, block_n, cap, y, num_sms(),
                                   reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_down_combine_workspace_size(int T, int H) {
  if (T < 1 || T > (1 << 20) || H < 128 || H % 128 != 0) return 0;
  return static_cast<size_t>(T) * (H / 128) * sizeof(int32_t);
}

int moe_down_combine(const uint16_t* h, int T, int H, int F, int E, int k, const void* w_packed, const int32_t* perm,
                     const int32_t* inv_perm, const float* topk_w, const int32_t* block_map,
                     const int32_t* num_blocks, int block_n, uint16_t* y, uint16_t* out, void* workspace,
                     size_t workspace_bytes, moe_stream_t stream) {
  int rc = check_shape(T, H, F, E, k, block_n);
  if (rc) return rc;
  if (H % 128 != 0 || F % 128 != 0 || block_n > 128) return MOE_ERR_SHAPE;
  rc = check_ptrs(h, w_packed, perm, inv_perm, topk_w, block_map, num_blocks, y, out, workspace);
  if (rc) return rc;
  if (workspace_bytes < moe_down_combine_workspace_size(T, H)) return MOE_ERR_WORKSPACE;
  if (!device_error_ptr()) return MOE_ERR_CUDA;
  const int cap = moe_block_map_capacity(T, E, k, block_n);
  return cuda_status(launch_gemm_tc(MOE_DOWN, h, T, H, F, E, k, w_packed, perm, topk_w, block_map, num_blocks,
                                    block_n, cap, y, num_sms(), reinterpret_cast<cudaStream_t>(stream), false, out,
                                    inv_perm, static_cast<int*>(workspace)));
}

size_t moe_expanded_bytes(int n_mat, int rows, int K) {
  if (n_mat < 1 || rows < 128 || rows % 128 != 0 || K < 64 || K % 64 != 0) return 0;
  return expanded_bytes(n_mat, rows, K);
}

int moe_expand_w4(const void* w_repacked, int n_mat, int rows, int K, void* out, moe_stream_t stream) {
  if (n_mat < 1 || rows < 128 || rows % 128 != 0 || K < 64 || K % 64 != 0) return MOE_ERR_SHAPE;
  int rc = check_ptrs(w_repacked, out);
  if (rc) return rc;
  return cuda_status(launch_expand(w_repacked, n_mat, rows, K, out, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_combine(const uint16_t* y, const int32_t* inv_perm, const float* topk_w, uint16_t* out, int T, int H,
                int k, moe_stream_t stream) {
  if (T < 1 || T > (1 << 20) || H < 8 || H % 8 != 0 || k < 1 || k > 32) return MOE_ERR_SHAPE;
  int rc = check_ptrs(y, inv_perm, topk_w, out);
  if (rc) return rc;
  if (!device_error_ptr()) return MOE_ERR_CUDA;
  return cuda_status(
      launch_combine(y, inv_perm, topk_w, out, T, H, k, num_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_decode_workspace_size(int T, int H) {
  if (T < 1 || T > decode_max_tokens() || H < 64 || H % 32 != 0) return 0;
  return decode_workspace_bytes(T, H);
}

// The layer.  chosen: the experts are chosen by `gate`, or without logits have been and stand in the buffers;
// else moe_route's way.  residual: what follows the combine's sum (null: it is written to out).
static int layer_forward(const uint16_t* x, const float* logits, bool chosen, const moe_gate_t* gate, uint16_t* out,
                         const moe_residual_t* residual, int T, int H, int F, int E, int k, int block_n, int impl,
                         const moe_weights_t* w, const moe_buffers_t* b, moe_stream_t stream) {
  auto combine = [&]() -> int {
    if (residual) return moe_combine_residual_norm(b->y, b->inv_perm, b->topk_w, T, H, k, residual, stream);
    return moe_combine(b->y, b->inv_perm, b->topk_w, out, T, H, k, stream);
  };
  const bool gemv = impl == MOE_IMPL_GEMV || (impl == MOE_IMPL_AUTO && block_n <= gemv_max_rows());
  if (gemv && b->decode_ws && T <= decode_max_tokens() && k <= 32) {
    // the fused decode kernel: routing, both GEMVs and the combine in one launch
    int rc = check_shape(T, H, F, E, k, block_n);
    if (rc) return rc;
    if (block_n > gemv_max_rows() || H % 128 != 0 || F % 128 != 0) return MOE_ERR_SHAPE;
    rc = check_ptrs(x, w->w13, w->w2, b->topk_ids, b->topk_w, b->counts, b->offsets, b->perm, b->inv_perm,
                    b->block_map, b->num_blocks, b->h, b->y, b->decode_ws);
    if (rc) return rc;
    // (in the place of what the call does without: x)
    rc = check_ptrs(chosen && !logits ? static_cast<const void*>(x) : logits,
                    residual ? static_cast<const void*>(x) : out);
    if (rc) return rc;
    if (b->decode_ws_bytes < decode_workspace_bytes(T, H)) return MOE_ERR_WORKSPACE;
    if (!device_error_ptr()) return MOE_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (chosen && logits && (rc = cuda_status(launch_gate(logits, T, gate, E, k, b->topk_ids, b->topk_w, s)))) return rc;
    rc = cuda_status(launch_decode(x, chosen ? nullptr : logits, w->w13, w->w2, T, H, F, E, k, block_n, b->topk_ids,
                                   b->topk_w, b->counts, b->offsets, b->perm, b->inv_perm, b->block_map, b->num_blocks,
                                   b->h, b->y, residual ? nullptr : out, b->decode_ws, wait_limit_ns(), num_sms(), s));
    return rc || !residual ? rc : combine();
  }
  int rc = chosen ? moe_route_gated(logits, T, E, k, gate, block_n, b->topk_ids, b->topk_w, b->counts, b->offsets,
                                    b->perm, b->inv_perm, b->block_map, b->num_blocks, b->workspace, b->workspace_bytes,
                                    stream)
                  : moe_route(logits, T, E, k, block_n, b->topk_ids, b->topk_w, b->counts, b->offsets, b->perm,
                              b->inv_perm, b->block_map, b->num_blocks, b->workspace, b->workspace_bytes, stream);
  if (rc) return rc;
  const int resolved = impl == MOE_IMPL_AUTO ? (block_n <= gemv_max_rows() ? MOE_IMPL_GEMV : MOE_IMPL_TC) : impl;
  const bool in_epilogue = b->combine_ws && !residual;
  if (resolved == MOE_IMPL_TC && !in_epilogue && block_n <= 64 && H % 128 == 0 && F % 256 == 0) {
    // tiles of at most 64 rows: both projections of a tile in one launch, h kept in shared memory
    // (the same bits of y; measured faster than the two GEMMs at these tile heights)
    rc = moe_expert_ffn_w4(x, T, H, F, E, k, w->w13, w->w2, b->perm, b->block_map, b->num_blocks, block_n, b->y,
                           stream);
    return rc ? rc : combine();
  }
  rc = moe_expert_gemm_w4(MOE_GATE_UP_SWIGLU, impl, x, T, H, F, E, k, w->w13, b->perm, b->topk_w, b->block_map,
                          b->num_blocks, block_n, b->h, stream);
  if (rc) return rc;
  if (resolved == MOE_IMPL_TC && in_epilogue) {
    // the down GEMM with the combine in its epilogue (one launch fewer, y read back from L2 at once)
    return moe_down_combine(b->h, T, H, F, E, k, w->w2, b->perm, b->inv_perm, b->topk_w, b->block_map,
                            b->num_blocks, block_n, b->y, out, b->combine_ws, b->combine_ws_bytes, stream);
  }
  rc = moe_expert_gemm_w4(MOE_DOWN, impl, b->h, T, H, F, E, k, w->w2, b->perm, b->topk_w, b->block_map,
                          b->num_blocks, block_n, b->y, stream);
  return rc ? rc : combine();
}

int moe_layer_forward(const uint16_t* x, const float* logits, uint16_t* out, int T, int H, int F, int E, int k,
                      int block_n, int impl, const moe_weights_t* w, const moe_buffers_t* b, moe_stream_t stream) {
  if (!w || !b) return MOE_ERR_NULL;
  return layer_forward(x, logits, false, nullptr, out, nullptr, T, H, F, E, k, block_n, impl, w, b, stream);
}

int moe_layer_forward_gated(const uint16_t* x, const float* logits, const moe_gate_t* gate, uint16_t* out,
                            const moe_residual_t* residual, int T, int H, int F, int E, int k, int block_n, int impl,
                            const moe_weights_t* w, const moe_buffers_t* b, moe_stream_t stream) {
  if (!w || !b) return MOE_ERR_NULL;
  // the choice and what follows the experts are checked before anything is enqueued
  int rc = check_shape(T, H, F, E, k, block_n);
  if (rc || (logits && (rc = check_gate(gate, E, k)))) return rc;
  if (!aligned16(logits)) return MOE_ERR_ALIGN;
  if (residual) {
    ResidualArgs a;
    if ((rc = check_ptrs(b->y)) || (rc = residual_args(b->y, H, (k + 1ll) * T, true, T, H, residual, &a))) return rc;
    if ((rc = check_places_overlap(b->inv_perm, b->topk_w, T, H, k, residual))) return rc;
  } else if ((rc = check_ptrs(out))) {
    return rc;
  }
  if (logits && (rc = check_gate_overlap(logits, T, E, k, gate, b->topk_ids, b->topk_w))) return rc;
  return layer_forward(x, logits, true, gate, out, residual, T, H, F, E, k, block_n, impl, w, b, stream);
}

int moe_kv_append(const uint16_t* k, int64_t k_token_stride, int64_t k_head_stride, const uint16_t* v,
                  int64_t v_token_stride, int64_t v_head_stride, const moe_kv_cache_t* cache,
                  const moe_kv_batch_t* batch, moe_stream_t stream) {
  kv::Args a;
  int rc = kv_args(cache, batch, &a);
  if (rc) return rc;
  if (!kv_strides_ok(k_token_stride, k_head_stride, a.T, a.heads) ||
      !kv_strides_ok(v_token_stride, v_head_stride, a.T, a.heads))
    return MOE_ERR_SHAPE;
  if (a.T == 0) return MOE_OK;
  rc = check_ptrs(k, v);
  if (rc) return rc;
  if (!(a.err = device_error_ptr())) return MOE_ERR_CUDA;
  return cuda_status(launch_kv_append(a, cache->format == MOE_KV_E4M3, k, k_token_stride, k_head_stride, v,
                                      v_token_stride, v_head_stride, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_kv_read(uint16_t* k, uint16_t* v, const moe_kv_cache_t* cache, const moe_kv_batch_t* batch,
                moe_stream_t stream) {
  kv::Args a;
  int rc = kv_args(cache, batch, &a);
  if (rc) return rc;
  if (a.T == 0) return MOE_OK;
  rc = check_ptrs(k, v);
  if (rc) return rc;
  if (!(a.err = device_error_ptr())) return MOE_ERR_CUDA;
  return cuda_status(
      launch_kv_read(a, cache->format == MOE_KV_E4M3, k, v, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_kv_attention_workspace_size(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, int q_heads) {
  kv::Args a;
  if (kv_args(cache, batch, &a) || q_heads < 1 || q_heads % a.heads != 0) return 0;
  return kv_attention_workspace_bytes(a, cache->format == MOE_KV_E4M3, q_heads);
}

int moe_kv_attention(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, int q_heads, float scale,
                     const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, uint16_t* out, float* lse,
                     void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  kv::Args a;
  int rc = kv_args(cache, batch, &a);
  if (rc) return rc;
  if (q_heads < 1 || q_heads % a.heads != 0 || q_heads / a.heads > 128) return MOE_ERR_SHAPE;
  if (!kv_strides_ok(q_token_stride, q_head_stride, a.T, q_heads)) return MOE_ERR_SHAPE;
  // scores are multiplied by scale * log2(e), which an infinite one would make NaN where they are 0
  if (!(scale > 0.0f) || !(scale * 1.44269504088896341f <= FLT_MAX)) return MOE_ERR_SHAPE;
  if (a.T == 0) return MOE_OK;
  rc = check_ptrs(q, out);
  if (rc) return rc;
  if (reinterpret_cast<uintptr_t>(lse) & 3u) return MOE_ERR_ALIGN;
  if (workspace_bytes < kv_attention_workspace_bytes(a, cache->format == MOE_KV_E4M3, q_heads))
    return MOE_ERR_WORKSPACE;
  rc = check_ptrs(workspace);
  if (rc) return rc;
  if (!(a.err = device_error_ptr())) return MOE_ERR_CUDA;
  return cuda_status(launch_kv_attention(a, cache->format == MOE_KV_E4M3, q, q_token_stride, q_head_stride, q_heads,
                                         scale, out, lse, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

// The device's address of host memory it can read and write directly (pinned or registered, and
// mapped), or nullptr (pageable memory, or an address the runtime does not know).
static void* host_device_view(const void* host) {
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, host) != cudaSuccess) {
    cudaGetLastError();  // an unknown pointer is not an error of this call
    return nullptr;
  }
  return a.type == cudaMemoryTypeHost ? a.devicePointer : nullptr;
}

int moe_layer_forward_host(const uint16_t* x_host, const float* logits_host, uint16_t* out_host, uint16_t* x_dev,
                           float* logits_dev, uint16_t* out_dev, int T, int H, int F, int E, int k, int block_n,
                           int impl, const moe_weights_t* w, const moe_buffers_t* b, moe_stream_t stream) {
  if (!x_host || !logits_host || !out_host) return MOE_ERR_NULL;
  int rc = check_shape(T, H, F, E, k, block_n);
  if (rc) return rc;
  rc = check_ptrs(x_dev, logits_dev, out_dev);
  if (rc) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const size_t xb = static_cast<size_t>(T) * H * sizeof(uint16_t);
  const size_t lb = static_cast<size_t>(T) * E * sizeof(float);
  // Pinned host buffers are read and written by the kernels over the host link where each byte
  // crosses it once anyway: the routing (or fused decode) kernel reads every logit once, and the
  // combine writes out straight to out_host, which saves two copy-engine operations and their
  // latency per call.  x, which the grouped GEMM gathers k + 1 times, is copied to x_dev first.
  // Pageable buffers go through logits_dev / out_dev with copies.
  const float* logits_view = static_cast<const float*>(host_device_view(logits_host));
  uint16_t* out_view = static_cast<uint16_t*>(host_device_view(out_host));
  if (logits_view && !aligned16(logits_view)) logits_view = nullptr;
  if (out_view && !aligned16(out_view)) out_view = nullptr;
  if (cudaMemcpyAsync(x_dev, x_host, xb, cudaMemcpyHostToDevice, s) != cudaSuccess) return MOE_ERR_CUDA;
  if (!logits_view &&
      cudaMemcpyAsync(logits_dev, logits_host, lb, cudaMemcpyHostToDevice, s) != cudaSuccess)
    return MOE_ERR_CUDA;
  rc = moe_layer_forward(x_dev, logits_view ? logits_view : logits_dev, out_view ? out_view : out_dev, T, H, F, E, k,
                         block_n, impl, w, b, stream);
  if (rc) return rc;
  if (!out_view && cudaMemcpyAsync(out_host, out_dev, xb, cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

int moe_get_device_error(int32_t* code) {
  if (!code) return MOE_ERR_NULL;
  if (cudaDeviceSynchronize() != cudaSuccess) return MOE_ERR_CUDA;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, MOE_ERROR_SYMBOL, sizeof(int)) != cudaSuccess) return MOE_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpyToSymbol(MOE_ERROR_SYMBOL, &zero, sizeof(int)) != cudaSuccess) return MOE_ERR_CUDA;
  *code = v;
  return MOE_OK;
}

size_t moe_repacked_bytes(int n_mat, int rows, int K) {
  if (n_mat < 1 || rows < 128 || rows % 128 != 0 || K < 64 || K % 64 != 0) return 0;
  return repacked_bytes(n_mat, rows, K);
}

int moe_repack_w4(const uint32_t* packed, const uint16_t* scale, const uint16_t* bias, int n_mat, int rows, int K,
                  int gate_up, void* out, moe_stream_t stream) {
  if (n_mat < 1 || rows < 128 || rows % 128 != 0 || K < 64 || K % 64 != 0) return MOE_ERR_SHAPE;
  if (gate_up < 0 || gate_up > 2) return MOE_ERR_MODE;
  if (gate_up == 1 && (rows / 2) % 128 != 0) return MOE_ERR_SHAPE;
  if (gate_up == 2 && (rows / 2) % 64 != 0) return MOE_ERR_SHAPE;
  int rc = check_ptrs(packed, scale, bias, out);
  if (rc) return rc;
  return cuda_status(launch_repack(packed, scale, bias, n_mat, rows, K, gate_up, out,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

void moe_set_wait_limit_ns(uint64_t ns) { set_wait_limit_ns(ns); }

int moe_exchange_capture_mode(int32_t* mode) {
  if (!mode) return MOE_ERR_NULL;
  if (*mode < 0 || *mode > 2) return MOE_ERR_MODE;
  static_assert(cudaStreamCaptureModeGlobal == 0 && cudaStreamCaptureModeThreadLocal == 1 && cudaStreamCaptureModeRelaxed == 2, "");
  cudaStreamCaptureMode m = static_cast<cudaStreamCaptureMode>(*mode);
  if (cudaThreadExchangeStreamCaptureMode(&m) != cudaSuccess) return MOE_ERR_CUDA;
  *mode = m;
  return MOE_OK;
}

size_t moe_trace_words(void) {
#ifdef MOE_TRACE
  return moe::TRACE_WORDS;
#else
  return 0;
#endif
}

int moe_trace_reset(moe_stream_t stream) {
#ifdef MOE_TRACE
  int* err = moe::device_error_ptr();
  if (!err) return MOE_ERR_CUDA;
  return moe::cuda_status(cudaMemsetAsync(err + moe::TRACE_ERR_INTS, 0,
                                          moe::TRACE_WORDS * sizeof(unsigned long long),
                                          reinterpret_cast<cudaStream_t>(stream)));
#else
  (void)stream;
  return MOE_ERR_MODE;
#endif
}

int moe_trace_read(uint64_t* host, size_t words) {
#ifdef MOE_TRACE
  if (!host) return MOE_ERR_NULL;
  int* err = moe::device_error_ptr();
  if (!err) return MOE_ERR_CUDA;
  const size_t n = words < moe::TRACE_WORDS ? words : moe::TRACE_WORDS;
  return cudaMemcpy(host, err + moe::TRACE_ERR_INTS, n * sizeof(uint64_t), cudaMemcpyDeviceToHost) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
#else
  (void)host;
  (void)words;
  return MOE_ERR_MODE;
#endif
}

}  // extern "C"
