// Router logits to experts and weights (moe_gate; see moe_gate_dev.cuh for the
// choice itself): one warp per token.
#include "moe_gate_dev.cuh"

namespace moe {

namespace {

using gate_dev::Gate;

constexpr int GATE_WARPS = 8;

template <int EPL, bool VEC>
__global__ void __launch_bounds__(32 * GATE_WARPS) gate_kernel(const float* logits, int T,
                                                               const __grid_constant__ Gate g, int32_t* ids, float* w) {
  const int lane = threadIdx.x & 31;
  const int t = static_cast<int>(blockIdx.x) * GATE_WARPS + (threadIdx.x >> 5);
  if (t >= T) return;
  int id;
  float x;
  gate_dev::warp_gate<EPL, VEC>(logits + static_cast<size_t>(t) * g.E, g, lane, &id, &x);
  if (lane < g.k) {
    ids[static_cast<size_t>(t) * g.k + lane] = id;
    w[static_cast<size_t>(t) * g.k + lane] = x;
  }
}

template <int EPL, bool VEC>
cudaError_t launch(const float* logits, int T, const Gate& g, int32_t* ids, float* w, cudaStream_t s) {
  gate_kernel<EPL, VEC><<<ceil_div(T, GATE_WARPS), 32 * GATE_WARPS, 0, s>>>(logits, T, g, ids, w);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace

// A checked moe_gate_t as the kernels take it.
Gate make_gate(const moe_gate_t* p, int E, int k) {
  Gate g;
  g.bias = p->bias;
  g.E = E;
  g.k = k;
  g.groups = p->groups;
  g.per_group = E / p->groups;
  g.top_groups = p->top_groups;
  g.lanes_log = 5;
  while ((32 >> g.lanes_log) < p->groups) --g.lanes_log;
  g.width = ceil_div(g.per_group, 1 << g.lanes_log);
  g.softmax = p->score == MOE_SCORE_SOFTMAX;
  g.top2 = p->group_score == MOE_GROUP_TOP2;
  g.renorm = p->renorm != 0;
  g.by_logit = !p->bias && (p->top_groups == p->groups || !g.top2);
  g.scale = p->scale;
  return g;
}

cudaError_t launch_gate(const float* logits, int T, const moe_gate_t* p, int E, int k, int32_t* ids, float* w,
                        cudaStream_t s) {
  const Gate g = make_gate(p, E, k);
  const bool vec = g.width % 4 == 0 && g.per_group % g.width == 0;
  if (g.width <= 1) return launch<1, false>(logits, T, g, ids, w, s);
  if (g.width <= 2) return launch<2, false>(logits, T, g, ids, w, s);
  if (g.width <= 4) return vec ? launch<4, true>(logits, T, g, ids, w, s) : launch<4, false>(logits, T, g, ids, w, s);
  if (g.width <= 8) return vec ? launch<8, true>(logits, T, g, ids, w, s) : launch<8, false>(logits, T, g, ids, w, s);
  if (g.width <= 16) return vec ? launch<16, true>(logits, T, g, ids, w, s) : launch<16, false>(logits, T, g, ids, w, s);
  if (g.width <= 32) return vec ? launch<32, true>(logits, T, g, ids, w, s) : launch<32, false>(logits, T, g, ids, w, s);
  return launch<64, false>(logits, T, g, ids, w, s);
}

}  // namespace moe
