// Router logits to experts and weights (moe_gate; see moe_gate_dev.cuh for the
// choice itself).
#include "moe_gate_dev.cuh"
#include "moe_launch.cuh"

namespace moe {

int num_sms();

namespace {

using gate_dev::Gate;
using gate_dev::Mode;

constexpr int GATE_WARPS = 8;
// Tokens per SM and token of a warp: a warp takes two or four tokens where there are enough for all warps (4096
// tokens routed: one each 23.2 us, two 21.2, four 22.4; 262144: two 185, four 145 at that time).
constexpr int GATE_BATCH_ROWS = 12;

template <int EPL, int IDX, Mode MODE, int BATCH, bool WHOLE>
__global__ void __launch_bounds__(32 * GATE_WARPS, BATCH == 4 ? 3 : 1) gate_kernel(const float* logits, int T,
                                                               const __grid_constant__ Gate g, int32_t* ids, float* w) {
  constexpr int SEG = 32 / BATCH;
  const int lane = threadIdx.x & 31;
  wait_for_earlier();
  int t = (static_cast<int>(blockIdx.x) * GATE_WARPS + (threadIdx.x >> 5)) * BATCH;
  const int step = static_cast<int>(gridDim.x) * GATE_WARPS * BATCH;
  if (t >= T) return;
  const gate_dev::Lane me(g, lane);
  // One or two tokens: their logits are asked for before the biases are looked at (at that time 1 token 3.5 -> 3.2 us, 777 of 160
  // 6.4 -> 5.5, captured).  Four: where they are used, or they cost registers all along (262144 tokens 137 us against 129).
  constexpr bool EARLY = BATCH < 4;
  float l[BATCH][EPL];
  if (EARLY) gate_dev::load_tokens<EPL, BATCH, WHOLE>(logits, t, T, g, me, l);
  const gate_dev::Units<EPL, IDX, MODE> units(g, me);
  while (t < T) {
    if (!EARLY) gate_dev::load_tokens<EPL, BATCH, WHOLE>(logits, t, T, g, me, l);
    int id;
    float x;
    gate_dev::warp_gate<EPL, IDX, MODE, BATCH, WHOLE>(logits, t, T, l, units, g, me, lane, &id, &x);
    if (t + lane / SEG < T && lane % SEG < g.k) {
      const size_t at = static_cast<size_t>(t + lane / SEG) * g.k + lane % SEG;
      ids[at] = id;
      w[at] = x;
    }
    t += step;
    if (EARLY && t < T) gate_dev::load_tokens<EPL, BATCH, WHOLE>(logits, t, T, g, me, l);
  }
}

template <int EPL, int IDX, Mode MODE, int BATCH, bool WHOLE>
cudaError_t launch(const float* logits, int T, const Gate& g, int32_t* ids, float* w, cudaStream_t s) {
  const auto kernel = gate_kernel<EPL, IDX, MODE, BATCH, WHOLE>;
  int per_sm = 0;
  const cudaError_t e = cached_occupancy(reinterpret_cast<const void*>(kernel), 32 * GATE_WARPS, 0, &per_sm);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return launch_early(kernel, min(ceil_div(T, GATE_WARPS * BATCH), num_sms() * per_sm), 32 * GATE_WARPS, 0, s, logits, T, g,
                      ids, w);
}

template <int EPL, int IDX, Mode MODE, bool WHOLE>
cudaError_t launch_batch(const float* logits, int T, const Gate& g, int32_t* ids, float* w, cudaStream_t s) {
  int batch = gate_dev::batch_of(g, EPL);
  while (batch > 1 && T < batch * GATE_BATCH_ROWS * num_sms()) batch >>= 1;
  if (EPL <= 8 && batch == 4) return launch<EPL, IDX, MODE, EPL <= 8 ? 4 : 1, WHOLE>(logits, T, g, ids, w, s);
  if (EPL <= 16 && batch == 2) return launch<EPL, IDX, MODE, EPL <= 16 ? 2 : 1, WHOLE>(logits, T, g, ids, w, s);
  return launch<EPL, IDX, MODE, 1, WHOLE>(logits, T, g, ids, w, s);
}

// Whole lanes (16-byte loads, keys without a branch for lanes' ends) are built for eight experts a lane, which 256 make:
// 262144 tokens, sigmoid, 4 of 8 groups 128.8 us, 136.0 without; softmax without bias 109 and 122; 4096 tokens 7.3 and 7.9.
template <Mode MODE>
cudaError_t launch_mode(const float* logits, int T, const Gate& g, int32_t* ids, float* w, cudaStream_t s) {
  const bool whole = g.per_group % g.width == 0 && 32 >> g.lanes_log == g.groups;
  if (g.E > 256) {  // keys of ten index bits
    if (g.width <= 16) return launch_batch<16, 10, MODE, false>(logits, T, g, ids, w, s);
    if (g.width > 32) return launch_batch<64, 10, MODE, false>(logits, T, g, ids, w, s);
    return launch_batch<32, 10, MODE, false>(logits, T, g, ids, w, s);
  }
  if (g.width <= 4) return launch_batch<4, 8, MODE, false>(logits, T, g, ids, w, s);
  if (g.width > 8) return launch_batch<16, 8, MODE, false>(logits, T, g, ids, w, s);
  return whole && g.width == 8 ? launch_batch<8, 8, MODE, true>(logits, T, g, ids, w, s)
                               : launch_batch<8, 8, MODE, false>(logits, T, g, ids, w, s);
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
  if (g.by_logit) return launch_mode<gate_dev::BY_LOGIT>(logits, T, g, ids, w, s);
  return g.softmax ? launch_mode<gate_dev::SOFTMAX>(logits, T, g, ids, w, s)
                   : launch_mode<gate_dev::SIGMOID>(logits, T, g, ids, w, s);
}

}  // namespace moe
