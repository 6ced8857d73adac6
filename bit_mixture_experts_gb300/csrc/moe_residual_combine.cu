// The combine with the residual addition that follows it (moe_residual.cu): y is
// each token's weighted sum of its expert rows and its shared expert's row.
#include "moe_residual_rows.cuh"

namespace moe {

cudaError_t launch_combine_residual(const ResidualArgs& p, bool vec, bool x32, cudaStream_t s) {
  if (vec) return x32 ? residual::launch<true, true, true>(p, s) : residual::launch<true, false, true>(p, s);
  return x32 ? residual::launch<false, true, true>(p, s) : residual::launch<false, false, true>(p, s);
}

}  // namespace moe
