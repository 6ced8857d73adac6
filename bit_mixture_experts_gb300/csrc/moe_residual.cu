// A block's residual addition between the norm of what the block gave and the
// norm of what the next one takes:
//
//   z = y / rms(y) * (w_post + offset)      (or y itself)
//   r = scale x + gate z                    (the residual stream)
//   n = r / rms(r) * (w_pre + offset)       rms(v) = sqrt(mean v^2 + eps)
//
// where y is a dense tensor, or each token's weighted sum of its expert rows and
// its shared expert's row (moe_combine's sum, not rounded in between).
//
// One pass: a row's values stay in its threads' registers between the two
// sums, so every input is read and every output written once.  All sums and
// products in FP32, r and n rounded once.
#include "moe_residual_rows.cuh"

namespace moe {

cudaError_t launch_combine_residual(const ResidualArgs& p, bool vec, bool x32, cudaStream_t s);

constexpr int RESIDUAL_MAX_H = 32768;

int residual_max_h() { return RESIDUAL_MAX_H; }

cudaError_t launch_residual(const ResidualArgs& p, bool combine, bool x32, cudaStream_t s) {
  // rows in pieces of eight values, if every row of every tensor starts on 16 bytes
  auto ok = [](const void* ptr, long long stride, int size) {
    return (reinterpret_cast<uintptr_t>(ptr) | static_cast<uintptr_t>(stride * size)) % 16 == 0;
  };
  const int xs = x32 ? 4 : 2, ps = p.param_f32 ? 4 : 2;
  const bool vec = p.H % 8 == 0 && ok(p.x, p.x_stride, xs) && ok(p.y, p.y_stride, 2) && ok(p.r, p.r_stride, xs) &&
                   ok(p.n, p.n_stride, 2) && ok(p.w_pre, 0, ps) && ok(p.w_post, 0, ps) &&
                   (!p.gate_channel || ok(p.gate, p.gate_token, p.gate_f32 ? 4 : 2));
  if (combine) return launch_combine_residual(p, vec, x32, s);
  if (vec) return x32 ? residual::launch<true, true, false>(p, s) : residual::launch<true, false, false>(p, s);
  return x32 ? residual::launch<false, true, false>(p, s) : residual::launch<false, false, false>(p, s);
}

}  // namespace moe
