// What the residual addition's entry points (moe_abi.cu) hand to its kernels
// (moe_residual.cu).
#pragma once
#include "moe_common.cuh"

namespace moe {

struct ResidualArgs {
  const uint16_t* y;
  long long y_stride;
  const int32_t* inv_perm;  // combine: y's rows; k experts per token
  const float* topk_w;
  int k;
  int T, H;
  const void* x;
  long long x_stride;
  void* r;
  long long r_stride;
  uint16_t* n;
  long long n_stride;
  const void* w_pre;
  const void* w_post;
  const void* gate;
  long long gate_token;
  int gate_channel;
  float offset, scale, eps;
  bool post, param_f32, gate_f32;
  int* err;
};

}  // namespace moe
