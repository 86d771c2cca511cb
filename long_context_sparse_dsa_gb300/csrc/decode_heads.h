// decode_heads.h -- host side of the head norm kernels (internal to the library);
// arguments are validated in decode_heads_api.cu.
#pragma once

#include "decode.h"

namespace dsa {

struct HeadsArgs {
  int64_t n_tokens;
  int Hq, d;                        // Hq 0: no queries
  int64_t q_stride, k_stride;       // elements
  const void *q, *k;                // k NULL: no keys
  const float *q_weight, *k_weight;
  float eps;
  RotationArgs rot;
  const int32_t* positions;
  void *q_out, *k_out;              // forward
  const float *dq_out, *dk_out;     // gradient
  float *dq, *dk, *dq_weight, *dk_weight;
  float* ws;                        // [CTAs][2][d]: sums for the weights' gradients
};
cudaError_t launch_qk_norm_rotate(bool bf16, const HeadsArgs& a, cudaStream_t s);
size_t qk_norm_bwd_ws_bytes(int d);
cudaError_t launch_qk_norm_rotate_bwd(bool bf16, const HeadsArgs& a, cudaStream_t s);

}  // namespace dsa
