// qk_norm_rope.cuh -- launch arguments of the q/k norm with rotation.
#pragma once

#include "photon_common.cuh"

namespace photon {

struct QkNormRopeArgs {
  const void* q;
  const void* k;
  const void* q_weight;      // null: no norm
  const void* k_weight;
  const int32_t* positions;  // [num_axes][T]
  const float2* cs;          // [max_pos][half] (cos, sin)
  void* q_out;
  void* k_out;
  uint32_t* err;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;   // elements from token to token
  float eps;
  int T, Hq, Hkv, D, max_pos, num_axes, dtype;
  int half;                  // pairs that turn: rotary_dim / 2
  uint32_t axis[4];          // two bits a pair: its axis (pair k in word k / 16)
};
cudaError_t launch_qk_norm_rope(const QkNormRopeArgs& a, cudaStream_t stream);

}  // namespace photon
