// prompt_attention.cuh -- launch arguments of the packed prompt attention.
#pragma once

#include "photon_common.cuh"

namespace photon {

struct PromptArgs {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* query_start;   // [B + 1]
  void* out;
  uint32_t* err;
  int64_t q_stride, k_stride, v_stride, out_stride;   // elements from token to token
  float qscale;                 // scale * log2(e)
  int B, Hq, Hkv, D, num_tokens, max_query_len, dtype, num_sms;
};
cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t stream);

}  // namespace photon
