// int4_common.cuh -- the 4-bit KV cache's record format and the launch
// arguments of its kernels (layout in include/photon_paged.h).
#pragma once

#include "photon_common.cuh"

namespace photon {

// Bytes of one (block, KV head) record: 16 rows of d / 2 code bytes, then 16
// (step, lo) pairs of two 16-bit values.
__host__ __device__ constexpr int int4_record_bytes(int d) { return 8 * d + 64; }

// 16-bit storage type as bits and as fp32.
template <typename T>
struct Bits16;
template <>
struct Bits16<__half> {
  static constexpr uint32_t kNan = 0x7e00u;
  __device__ __forceinline__ static float to_f32(uint32_t b) {
    return __half2float(__ushort_as_half((unsigned short)b));
  }
};
template <>
struct Bits16<__nv_bfloat16> {
  static constexpr uint32_t kNan = 0x7fc0u;
  __device__ __forceinline__ static float to_f32(uint32_t b) { return __uint_as_float(b << 16); }
};

struct CacheWriteInt4Args {
  const void* k;
  const void* v;
  int64_t k_stride, v_stride;   // elements from token to token
  const int64_t* slot_mapping;
  void* k_cache;
  void* v_cache;
  uint32_t* err;
  int T, Hkv, D, NB, dtype, num_sms;
};
cudaError_t launch_cache_write_int4(const CacheWriteInt4Args& a, cudaStream_t stream);

struct GatherInt4Args {
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  void* k_dense;
  void* v_dense;
  uint32_t* err;
  int B, Hkv, D, NB, MBS, dtype;
};
cudaError_t launch_gather_int4(const GatherInt4Args& a, cudaStream_t stream);

struct DecodeInt4Args {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  void* out;
  int2* ws_pair;   // [B][Hkv] first partial slot (the next is `team` on) and number of partials
  float2* ws_ml;   // [slot][G] running max (log2 domain) and sum of weights
  float* ws_o;     // [slot][G][D] unnormalised weighted V sum
  uint32_t* err;
  float qscale;    // scale * log2(e): scores are kept in the log2 domain
  int B, Hq, Hkv, D, NB, MBS, dtype;
  int num_sms, max_warps;
  int team;        // warps that walk the same blocks, one KV head each: 8, 4, 2 or 1
  cudaEvent_t ev_start, ev_stop;   // optional timing hook around the kernels
};
cudaError_t launch_paged_decode_int4(const DecodeInt4Args& a, cudaStream_t stream);
// Most warps the decode's attention grid has (the partials' slots are counted
// from it, so the workspace does not depend on the device).
constexpr int kInt4MaxWarps = 152 * 16;
constexpr int kInt4CtaWarps = 8;

}  // namespace photon
