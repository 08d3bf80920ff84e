// row_access.cuh -- 8 elements of a head row at a time: loaded, widened to fp32,
// rounded and stored.
#pragma once

#include "photon_common.cuh"

namespace photon {

// 8 elements as they lie in memory, and widened.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T>& r, float* f) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    Elem<T>::widen(r.v[i], f + i * Elem<T>::kPerChunk);
}
__device__ __forceinline__ void store8(float* p, const float* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* f) {
  *reinterpret_cast<uint4*>(p) = make_uint4(Mma<T>::pack(f[0], f[1]), Mma<T>::pack(f[2], f[3]),
                                            Mma<T>::pack(f[4], f[5]), Mma<T>::pack(f[6], f[7]));
}

}  // namespace photon
