// qk_norm_rope.cu -- RMS norm of every q and k head row and its rotation by
// the token's position, on one axis or several, in one pass over both tensors.
//
// PhotonInfer README, "Key features / GPU-optimized kernels": batched RoPE and
// norms are among the fused kernels.
//
// For a head row x:  y = x / sqrt(mean(x^2) + eps) * w, then for pair k
//   z[k] = y[k] cos - y[k + r/2] sin,  z[k + r/2] = y[k + r/2] cos + y[k] sin
// with (cos, sin) of the position on the pair's axis.  It is a pass over
// memory, so a row is read once and written once: D / 16 lanes hold it, each
// with two runs of 8 elements that lie r/2 apart, so that both halves of every
// pair are in one lane and only the sum of squares crosses lanes (2 or 3
// shuffles).  A warp takes one token, so the (cos, sin) row is loaded once
// for all of the warp's heads, and three head rows a lane, all loaded before
// the first is used (with one row a lane in flight: 69 us where it is 35.0).
//
// Measured (16 q, 8 kv heads, d = 128, bf16): 16 x 1024 tokens in 35.0 us = 5.8
// TB/s, 85 % of the measured copy rate; 64 tokens in 2.6 us, a launch's time.
#include "photon_common.cuh"
#include "qk_norm_rope.cuh"
#include "row_access.cuh"

namespace photon {
namespace {

// Sum over the `kLanes` lanes of a row.
template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
template <int kLanes>
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// In one run with 32, 64, 96, 128, 256: 16 x 1024 tokens in 37.2, 34.6, 35.6, 35.4,
// 38.5 us, 6190 f32 tokens on three axes in 24.2, 24.8, 25.1, 25.3, 26.8
constexpr int kQkThreads = 64;
constexpr int kQkHeads = 3;   // head rows a lane takes, all loaded before the first is used

template <typename T, int D, bool kOneAxis>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_kernel(const QkNormRopeArgs a) {
  constexpr int kLanes = D / 16, kGroups = 32 / kLanes;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int lane = threadIdx.x & 31, j = lane % kLanes, group = lane / kLanes;
  const int heads = a.Hq + a.Hkv;
  const int chunks = (heads + kGroups * kQkHeads - 1) / (kGroups * kQkHeads);
  const int64_t item = ((int64_t)blockIdx.x * kQkThreads + threadIdx.x) >> 5;
  const int64_t t = item / chunks;
  if (t >= a.T) return;
  const int pos0 = __ldg(a.positions + t);
  if (pos0 < 0) return;   // padding
  const int h0 = (int)(item - t * chunks) * (kGroups * kQkHeads) + group;

  // the lane's two runs of 8 elements: both halves of its pairs, or, past the
  // turned part of the row, two neighbouring runs that only the norm changes
  const bool turned = 8 * j < a.half;
  const int e0 = turned ? 8 * j : 2 * a.half + 16 * (j - a.half / 8);
  const int e1 = turned ? a.half + 8 * j : e0 + 8;

  Raw8<T> raw[kQkHeads][2];
  const T* qrow = static_cast<const T*>(a.q) + t * a.q_stride;
  const T* krow = static_cast<const T*>(a.k) + t * a.k_stride - (int64_t)a.Hq * D;
#pragma unroll
  for (int i = 0; i < kQkHeads; ++i) {
    const int h = min(h0 + i * kGroups, heads - 1);   // past the last head: loaded, not used
    const T* src = (h >= a.Hq ? krow : qrow) + h * D;
    raw[i][0] = load8(src + e0);
    raw[i][1] = load8(src + e1);
  }

  T* qdst = static_cast<T*>(a.q_out) + t * a.q_out_stride;
  T* kdst = static_cast<T*>(a.k_out) + t * a.k_out_stride - (int64_t)a.Hq * D;

  // (cos, sin) of the lane's 8 pairs
  float2 cs[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) cs[e] = make_float2(1.f, 0.f);
  bool in_table = pos0 < a.max_pos;
  if constexpr (kOneAxis) {
    if (turned && in_table) {
      const float4* row =
          reinterpret_cast<const float4*>(a.cs + (int64_t)pos0 * a.half + 8 * j);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 w = __ldg(row + e);
        cs[2 * e] = make_float2(w.x, w.y);
        cs[2 * e + 1] = make_float2(w.z, w.w);
      }
    }
  } else {
    int pos[4];
#pragma unroll
    for (int x4 = 0; x4 < 4; ++x4) {
      pos[x4] = x4 < a.num_axes ? __ldg(a.positions + (int64_t)x4 * a.T + t) : 0;
      in_table = in_table && pos[x4] >= 0 && pos[x4] < a.max_pos;
    }
    if (turned && in_table) {
      // two bits a pair name its axis
      const uint32_t word = j < 2 ? a.axis[0] : j < 4 ? a.axis[1] : j < 6 ? a.axis[2] : a.axis[3];
      const uint32_t mine = word >> (16 * (j & 1));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t ax = (mine >> (2 * e)) & 3u;
        const int p = ax == 0 ? pos[0] : ax == 1 ? pos[1] : ax == 2 ? pos[2] : pos[3];
        cs[e] = __ldg(a.cs + (int64_t)p * a.half + 8 * j + e);
      }
    }
  }
  if (!in_table && lane == 0 && item == t * chunks) raise_error(a.err, kErrPosition);

#pragma unroll
  for (int i = 0; i < kQkHeads; ++i) {
    const int h = h0 + i * kGroups;
    const bool is_k = h >= a.Hq;
    const T* weight = static_cast<const T*>(is_k ? a.k_weight : a.q_weight);
    float x[16];
    widen8<T>(raw[i][0], x);
    widen8<T>(raw[i][1], x + 8);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
    ss = row_sum<kLanes>(ss);
    float mean = ss * (1.f / D), eps = a.eps;
    // squares that left fp32's range: the row is brought near 1 by a power of
    // two first (rows of a warp differ, so every lane takes the shuffles)
    const bool far_off = !(mean <= 1e36f) || mean + eps < 1e-30f;
    if (__any_sync(0xffffffffu, far_off)) {
      float big = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) big = fmaxf(big, fabsf(x[e]));
      big = row_max<kLanes>(big);
      const int ex = (int)((__float_as_uint(big) >> 23) & 255u);   // biased exponent
      // 2^-exponent, at most 2^100 (below that the squares are in range again)
      const float sc = far_off && ex < 255 ? __uint_as_float((uint32_t)max(1, min(254 - ex, 227)) << 23) : 1.f;
      float s2 = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float y = x[e] * sc;
        s2 = fmaf(y, y, s2);
      }
      s2 = row_sum<kLanes>(s2);
      if (far_off && weight) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= sc;
        mean = s2 * (1.f / D);
        eps = eps * sc * sc;
      }
    }
    if (h >= heads) continue;
    if (weight) {
      const float r = 1.f / sqrtf(mean + eps);
      float w[16];
      widen8<T>(load8(weight + e0), w);
      widen8<T>(load8(weight + e1), w + 8);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = x[e] * r * w[e];
    }
    float z[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      z[e] = turned && in_table ? x[e] * cs[e].x - x[8 + e] * cs[e].y : x[e];
      z[8 + e] = turned && in_table ? x[8 + e] * cs[e].x + x[e] * cs[e].y : x[8 + e];
    }
    T* dst = (is_k ? kdst : qdst) + h * D;
    store8(dst + e0, z);
    store8(dst + e1, z + 8);
  }
}

template <typename T, int D>
cudaError_t launch_t(const QkNormRopeArgs& a, cudaStream_t stream) {
  constexpr int kChunk = (32 / (D / 16)) * kQkHeads, kWarps = kQkThreads / 32;
  const int64_t items = (int64_t)a.T * ((a.Hq + a.Hkv + kChunk - 1) / kChunk);
  const int64_t grid = (items + kWarps - 1) / kWarps;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  return a.num_axes == 1
             ? launch_pdl(qk_norm_rope_kernel<T, D, true>, dim3((unsigned)grid), dim3(kQkThreads),
                          0, stream, a)
             : launch_pdl(qk_norm_rope_kernel<T, D, false>, dim3((unsigned)grid), dim3(kQkThreads),
                          0, stream, a);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRopeArgs& a, cudaStream_t stream) {
  switch (a.dtype) {
    case 0: return a.D == 64 ? launch_t<float, 64>(a, stream) : launch_t<float, 128>(a, stream);
    case 1: return a.D == 64 ? launch_t<__half, 64>(a, stream) : launch_t<__half, 128>(a, stream);
    default:
      return a.D == 64 ? launch_t<__nv_bfloat16, 64>(a, stream)
                       : launch_t<__nv_bfloat16, 128>(a, stream);
  }
}

}  // namespace photon
