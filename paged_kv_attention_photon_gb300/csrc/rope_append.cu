// rope_append.cu -- q and k of new tokens turned by their positions, and k and v
// stored at their slots of the paged cache, in one pass over all three.
//
// PhotonInfer README, "Key features / GPU-optimized kernels" (batched RoPE) and
// "Technical details / Paged attention" (one kernel writes the K/V rows of many
// sequences).
//
// For pair k of a head row with (cos, sin) of the token's position
//   z[a] = x[a] cos - x[b] sin,  z[b] = x[b] cos + x[a] sin
// where (a, b) is (k, k + r/2), or (2k, 2k + 1) with neighbours paired; elements
// past r and all of v are copied.  A pass over memory: every row is read once and
// written once.  D / 16 lanes hold a row, each with two runs of 8 elements that
// hold both halves of its 8 pairs in either layout, so nothing crosses lanes and
// both layouts take the same eight (cos, sin); a warp takes one token's rows of all
// three tensors, a few of them a lane, all loaded before the first is used.
//
// Measured: 16 x 1024 tokens of 16 q and 8 kv heads x 128 in bf16, 39.9 us = 6.7 TB/s,
// 99.5 % of the measured copy rate, paired either way; ragged chunks of 32 + 8 + 8 heads
// x 64 in f32 34.6 us = 6.4 TB/s; 1024 tokens 3.6 us, a launch and one round trip.
#include "row_access.cuh"
#include "speculate.cuh"

namespace photon {
namespace {

constexpr int kAppendThreads = 64;   // with 32, 64, 128: 16 x 1024 tokens in 39.9 us each

__device__ __forceinline__ void turn(float a, float b, float2 cs, float& x, float& y) {
  x = a * cs.x - b * cs.y;
  y = b * cs.x + a * cs.y;
}

// kAppendHeads: head rows a lane takes, all loaded before the first is used
template <typename T, int D, int kAppendHeads>
__global__ void __launch_bounds__(kAppendThreads) rope_append_kernel(const RopeAppendArgs a) {
  constexpr int kLanes = D / 16, kGroups = 32 / kLanes;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int lane = threadIdx.x & 31, j = lane % kLanes, group = lane / kLanes;
  const int heads = a.Hq + 2 * a.Hkv;
  const int chunks = (heads + kGroups * kAppendHeads - 1) / (kGroups * kAppendHeads);
  const int64_t item = ((int64_t)blockIdx.x * kAppendThreads + threadIdx.x) >> 5;
  const int64_t t = item / chunks;
  if (t >= a.T) return;
  const int pos = __ldg(a.positions + t);
  const int64_t slot = __ldg(a.slots + t);
  const int h0 = (int)(item - t * chunks) * (kGroups * kAppendHeads) + group;

  // the lane's two runs of 8 elements; the first 2 half of a row turn
  const bool turned = 8 * j < a.half;
  const bool apart = turned && !a.interleaved;
  const int e0 = apart ? 8 * j : 16 * j;
  const int e1 = apart ? a.half + 8 * j : e0 + 8;

  Raw8<T> raw[kAppendHeads][2];
  const T* qrow = static_cast<const T*>(a.q) + t * a.q_stride;
  const T* krow = static_cast<const T*>(a.k) + t * a.k_stride - (int64_t)a.Hq * D;
  const T* vrow = static_cast<const T*>(a.v) + t * a.v_stride - (int64_t)(a.Hq + a.Hkv) * D;
#pragma unroll
  for (int i = 0; i < kAppendHeads; ++i) {
    const int h = min(h0 + i * kGroups, heads - 1);   // past the last head: loaded, not used
    const T* src = (h < a.Hq ? qrow : h < a.Hq + a.Hkv ? krow : vrow) + (int64_t)h * D;
    raw[i][0] = load8(src + e0);
    raw[i][1] = load8(src + e1);
  }
  if (pos < 0) return;   // padding

  const bool in_table = pos < a.max_pos;
  float2 cs[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) cs[e] = make_float2(1.f, 0.f);
  if (turned && in_table) {
    const float4* row = reinterpret_cast<const float4*>(a.cs + (int64_t)pos * a.half + 8 * j);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 w = __ldg(row + e);
      cs[2 * e] = make_float2(w.x, w.y);
      cs[2 * e + 1] = make_float2(w.z, w.w);
    }
  }
  const bool stored = slot >= 0 && slot < (int64_t)a.NB * kBlockSize;
  if (lane == 0 && item == t * chunks) {
    if (!in_table) raise_error(a.err, kErrPosition);
    if (slot >= 0 && !stored) raise_error(a.err, kErrSlot);
  }
  T* qdst = static_cast<T*>(a.q_out) + t * a.q_out_stride;
  // row h of the slot in a pool [block][Hkv][16][D]
  const int64_t at = stored ? ((slot / kBlockSize) * a.Hkv * kBlockSize + slot % kBlockSize) * D : 0;

#pragma unroll
  for (int i = 0; i < kAppendHeads; ++i) {
    const int h = h0 + i * kGroups;
    if (h >= heads) break;
    const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
    if (!is_q && !stored) continue;
    T* dst = is_q   ? qdst + (int64_t)h * D
             : is_v ? static_cast<T*>(a.v_cache) + at + (int64_t)(h - a.Hq - a.Hkv) * kBlockSize * D
                    : static_cast<T*>(a.k_cache) + at + (int64_t)(h - a.Hq) * kBlockSize * D;
    if (is_v || !turned || !in_table) {   // as it is, bit for bit
      reinterpret_cast<Raw8<T>*>(dst + e0)[0] = raw[i][0];
      reinterpret_cast<Raw8<T>*>(dst + e1)[0] = raw[i][1];
      continue;
    }
    float x[16], z[16];
    widen8<T>(raw[i][0], x);
    widen8<T>(raw[i][1], x + 8);
    if (apart) {
#pragma unroll
      for (int e = 0; e < 8; ++e) turn(x[e], x[8 + e], cs[e], z[e], z[8 + e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) turn(x[2 * e], x[2 * e + 1], cs[e], z[2 * e], z[2 * e + 1]);
    }
    store8(dst + e0, z);
    store8(dst + e1, z + 8);
  }
}

template <typename T, int D, int kHeads>
cudaError_t launch_heads(const RopeAppendArgs& a, cudaStream_t stream) {
  constexpr int kChunk = (32 / (D / 16)) * kHeads, kWarps = kAppendThreads / 32;
  const int64_t items = (int64_t)a.T * ((a.Hq + 2 * a.Hkv + kChunk - 1) / kChunk);
  const int64_t grid = (items + kWarps - 1) / kWarps;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(rope_append_kernel<T, D, kHeads>, dim3((unsigned)grid), dim3(kAppendThreads), 0,
                    stream, a);
}

// Four head rows a lane, or three where that leaves fewer places empty.  Four and
// three: 32 heads of 128 (36 places with three), 16 x 1024 tokens in bf16, 39.9 and 41.3
// us; 48 heads of 64 (64 places with four) 33.2 and 30.6, 7 800 tokens of them in f32
// 36.5 and 34.6.  (Two: 42.5, 32.4, 34.1; six 44.6, 30.9, 36.4.)
template <typename T, int D>
cudaError_t launch_t(const RopeAppendArgs& a, cudaStream_t stream) {
  constexpr int kGroups = 32 / (D / 16);
  const int heads = a.Hq + 2 * a.Hkv;
  auto places = [&](int each) { return (heads + kGroups * each - 1) / (kGroups * each) * each; };
  return places(3) < places(4) ? launch_heads<T, D, 3>(a, stream) : launch_heads<T, D, 4>(a, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendArgs& a, cudaStream_t stream) {
  switch (a.dtype) {
    case 0: return a.D == 64 ? launch_t<float, 64>(a, stream) : launch_t<float, 128>(a, stream);
    case 1: return a.D == 64 ? launch_t<__half, 64>(a, stream) : launch_t<__half, 128>(a, stream);
    default:
      return a.D == 64 ? launch_t<__nv_bfloat16, 64>(a, stream)
                       : launch_t<__nv_bfloat16, 128>(a, stream);
  }
}

}  // namespace photon
