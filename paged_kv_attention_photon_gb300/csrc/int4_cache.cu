// int4_cache.cu -- the 4-bit KV cache: quantising write of new rows, and the
// contexts' rows read back as values.
//
// PhotonInfer README, "Technical details / Paged attention" (the K/V rows of
// many sequences are written by one kernel) and "Roadmap" (lower-precision KV).
//
// A row x (head_dim elements of one token and KV head) is held as
//   lo = min x,  step = rn16((max x - lo) / 15),
//   n  = clamp(rne((x - lo) / step), 0, 15),  value lo + n step.
// Both kernels move bytes: the write reads 2 d and writes d / 2 + 4 bytes a
// row, the gather the reverse, so one row's lanes load 16 contiguous bytes
// each and the arithmetic must stay below the memory time.  It runs in fp32,
// and only what fp32 cannot decide goes to double: a step whose fp32 value is
// within two units of the border between two 16-bit values, and an element
// whose quotient is within 1e-5 of a half (the fp32 quotient is off by less
// than 15 x 3 x 2^-24 = 2.7e-6).
#include "int4_common.cuh"

namespace photon {
namespace {

__device__ __forceinline__ __half2 min2_nan(__half2 a, __half2 b) { return __hmin2_nan(a, b); }
__device__ __forceinline__ __nv_bfloat162 min2_nan(__nv_bfloat162 a, __nv_bfloat162 b) {
  return __hmin2_nan(a, b);
}
__device__ __forceinline__ __half2 max2_nan(__half2 a, __half2 b) { return __hmax2_nan(a, b); }
__device__ __forceinline__ __nv_bfloat162 max2_nan(__nv_bfloat162 a, __nv_bfloat162 b) {
  return __hmax2_nan(a, b);
}

template <typename T>
struct Pair16;
template <>
struct Pair16<__half> { using type = __half2; };
template <>
struct Pair16<__nv_bfloat16> { using type = __nv_bfloat162; };

// (hi - lo) / 15 rounded once to the storage type, as bits; lo and hi are
// finite values of that type.
template <typename T>
__device__ __forceinline__ uint32_t int4_step_bits(float lo, float hi) {
  const float s = (hi - lo) / 15.f;
  const uint32_t b = __float_as_uint(s);
  if constexpr (sizeof(T) == 2 && Bits16<T>::kNan == 0x7e00u) {
    // fp16 keeps 10 of fp32's 23 fraction bits; below 2^-14 it keeps fewer
    if (((b & 0x1fffu) - 0x0ffeu) > 4u && s >= 6.103515625e-5f)
      return __half_as_ushort(__float2half_rn(s));
    return __half_as_ushort(__double2half(((double)hi - (double)lo) / 15.0));
  } else {
    // bf16 keeps 7; hi - lo may pass fp32's largest value
    if (((b & 0xffffu) - 0x7ffeu) > 4u && s >= 1e-36f && s <= 1e37f)
      return __bfloat16_as_ushort(__float2bfloat16_rn(s));
    return __bfloat16_as_ushort(__double2bfloat16(((double)hi - (double)lo) / 15.0));
  }
}

__device__ __forceinline__ float int4_code(float x, float lo, float step, float inv) {
  const float q = (x - lo) * inv;
  float n = rintf(q);
  if (!(fabsf(q - n) <= 0.5f - 1e-5f)) {
    // next to a border, or out of fp32's range
    n = (float)rint(((double)x - (double)lo) / (double)step);
  }
  return fminf(fmaxf(n, 0.f), 15.f);
}

constexpr int kWriteThreads = 256;
constexpr int kWriteUnroll = 4;   // rows a lane takes, all loaded before the first is used

// D / 8 lanes a row, 8 elements a lane.
template <typename T, int D>
__global__ void __launch_bounds__(kWriteThreads) cache_write_int4_kernel(CacheWriteInt4Args a) {
  using T2 = typename Pair16<T>::type;
  constexpr int kLanes = D / 8, kRowsPerWarp = 32 / kLanes;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int lane = threadIdx.x & 31, j = lane % kLanes;
  const bool is_v = blockIdx.y != 0;
  const int64_t rows = (int64_t)a.T * a.Hkv;
  const int64_t nslots = (int64_t)a.NB * kBlockSize;
  const int64_t warp = ((int64_t)blockIdx.x * kWriteThreads + threadIdx.x) >> 5;
  const int64_t row0 = warp * (kRowsPerWarp * kWriteUnroll) + lane / kLanes;
  const T* src = static_cast<const T*>(is_v ? a.v : a.k);
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  unsigned char* pool = static_cast<unsigned char*>(is_v ? a.v_cache : a.k_cache);

  uint4 raw[kWriteUnroll];
  int64_t slot[kWriteUnroll];
  int head[kWriteUnroll];
#pragma unroll
  for (int u = 0; u < kWriteUnroll; ++u) {
    const int64_t r = row0 + u * kRowsPerWarp;
    slot[u] = -1;
    raw[u] = make_uint4(0u, 0u, 0u, 0u);
    head[u] = 0;
    if (r < rows) {
      const int64_t t = r / a.Hkv;
      head[u] = (int)(r - t * a.Hkv);
      slot[u] = __ldg(a.slot_mapping + t);
      if (slot[u] >= nslots) {
        if (j == 0 && head[u] == 0 && !is_v) raise_error(a.err, kErrSlot);
        slot[u] = -1;
      }
      if (slot[u] >= 0) raw[u] = ld_stream16(src + t * stride + (int64_t)head[u] * D + 8 * j);
    }
  }
#pragma unroll
  for (int u = 0; u < kWriteUnroll; ++u) {
    // (min, -max) of the row in one register: one shuffle serves both
    const T2* h = reinterpret_cast<const T2*>(&raw[u]);
    T2 mn = min2_nan(min2_nan(h[0], h[1]), min2_nan(h[2], h[3]));
    T2 mx = max2_nan(max2_nan(h[0], h[1]), max2_nan(h[2], h[3]));
    T2 m;
    m.x = min2_nan(mn, __lowhigh2highlow(mn)).x;
    m.y = __hneg(max2_nan(mx, __lowhigh2highlow(mx)).x);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) m = min2_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (slot[u] < 0) continue;
    const float lo = Elem<T>::to_f32(m.x), hi = -Elem<T>::to_f32(m.y);
    float x[8];
    Elem<T>::widen(raw[u], x);
    uint32_t step_bits = Bits16<T>::kNan, lo_bits = Bits16<T>::kNan, codes = 0u;
    if (isfinite(lo) && isfinite(hi)) {
      step_bits = int4_step_bits<T>(lo, hi);
      lo_bits = *reinterpret_cast<const uint32_t*>(&m) & 0xffffu;
      const float step = Bits16<T>::to_f32(step_bits);
      if (step > 0.f) {
        const float inv = 1.f / step;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          codes |= (uint32_t)int4_code(x[e], lo, step, inv) << (4 * e);
      }
    }
    const int off = (int)(slot[u] % kBlockSize);
    unsigned char* rec = pool + ((slot[u] / kBlockSize) * a.Hkv + head[u]) * int4_record_bytes(D);
    if (is_v) {
      unsigned char* p = rec + ((off >> 1) * (D / 4) + 2 * j) * 4 + (off & 1) * 2;
      *reinterpret_cast<unsigned short*>(p) = (unsigned short)codes;
      *reinterpret_cast<unsigned short*>(p + 4) = (unsigned short)(codes >> 16);
    } else {
      *reinterpret_cast<uint32_t*>(rec + off * (D / 2) + 4 * j) = codes;
    }
    if (j == 0)
      *reinterpret_cast<uint32_t*>(rec + 8 * D + 4 * off) = step_bits | (lo_bits << 16);
  }
}

// One warp per (sequence, logical block, KV head, K or V): 16 rows of values,
// D / 8 lanes a row, 8 elements (16 bytes) a lane and pass.
template <typename T, int D>
__global__ void __launch_bounds__(256) gather_int4_kernel(GatherInt4Args a) {
  constexpr int kLanes = D / 8, kPasses = kBlockSize * kLanes / 32;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)a.B * a.Hkv * a.MBS * 2;
  for (int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; w < warps;
       w += ((int64_t)gridDim.x * blockDim.x) >> 5) {
    int64_t r = w;
    const int blk = (int)(r % a.MBS);
    r /= a.MBS;
    const bool is_v = r & 1;
    r >>= 1;
    const int h = (int)(r % a.Hkv), b = (int)(r / a.Hkv);
    int ctx = __ldg(a.context_lens + b);
    if (ctx < 0 || ctx > a.MBS * kBlockSize) {
      if (lane == 0 && blk == 0 && h == 0 && !is_v) raise_error(a.err, kErrContext);
      ctx = 0;
    }
    int valid = min(kBlockSize, max(0, ctx - blk * kBlockSize));
    const unsigned char* rec = nullptr;
    if (valid > 0) {
      const int phys = __ldg(a.block_tables + (int64_t)b * a.MBS + blk);
      if (phys < 0 || phys >= a.NB) {
        if (lane == 0) raise_error(a.err, kErrBlock);
        valid = 0;
      } else {
        rec = static_cast<const unsigned char*>(is_v ? a.v_cache : a.k_cache) +
              ((int64_t)phys * a.Hkv + h) * int4_record_bytes(D);
      }
    }
    T* dst = static_cast<T*>(is_v ? a.v_dense : a.k_dense) +
             (((int64_t)b * a.Hkv + h) * a.MBS + blk) * (kBlockSize * D);
    uint32_t codes[kPasses], pair[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int row = (i * 32 + lane) / kLanes, j = lane % kLanes;
      codes[i] = pair[i] = 0u;
      if (row < valid) {
        pair[i] = __ldg(reinterpret_cast<const uint32_t*>(rec + 8 * D) + row);
        if (is_v) {
          // words 2j and 2j + 1 of the row pair, this row's halves
          const uint2 c = __ldg(reinterpret_cast<const uint2*>(rec + (row >> 1) * D + 8 * j));
          codes[i] = __byte_perm(c.x, c.y, row & 1 ? 0x7632 : 0x5410);
        } else {
          codes[i] = __ldg(reinterpret_cast<const uint32_t*>(rec + row * (D / 2) + 4 * j));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int row = (i * 32 + lane) / kLanes, j = lane % kLanes;
      const float step = Bits16<T>::to_f32(pair[i] & 0xffffu), lo = Bits16<T>::to_f32(pair[i] >> 16);
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = Mma<T>::pack(fmaf((float)((codes[i] >> (8 * e)) & 15u), step, lo),
                            fmaf((float)((codes[i] >> (8 * e + 4)) & 15u), step, lo));
      *reinterpret_cast<uint4*>(dst + row * D + 8 * j) =
          row < valid ? make_uint4(o[0], o[1], o[2], o[3]) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

template <typename T, int D>
cudaError_t launch_write(const CacheWriteInt4Args& a, cudaStream_t stream) {
  constexpr int kRowsPerCta = (kWriteThreads / 32) * (32 / (D / 8)) * kWriteUnroll;
  const int64_t rows = (int64_t)a.T * a.Hkv;
  const int64_t grid = (rows + kRowsPerCta - 1) / kRowsPerCta;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(cache_write_int4_kernel<T, D>, dim3((unsigned)grid, 2), dim3(kWriteThreads), 0,
                    stream, a);
}

template <typename T, int D>
cudaError_t launch_gather_t(const GatherInt4Args& a, cudaStream_t stream) {
  const int64_t warps = (int64_t)a.B * a.Hkv * a.MBS * 2;
  int64_t grid = (warps + 7) / 8;
  if (grid > 152 * 64) grid = 152 * 64;
  return launch_pdl(gather_int4_kernel<T, D>, dim3((unsigned)grid), dim3(256), 0, stream, a);
}

}  // namespace

cudaError_t launch_cache_write_int4(const CacheWriteInt4Args& a, cudaStream_t stream) {
  if (a.dtype == 1)
    return a.D == 64 ? launch_write<__half, 64>(a, stream) : launch_write<__half, 128>(a, stream);
  return a.D == 64 ? launch_write<__nv_bfloat16, 64>(a, stream)
                   : launch_write<__nv_bfloat16, 128>(a, stream);
}

cudaError_t launch_gather_int4(const GatherInt4Args& a, cudaStream_t stream) {
  if (a.dtype == 1)
    return a.D == 64 ? launch_gather_t<__half, 64>(a, stream)
                     : launch_gather_t<__half, 128>(a, stream);
  return a.D == 64 ? launch_gather_t<__nv_bfloat16, 64>(a, stream)
                   : launch_gather_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace photon
