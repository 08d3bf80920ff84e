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
// each and the arithmetic must stay below the memory time.  It runs in fp32.
// A step whose fp32 value is within a few units of the border between two
// 16-bit values goes to double (fp16: about one row in a thousand, bf16: fewer).
// Elements on the border between two codes are common (with bf16 rows nearly
// every warp meets one) and are decided in line by the exact remainder; a
// double division for them made the write 87 us where it is now 24.2.
//
// Measured (8 heads, d = 128, bf16): 16 x 1024 tokens written in 24.2 us (85 MB,
// 3.5 TB/s: the arithmetic, not the memory), the same read back in 15.9 us (5.4
// TB/s, 79 % of the measured copy rate); 64 tokens in 2.0 us, a launch's time.
#include <algorithm>

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

template <typename T>
__device__ __noinline__ uint32_t int4_step_bits_exact(float lo, float hi) {
  const double s = ((double)hi - (double)lo) / 15.0;
  if constexpr (Bits16<T>::kNan == 0x7e00u)
    return __half_as_ushort(__double2half(s));
  else
    return __bfloat16_as_ushort(__double2bfloat16(s));
}

// (hi - lo) / 15 rounded once to the storage type, as bits; lo and hi are
// finite values of that type.
template <typename T>
__device__ __forceinline__ uint32_t int4_step_bits(float lo, float hi) {
  const float s = (hi - lo) * (1.f / 15.f);   // off by less than 2 units
  const uint32_t b = __float_as_uint(s);
  if constexpr (Bits16<T>::kNan == 0x7e00u) {
    // fp16 keeps 10 of fp32's 23 fraction bits; below 2^-14 it keeps fewer
    if (((b & 0x1fffu) - 0x0ffcu) > 8u && s >= 6.103515625e-5f)
      return __half_as_ushort(__float2half_rn(s));
  } else {
    // bf16 keeps 7; hi - lo may pass fp32's largest value
    if (((b & 0xffffu) - 0x7ffcu) > 8u && s >= 1e-36f && s <= 1e37f)
      return __bfloat16_as_ushort(__float2bfloat16_rn(s));
  }
  return int4_step_bits_exact<T>(lo, hi);
}

// The code of one element in full: x - lo need not be a 32-bit number, or may
// pass their range.  Rare, and a call, so that it takes no registers of the rest.
__device__ __noinline__ float int4_code_exact(float x, float lo, float step) {
  const float q = (x - lo) / step;
  if (!(q < 16.f)) return fminf((float)rint(((double)x - (double)lo) / (double)step), 15.f);
  // On which side of 0 is x - lo - (f + 1/2) step?  The product has 5 + 11 bits
  // and where it matters lies within 2^-16 of d = x - lo, so both it and the
  // difference are exact, and so is what the subtraction x - lo lost.
  const float d = x - lo, f = fminf(floorf(q), 15.f), r = d - (f + 0.5f) * step;
  const float back = d - x, lost = (x - (d - back)) - (lo + back);
  const float side = r + lost;
  const float n = side > 0.f ? f + 1.f : side < 0.f ? f : 2.f * rintf(0.5f * (f + 0.5f));   // tie: even
  return fminf(fmaxf(n, 0.f), 15.f);
}

// Codes of 8 elements, 4 bits each, element 0 lowest.  Rounding and packing
// stay on the fp32 pipe: adding 1.5 x 2^23 rounds to an integer, four codes are
// summed as n0 + 16 n1 + 256 n2 + 4096 n3, exact below 2^24 (conversion
// instructions run at a quarter of the rate).
//
// The quotient q = (x - lo) / step is corrected by its remainder, which one
// fused operation gives exactly, so that on a border between two codes it is
// the half itself and rounding to an integer takes the even one.  This needs x
// and lo without bits below 2^-22 of the range: then d = x - lo is exact, and a
// quotient that is not on a border is 2^-22 x 15 away from it, four of its
// units.  Smaller x (a last place is at least 2^-11 of x, bf16 2^-8: `least` is
// their bound) all have quotients near -lo / step, so they matter in rows whose
// -lo / step is near a border (`near`), and there only next to it; they are
// looked at again, and so is every element of a row with a tiny lo or a step
// of few bits (`odd`: an fp16 subnormal; bf16 has fp32's exponents and keeps
// all its bits, so there only what would leave fp32's own range counts.  16 x
// 1024 bf16 rows with steps of 3e-5: 24 us, as others; through `odd` 158).
template <typename T>
__device__ __forceinline__ uint32_t int4_codes8(const uint4& raw, float lo, float step, float inv,
                                                float least, bool near, bool odd) {
  constexpr float kRound = 12582912.f;
  float x[8], n[8];
  Elem<T>::widen(raw, x);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float d = x[e] - lo, q = d * inv;
    n[e] = (fmaf(fmaf(-q, step, d), inv, q) + kRound) - kRound;
  }
  if (near) {
    uint32_t again = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (odd || (fabsf(x[e]) < least && fabsf((x[e] - lo) * inv - n[e]) > 0.4999f))
        again |= 1u << e;
    while (again) {
      const int e = __ffs(again) - 1;
      again &= again - 1;
      // (indexed by a variable the array would go into memory)
      float xe = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) xe = i == e ? x[i] : xe;
      const float ne = int4_code_exact(xe, lo, step);
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = i == e ? ne : n[i];
    }
  }
  const float c0 = fmaf(4096.f, n[3], fmaf(256.f, n[2], fmaf(16.f, n[1], n[0])));
  const float c1 = fmaf(4096.f, n[7], fmaf(256.f, n[6], fmaf(16.f, n[5], n[4])));
  return __byte_perm(__float_as_uint(c0 + 8388608.f), __float_as_uint(c1 + 8388608.f), 0x5410);
}

constexpr int kWriteThreads = 256;
// CTAs per SM; 4 leave too few registers (16 x 1024 tokens 25.0 against 24.2 us).
constexpr int kWriteCtas = 3;

// D / 16 lanes a row: lane j has elements 8j .. 8j + 7 of both halves (16 a
// lane rather than 8 halve what a row costs beside its elements).
template <typename T, int D>
__global__ void __launch_bounds__(kWriteThreads, kWriteCtas)
    cache_write_int4_kernel(CacheWriteInt4Args a) {
  using T2 = typename Pair16<T>::type;
  constexpr int kLanes = D / 16, kGroup = 32 / kLanes;   // rows a warp takes at once
  pdl_launch_dependents();
  pdl_wait_primary();
  const int lane = threadIdx.x & 31, j = lane % kLanes;
  const bool is_v = blockIdx.y != 0;
  const int64_t nslots = (int64_t)a.NB * kBlockSize;
  const T* src = static_cast<const T*>(is_v ? a.v : a.k) + 8 * j;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  unsigned char* pool = static_cast<unsigned char*>(is_v ? a.v_cache : a.k_cache);

  // A warp's groups of rows lie gridDim.x * 8 groups apart; the next group's
  // rows and slots are on their way while one is worked on.
  const int64_t ahead = (int64_t)gridDim.x * (kWriteThreads / 32) * kGroup;
  const int ahead_t = (int)(ahead / a.Hkv), ahead_h = (int)(ahead % a.Hkv);
  const int64_t row =
      ((int64_t)blockIdx.x * (kWriteThreads / 32) + (threadIdx.x >> 5)) * kGroup + lane / kLanes;
  int64_t t = row / a.Hkv;
  int h = (int)(row - t * a.Hkv);
  uint4 next0 = make_uint4(0u, 0u, 0u, 0u), next1 = next0;
  int64_t next_slot = -1;
  auto load = [&]() {
    if (t < a.T) {
      const T* p = src + t * stride + (int64_t)h * D;
      next_slot = __ldg(a.slot_mapping + t);
      next0 = ld_stream16(p);
      next1 = ld_stream16(p + D / 2);
    } else {
      next_slot = -1;
    }
  };
  load();
  // (a warp leaves together: its lanes' rows end within one group)
  while (__any_sync(0xffffffffu, t < a.T)) {
    const uint4 raw0 = next0, raw1 = next1;
    int64_t slot = next_slot;
    const int head = h;
    if (slot >= nslots) {
      if (j == 0 && head == 0 && !is_v) raise_error(a.err, kErrSlot);
      slot = -1;
    }
    t += ahead_t;
    h += ahead_h;
    if (h >= a.Hkv) {
      h -= a.Hkv;
      ++t;
    }
    load();
    // (min, -max) of the row in one register: one shuffle serves both
    const T2* p0 = reinterpret_cast<const T2*>(&raw0);
    const T2* p1 = reinterpret_cast<const T2*>(&raw1);
    T2 mn = min2_nan(p0[0], p1[0]), mx = max2_nan(p0[0], p1[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      mn = min2_nan(mn, min2_nan(p0[i], p1[i]));
      mx = max2_nan(mx, max2_nan(p0[i], p1[i]));
    }
    T2 m;
    m.x = min2_nan(mn, __lowhigh2highlow(mn)).x;
    m.y = __hneg(max2_nan(mx, __lowhigh2highlow(mx)).x);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) m = min2_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (slot < 0) continue;   // padding
    const float lo = Elem<T>::to_f32(m.x), hi = -Elem<T>::to_f32(m.y);
    uint32_t step_bits = Bits16<T>::kNan, lo_bits = Bits16<T>::kNan, codes0 = 0u, codes1 = 0u;
    if (isfinite(lo) && isfinite(hi)) {
      step_bits = int4_step_bits<T>(lo, hi);
      lo_bits = *reinterpret_cast<const uint32_t*>(&m) & 0xffffu;
      const float step = Bits16<T>::to_f32(step_bits);
      if (step > 0.f) {
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(step));   // 1 unit
        const float range = hi - lo, at0 = fminf(-lo * inv, 1e6f);
        const float least =
            range * (Bits16<T>::kNan == 0x7e00u ? 4.8828125e-4f : 6.103515625e-5f);
        const bool odd = (lo != 0.f && fabsf(lo) < least) ||
                         !(step >= (Bits16<T>::kNan == 0x7e00u ? 6.2e-5f : 1e-30f)) ||
                         !(range < 1e37f);
        const bool near = odd || fabsf(at0 - rintf(at0)) > 0.49f;
        codes0 = int4_codes8<T>(raw0, lo, step, inv, least, near, odd);
        codes1 = int4_codes8<T>(raw1, lo, step, inv, least, near, odd);
      }
    }
    const int off = (int)slot & (kBlockSize - 1);
    unsigned char* rec = pool + ((slot >> 4) * a.Hkv + head) * (int64_t)int4_record_bytes(D);
    if (is_v) {
      unsigned char* p = rec + (off >> 1) * D + 8 * j + (off & 1) * 2;
      *reinterpret_cast<unsigned short*>(p) = (unsigned short)codes0;
      *reinterpret_cast<unsigned short*>(p + 4) = (unsigned short)(codes0 >> 16);
      *reinterpret_cast<unsigned short*>(p + D / 2) = (unsigned short)codes1;
      *reinterpret_cast<unsigned short*>(p + D / 2 + 4) = (unsigned short)(codes1 >> 16);
    } else {
      *reinterpret_cast<uint32_t*>(rec + off * (D / 2) + 4 * j) = codes0;
      *reinterpret_cast<uint32_t*>(rec + off * (D / 2) + D / 4 + 4 * j) = codes1;
    }
    if (j == 0)
      *reinterpret_cast<uint32_t*>(rec + 8 * D + 4 * off) = step_bits | (lo_bits << 16);
  }
}

// p + lo, inexact in 32 bits, rounded to odd: rounded once more to 16 bits it
// is the exact sum's rounding.
__device__ __forceinline__ float sum_to_odd(float p, float lo) {
  const float s = p + lo, back = s - p, off = (p - (s - back)) + (lo - back);
  const uint32_t b = __float_as_uint(s);
  if (off == 0.f || (b & 1u) || !isfinite(s)) return s;
  return __uint_as_float((off > 0.f) == (s > 0.f) ? b + 1u : b - 1u);
}

// One warp per (sequence, logical block, KV head): 16 rows of K values, then of
// V, D / 8 lanes a row, 8 elements (16 bytes) a lane and pass.
constexpr int kGatherWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kGatherWarps) gather_int4_kernel(GatherInt4Args a) {
  constexpr int kLanes = D / 8, kPasses = kBlockSize * kLanes / 32;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int lane = threadIdx.x & 31;
  const int blk = (int)blockIdx.x * kGatherWarps + (threadIdx.x >> 5);
  const int h = blockIdx.y, b = blockIdx.z;
  if (blk >= a.MBS) return;
  int ctx = __ldg(a.context_lens + b);
  if (ctx < 0 || ctx > a.MBS * kBlockSize) {
    if (lane == 0 && blk == 0 && h == 0) raise_error(a.err, kErrContext);
    ctx = 0;
  }
  int valid = min(kBlockSize, max(0, ctx - blk * kBlockSize));
  int64_t rec = 0;
  if (valid > 0) {
    const int phys = __ldg(a.block_tables + (int64_t)b * a.MBS + blk);
    if (phys < 0 || phys >= a.NB) {
      if (lane == 0) raise_error(a.err, kErrBlock);
      valid = 0;
    } else {
      rec = ((int64_t)phys * a.Hkv + h) * int4_record_bytes(D);
    }
  }
  const unsigned char* kr = static_cast<const unsigned char*>(a.k_cache) + rec;
  const unsigned char* vr = static_cast<const unsigned char*>(a.v_cache) + rec;
  const int j = lane % kLanes, r0 = lane / kLanes;
  uint32_t kc[kPasses], kp[kPasses], vc[kPasses], vp[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int row = i * (32 / kLanes) + r0;
    kc[i] = kp[i] = vc[i] = vp[i] = 0u;
    if (row < valid) {
      kp[i] = __ldg(reinterpret_cast<const uint32_t*>(kr + 8 * D) + row);
      vp[i] = __ldg(reinterpret_cast<const uint32_t*>(vr + 8 * D) + row);
      kc[i] = __ldg(reinterpret_cast<const uint32_t*>(kr + row * (D / 2) + 4 * j));
      // words 2j and 2j + 1 of the row pair, this row's halves
      const uint2 c = __ldg(reinterpret_cast<const uint2*>(vr + (row >> 1) * D + 8 * j));
      vc[i] = __byte_perm(c.x, c.y, row & 1 ? 0x7632 : 0x5410);
    }
  }
  const int64_t to = (((int64_t)b * a.Hkv + h) * a.MBS + blk) * (kBlockSize * D) + r0 * D + 8 * j;
  uint32_t odd = 0u;   // bit 2 i + which: a row that is rounded below
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    T* dst = static_cast<T*>(which ? a.v_dense : a.k_dense) + to;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const uint32_t c = which ? vc[i] : kc[i], pair = which ? vp[i] : kp[i];
      const float step = Bits16<T>::to_f32(pair & 0xffffu), lo = Bits16<T>::to_f32(pair >> 16);
      // an integer below 2^23 in the fraction of 2^23, less 2^23: the code as
      // fp32 without a conversion
      // lo + n step has a few more bits than 16 for a lo of some size, and is
      // exact in 32; below step / 256 it need not be
      if (lo != 0.f && fabsf(lo) * 256.f < step) odd |= 1u << (2 * i + which);
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float n0 = __uint_as_float(0x4b000000u | ((c >> (8 * e)) & 15u)) - 8388608.f;
        const float n1 = __uint_as_float(0x4b000000u | ((c >> (8 * e + 4)) & 15u)) - 8388608.f;
        o[e] = Mma<T>::pack(fmaf(n0, step, lo), fmaf(n1, step, lo));
      }
      // rows behind the context: code, step and lo are 0, and so are the values
      __stcs(reinterpret_cast<uint4*>(dst + i * (32 / kLanes) * D),
             make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
  // once more for the rare rows, from memory (kept out of the loop above, where
  // it costs registers: 16.3 against 15.9 us)
  while (odd) {
    const int bit = __ffs(odd) - 1, i = bit >> 1, which = bit & 1;
    odd &= odd - 1;
    const int row = i * (32 / kLanes) + r0;
    const unsigned char* rp = which ? vr : kr;
    const uint32_t pair = __ldg(reinterpret_cast<const uint32_t*>(rp + 8 * D) + row);
    const float step = Bits16<T>::to_f32(pair & 0xffffu), lo = Bits16<T>::to_f32(pair >> 16);
    T* dst = static_cast<T*>(which ? a.v_dense : a.k_dense) + to + i * (32 / kLanes) * D;
#pragma unroll 1
    for (int e = 0; e < 4; ++e) {
      // elements 2e and 2e + 1: a byte of the K row, of word e / 2 of the V pair
      const unsigned char* p = which ? rp + (row >> 1) * D + 8 * j + 4 * (e >> 1) + 2 * (row & 1) + (e & 1)
                                     : rp + row * (D / 2) + 4 * j + e;
      const uint32_t c = __ldg(p);
      reinterpret_cast<uint32_t*>(dst)[e] = Mma<T>::pack(
          sum_to_odd((float)(c & 15u) * step, lo), sum_to_odd((float)(c >> 4) * step, lo));
    }
  }
}

template <typename T, int D>
cudaError_t launch_write(const CacheWriteInt4Args& a, cudaStream_t stream) {
  constexpr int kRowsPerCta = (kWriteThreads / 32) * (32 / (D / 16));
  const int64_t rows = (int64_t)a.T * a.Hkv;
  // two halves (K, V) of as many CTAs as stay resident
  const int64_t grid = std::min<int64_t>((rows + kRowsPerCta - 1) / kRowsPerCta,
                                         (int64_t)a.num_sms * kWriteCtas / 2);
  return launch_pdl(cache_write_int4_kernel<T, D>, dim3((unsigned)grid, 2), dim3(kWriteThreads), 0,
                    stream, a);
}

template <typename T, int D>
cudaError_t launch_gather_t(const GatherInt4Args& a, cudaStream_t stream) {
  return launch_pdl(gather_int4_kernel<T, D>,
                    dim3((a.MBS + kGatherWarps - 1) / kGatherWarps, a.Hkv, a.B),
                    dim3(32 * kGatherWarps), 0, stream, a);
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
