// paged_decode_int4.cu -- decode attention over the 4-bit paged KV cache.
//
// PhotonInfer README, "Key features / GPU-optimized kernels" (batched paged
// attention, numerically stable softmax) and "Roadmap" (lower-precision KV).
//
// With K_j = lo_j + n_j step_j and V_j likewise,
//   score_j = scale (step_j (q . n_j) + lo_j sum(q)),
//   out     = sum_j (p_j step_j) n_j + sum_j p_j lo_j       (p_j: softmax),
// so both products run on the codes n alone and the pairs (step, lo) come in
// afterwards, once per row.  A code widens to fp16 with one AND: the bits 0x000n
// are the fp16 subnormal n 2^-24, 0x00n0 is 16 n 2^-24, both exact and both
// what the tensor cores take; 2^24 and 1/16 go into the other operand and the
// result.  Eight codes cost four ANDs and a shift, against eight conversions.
//
// The record's layout (include/photon_paged.h) is made for mma.sync m16n8k16:
//   S^T (16 keys x 8) = K Q^T: lane (g, t) = (lane / 4, lane % 4) reads D / 8
//     bytes of key rows g and g + 8; word w's nibbles 0, 4 | 1, 5 | 2, 6 | 3, 7
//     are the k index pairs of two products, q's dims follow that order;
//   O^T (D x 8) += V^T P^T: a V word holds four dims of two neighbouring keys,
//     nibble i of both halves is dim 4c + i of keys 2p, 2p + 1; lane (g, t)
//     reads D / 8 bytes of row pairs t and t + 4.
// So every fragment comes from one 16-byte (D = 64: 8-byte) shared-memory read
// per row or row pair, contiguous over the warp: no bank conflicts, no
// swizzle, no ldmatrix.  P^T is the score fragment packed and transposed with
// movmatrix; p_j step_j enters as its fp16 rounding plus the residual: for
// G <= 4 the residual rides in the unused columns 4 .. 7 of the same product.
//
// Work: the batch's (sequence, KV head, block) triples in that order are one
// line of units of 16 keys, cut into equal runs, one per warp; a warp has its
// own ring of cp.async stages and no barrier with any other warp.  A run may
// span several (sequence, KV head) pairs; a pair that lies in one run is
// written out directly, the others leave (m, l, o) partials, merged by a
// second kernel.  Every warp gets the same number of units whatever the mix of
// lengths, without a queue or atomics, so results do not depend on timing.
#include <math.h>

#include <algorithm>

#include "int4_common.cuh"

namespace photon {
namespace {

constexpr int kI4Warps = 4;               // warps per CTA
constexpr int kI4Threads = 32 * kI4Warps;
constexpr int kI4MinUnits = 4;            // shortest run of a warp, in units
// Running maximum before the first key: below the scores, and finite, so that
// no exponent is inf - inf.
constexpr float kI4NoMax = -3e38f;

template <int D>
struct I4Cfg {
  static constexpr int kRec = int4_record_bytes(D);
  static constexpr int kUnit = 2 * kRec;                 // K record, V record
  static constexpr int kStages = D == 128 ? 6 : 8;
  static constexpr int kCtas = D == 128 ? 4 : 5;          // per SM
  static constexpr int kSmem = kI4Warps * kStages * kUnit;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// A raise of the exponent is exact: 2^(e - 127) from a biased exponent.
__device__ __forceinline__ float pow2_biased(int e) {
  return __uint_as_float((uint32_t)min(max(e, 1), 254) << 23);
}

// A warp's place on the line of units: unit `blk` of KV head kvh of sequence b,
// whose context has n blocks.
struct I4Cursor {
  int b, kvh, blk, n, ctx;
};

template <typename T, int D, bool kFull>
__global__ void __launch_bounds__(kI4Threads, I4Cfg<D>::kCtas)
    paged_decode_int4_kernel(const DecodeInt4Args a) {
  using C = I4Cfg<D>;
  constexpr int NW = D / 32;        // code words of a lane per row (or row pair)
  extern __shared__ __align__(16) unsigned char i4_smem[];
  __shared__ long long pre[kI4Threads];      // units before a thread's sequences
  __shared__ long long warp_sum[kI4Warps];

  pdl_launch_dependents();
  pdl_wait_primary();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int G = a.Hq / a.Hkv;
  const int span = a.MBS * kBlockSize;
  auto ctx_of = [&](int b) -> int {
    const int c = __ldg(a.context_lens + b);
    return c > 0 && c <= span ? c : 0;   // the merge kernel flags rejected lengths
  };
  auto blocks_of = [](int ctx) -> int { return (ctx + kBlockSize - 1) / kBlockSize; };

  // ---- the line of units: thread i sums sequences [i c, (i + 1) c)
  const int per_thread = (a.B + kI4Threads - 1) / kI4Threads;
  long long mine = 0;
  for (int i = 0; i < per_thread; ++i) {
    const int b = tid * per_thread + i;
    if (b < a.B) mine += blocks_of(ctx_of(b));
  }
  mine *= a.Hkv;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kI4Warps; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  pre[tid] = before + incl - mine;
  __syncthreads();
  const long long W = (long long)gridDim.x * kI4Warps;
  long long per = (total + W - 1) / W;
  if (per < kI4MinUnits) per = kI4MinUnits;
  const long long w_id = (long long)blockIdx.x * kI4Warps + warp;
  const long long u0 = w_id * per;
  if (u0 >= total) return;
  int count = (int)(u0 + per <= total ? per : total - u0);

  // ---- the run's first unit: the last thread whose sequences begin at or
  // before it, then a walk over that thread's sequences
  I4Cursor cur;
  {
    int owner = 0;
#pragma unroll
    for (int i = 0; i < kI4Warps; ++i) {
      const unsigned at = __ballot_sync(0xffffffffu, pre[i * 32 + lane] <= u0);
      if (at) owner = i * 32 + 31 - __clz(at);
    }
    long long left = u0 - pre[owner];
    cur.b = owner * per_thread;
    while (true) {   // ends inside the owner's sequences: u0 < total
      cur.ctx = ctx_of(cur.b);
      cur.n = blocks_of(cur.ctx);
      const long long units = (long long)cur.n * a.Hkv;
      if (left < units || cur.b + 1 >= a.B) break;
      left -= units;
      ++cur.b;
    }
    cur.kvh = (int)(left / cur.n);
    cur.blk = (int)(left - (long long)cur.kvh * cur.n);
  }
  // to the next unit; past the last sequence the cursor stays (no unit is left)
  auto advance = [&](I4Cursor& c) {
    if (++c.blk < c.n) return;
    c.blk = 0;
    if (++c.kvh < a.Hkv) return;
    c.kvh = 0;
    do {
      if (++c.b >= a.B) {
        c.n = 0;
        return;
      }
      c.ctx = ctx_of(c.b);
      c.n = blocks_of(c.ctx);
    } while (c.n == 0);
  };

  // ---- the ring
  unsigned char* ring = i4_smem + warp * (C::kStages * C::kUnit);
  const uint32_t ring_addr = smem_addr(ring);
  const unsigned char* kpool = static_cast<const unsigned char*>(a.k_cache);
  const unsigned char* vpool = static_cast<const unsigned char*>(a.v_cache);
  I4Cursor fetch = cur;
  int to_fetch = count, table = -1, table_b = -1, table_at = -1;
  uint32_t absent = 0;   // bit s: the block in stage s is not in the pool
  auto issue = [&](int s) {
    if (to_fetch > 0) {
      // lane i holds the table's entry for block table_at + i
      const int at = fetch.blk & ~31;
      if (table_b != fetch.b || table_at != at) {
        table_b = fetch.b;
        table_at = at;
        table = at + lane < fetch.n ? __ldg(a.block_tables + (size_t)fetch.b * a.MBS + at + lane)
                                    : -1;
      }
      const int phys = __shfl_sync(0xffffffffu, table, fetch.blk & 31);
      if (phys >= 0 && phys < a.NB) {
        const size_t off = ((size_t)phys * a.Hkv + fetch.kvh) * C::kRec;
        const uint32_t dst = ring_addr + s * C::kUnit;
#pragma unroll
        for (int i = 0; i < 8 * D; i += 512) {
          const int o = i + 16 * lane;
          cp_async16(dst + o, kpool + off + o);
          cp_async16(dst + C::kRec + o, vpool + off + o);
        }
        if (lane < 8) {   // the 64 bytes of pairs of each
          const int o = 8 * D + 16 * (lane & 3);
          cp_async16(dst + (lane < 4 ? 0 : C::kRec) + o, (lane < 4 ? kpool : vpool) + off + o);
        }
        absent &= ~(1u << s);
      } else {
        if (lane == 0) raise_error(a.err, kErrBlock);
        absent |= 1u << s;
      }
      --to_fetch;
      advance(fetch);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) issue(s);

  // ---- a pair's state.  Columns (slots) 2t and 2t + 1 of the score fragment
  // are this lane's; with G <= 4 column 4 + s repeats slot s.
  uint32_t bq[NW][2][2];   // Q^T fragments: column g, products 2j and 2j + 1 of word j
  float c1[2], c2[2];      // score = step (acc c1) + lo c2
  float m[2], l[2], z[2];  // running max, sum of weights, sum of weights x lo of V
  float o[NW][2][4];       // O^T: dims (D / 8) g + 4j + 2h (rows g) and + 1 (rows g + 8)
  float vs = 0.f;          // power of two that the V steps are brought near 1 with
  auto begin_pair = [&]() {
    const int s = kFull ? g : g & 3;
    float x[NW * 8];
#pragma unroll
    for (int i = 0; i < NW * 8; ++i) x[i] = 0.f;
    if (s < G) {
      const T* row = static_cast<const T*>(a.q) +
                     ((size_t)cur.b * a.Hq + (size_t)cur.kvh * G + s) * D + (D / 4) * t;
#pragma unroll
      for (int i = 0; i < NW; ++i) Elem<T>::widen(__ldg(reinterpret_cast<const uint4*>(row) + i), x + 8 * i);
    }
    float big = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < NW * 8; ++i) {
      big = fmaxf(big, fabsf(x[i]));
      sum += x[i];
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
      sum += __shfl_xor_sync(0xffffffffu, sum, off);
    }
    // the row is scaled by a power of two to [2^14, 2^15): fp16 then holds
    // every fp16 or bf16 q, and its 16th, to 2^-25 of that
    const int ex = (int)((__float_as_uint(big) >> 23) & 255u);
    const float sc = pow2_biased(268 - ex);   // 2^(14 - (ex - 127))
    const float s16 = sc * 0.0625f;
#pragma unroll
    for (int j = 0; j < NW; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float* w = x + 8 * j + 2 * h;
        bq[j][h][0] = Mma<__half>::pack(w[0] * sc, w[4] * sc);
        bq[j][h][1] = Mma<__half>::pack(w[1] * s16, w[5] * s16);
      }
    // 2^24 of the codes; 1 / sc is exact
    const float k1 = a.qscale * (16777216.f * (1.f / sc)), k2 = a.qscale * sum;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int col = 2 * t + i;
      c1[i] = __shfl_sync(0xffffffffu, k1, (kFull ? col : col & 3) * 4);
      c2[i] = __shfl_sync(0xffffffffu, k2, (kFull ? col : col & 3) * 4);
      m[i] = kI4NoMax;
      l[i] = z[i] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < NW; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][h][i] = 0.f;
    vs = 1.2676506e30f;   // 2^100: the first step sets it
  };

  auto words = [&](const unsigned char* p, uint32_t (&w)[NW]) {
    if constexpr (NW == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    }
  };

  auto attend = [&](const unsigned char* kr, int valid) {
    const unsigned char* vr = kr + C::kRec;
    // K: rows g and g + 8
    uint32_t k0[NW], k8[NW];
    words(kr + g * (D / 2) + t * (D / 8), k0);
    words(kr + (g + 8) * (D / 2) + t * (D / 8), k8);
    const uint32_t kp0 = *reinterpret_cast<const uint32_t*>(kr + 8 * D + 4 * g);
    const uint32_t kp8 = *reinterpret_cast<const uint32_t*>(kr + 8 * D + 4 * g + 32);
    const uint32_t vp0 = *reinterpret_cast<const uint32_t*>(vr + 8 * D + 4 * g);
    const uint32_t vp8 = *reinterpret_cast<const uint32_t*>(vr + 8 * D + 4 * g + 32);
    float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      const uint32_t x = k0[j], y = k8[j], x8 = x >> 8, y8 = y >> 8;
      const uint32_t f0[4] = {x & 0x000f000fu, y & 0x000f000fu, x & 0x00f000f0u, y & 0x00f000f0u};
      const uint32_t f1[4] = {x8 & 0x000f000fu, y8 & 0x000f000fu, x8 & 0x00f000f0u,
                              y8 & 0x00f000f0u};
      Mma<__half>::run(sa, f0, bq[j][0][0], bq[j][0][1]);
      Mma<__half>::run(sb, f1, bq[j][1][0], bq[j][1][1]);
    }
    const bool ok0 = g < valid, ok8 = g + 8 < valid;
    const float ks0 = Bits16<T>::to_f32(kp0 & 0xffffu), kl0 = Bits16<T>::to_f32(kp0 >> 16);
    const float ks8 = Bits16<T>::to_f32(kp8 & 0xffffu), kl8 = Bits16<T>::to_f32(kp8 >> 16);
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float raw = fmaf(i < 2 ? ks0 : ks8, (sa[i] + sb[i]) * c1[i & 1],
                             (i < 2 ? kl0 : kl8) * c2[i & 1]);
      x[i] = (i < 2 ? ok0 : ok8) ? raw : -INFINITY;
    }
    const float vs0 = ok0 ? Bits16<T>::to_f32(vp0 & 0xffffu) : 0.f;
    const float vs8 = ok8 ? Bits16<T>::to_f32(vp8 & 0xffffu) : 0.f;
    const float vl0 = ok0 ? Bits16<T>::to_f32(vp0 >> 16) : 0.f;
    const float vl8 = ok8 ? Bits16<T>::to_f32(vp8 >> 16) : 0.f;
    // The maximum only moves when a score passes it by more than 2^8 (then
    // weights stay below 2^8), the V steps' power of two when a step passes
    // 8; what is summed so far is rescaled then.  Both cancel in O / l.
    const bool over = fmaxf(x[0], x[2]) > m[0] + 8.f || fmaxf(x[1], x[3]) > m[1] + 8.f ||
                      fmaxf(vs0, vs8) * vs > 8.f;
    if (__any_sync(0xffffffffu, over)) {
      float n0 = fmaxf(m[0], fmaxf(x[0], x[2])), n1 = fmaxf(m[1], fmaxf(x[1], x[3]));
      float sm = fmaxf(vs0, vs8);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, off));
        n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, off));
        sm = fmaxf(sm, __shfl_xor_sync(0xffffffffu, sm, off));
      }
      const float r0 = softmax_exp2(m[0] - n0), r1 = softmax_exp2(m[1] - n1);
      float up = 1.f;
      if (sm * vs > 1.f) {
        // 2^-(exponent of sm + 1)
        const float next = pow2_biased(253 - (int)((__float_as_uint(sm) >> 23) & 255u));
        up = next * (1.f / vs);
        vs = next;
      }
      m[0] = n0;
      m[1] = n1;
      l[0] *= r0, z[0] *= r0;
      l[1] *= r1, z[1] *= r1;
#pragma unroll
      for (int j = 0; j < NW; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][h][i] *= (i & 1 ? r1 : r0) * up;
    }
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = softmax_exp2(x[i] - m[i & 1]);   // 0 for masked rows
      l[i & 1] += p;
      z[i & 1] = fmaf(p, i < 2 ? vl0 : vl8, z[i & 1]);
      w[i] = p * ((i < 2 ? vs0 : vs8) * vs);
    }
    const uint32_t h01 = Mma<__half>::pack(w[0], w[1]), h23 = Mma<__half>::pack(w[2], w[3]);
    const float2 r01 = Mma<__half>::unpack(h01), r23 = Mma<__half>::unpack(h23);
    const uint32_t e01 = Mma<__half>::pack(w[0] - r01.x, w[1] - r01.y);
    const uint32_t e23 = Mma<__half>::pack(w[2] - r23.x, w[3] - r23.y);
    // P^T fragments: the rounding, and its residual in columns 4 .. 7 (their
    // scores repeat columns 0 .. 3) or, with eight slots, in a second product
    const bool upper = !kFull && t >= 2;
    const uint32_t b0 = movmatrix_trans(upper ? e01 : h01), b1 = movmatrix_trans(upper ? e23 : h23);
    uint32_t d0 = 0u, d1 = 0u;
    if constexpr (kFull) {
      d0 = movmatrix_trans(e01);
      d1 = movmatrix_trans(e23);
    }
    // V: row pairs t and t + 4
    uint32_t v0[NW], v4[NW];
    words(vr + t * D + g * (D / 8), v0);
    words(vr + (t + 4) * D + g * (D / 8), v4);
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      const uint32_t p = v0[j], q = v4[j], p8 = p >> 8, q8 = q >> 8;
      const uint32_t f0[4] = {p & 0x000f000fu, p & 0x00f000f0u, q & 0x000f000fu, q & 0x00f000f0u};
      const uint32_t f1[4] = {p8 & 0x000f000fu, p8 & 0x00f000f0u, q8 & 0x000f000fu,
                              q8 & 0x00f000f0u};
      Mma<__half>::run(o[j][0], f0, b0, b1);
      Mma<__half>::run(o[j][1], f1, b0, b1);
      if constexpr (kFull) {
        Mma<__half>::run(o[j][0], f0, d0, d1);
        Mma<__half>::run(o[j][1], f1, d0, d1);
      }
    }
  };

  // the pair's sums over the warp; then out, or a partial
  auto end_pair = [&](long long pair_u0) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
        z[i] += __shfl_xor_sync(0xffffffffu, z[i], off);
      }
    const float unscale = 1.f / vs;   // a power of two
#pragma unroll
    for (int j = 0; j < NW; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (!kFull) o[j][h][i] += __shfl_xor_sync(0xffffffffu, o[j][h][i], 2);
          o[j][h][i] = fmaf(o[j][h][i] * (i < 2 ? 16777216.f : 1048576.f), unscale, z[i & 1]);
        }
    const int pair = cur.b * a.Hkv + cur.kvh;
    const long long w_first = pair_u0 / per, w_last = (pair_u0 + cur.n - 1) / per;
    if (w_id == w_first && lane == 0)
      a.ws_pair[pair] = make_int2((int)w_first + pair, (int)(w_last - w_first) + 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = 2 * t + i;
      if (s >= G || (!kFull && t >= 2)) continue;
      if (w_first == w_last) {
        const float inv = l[i] > 0.f || l[i] != l[i] ? 1.f / l[i] : 0.f;
        T* dst = static_cast<T*>(a.out) + ((size_t)cur.b * a.Hq + (size_t)cur.kvh * G + s) * D +
                 (D / 8) * g;
#pragma unroll
        for (int j = 0; j < NW; j += 2)
          *reinterpret_cast<uint4*>(dst + 4 * j) =
              make_uint4(Mma<T>::pack(o[j][0][i] * inv, o[j][0][2 + i] * inv),
                         Mma<T>::pack(o[j][1][i] * inv, o[j][1][2 + i] * inv),
                         Mma<T>::pack(o[j + 1][0][i] * inv, o[j + 1][0][2 + i] * inv),
                         Mma<T>::pack(o[j + 1][1][i] * inv, o[j + 1][1][2 + i] * inv));
      } else {
        const size_t row = (size_t)(w_id + pair) * G + s;
        if (g == 0) a.ws_ml[row] = make_float2(m[i], l[i]);
        float4* dst = reinterpret_cast<float4*>(a.ws_o + row * D + (D / 8) * g);
#pragma unroll
        for (int j = 0; j < NW; ++j)
          dst[j] = make_float4(o[j][0][i], o[j][0][2 + i], o[j][1][i], o[j][1][2 + i]);
      }
    }
  };

  long long u = u0, pair_u0 = u0 - cur.blk;
  int stage = 0;
  begin_pair();
  for (; count > 0; --count, ++u) {
    cp_async_wait<C::kStages - 2>();
    __syncwarp();
    const int left = cur.ctx - cur.blk * kBlockSize;
    const int valid = (absent >> stage) & 1u ? 0 : min(left, kBlockSize);
    attend(ring + stage * C::kUnit, valid);
    __syncwarp();   // every lane has read the stage before it is filled again
    const bool last = cur.blk + 1 == cur.n;
    if (last || count == 1) {
      end_pair(pair_u0);
      if (count > 1) {
        pair_u0 += cur.n;
        advance(cur);
        begin_pair();
      }
    } else {
      ++cur.blk;
    }
    issue(stage == 0 ? C::kStages - 1 : stage - 1);
    stage = stage + 1 == C::kStages ? 0 : stage + 1;
  }
  cp_async_wait<0>();
}

// One CTA per (sequence, q head): out = sum_p w_p o_p / sum_p w_p l_p with
// w_p = 2^(m_p - max m) over the pair's partials, and the zero rows of empty
// sequences.  A warp takes every fourth group of 8 partials, all loaded at
// once, so up to 32 partials cost one round trip.
constexpr int kI4MergeRows = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kI4Threads) paged_decode_int4_merge_kernel(const DecodeInt4Args a) {
  constexpr int EPL = D / 32;
  __shared__ float sm[kI4Warps], sl[kI4Warps], so[kI4Warps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq;
  const int G = a.Hq / a.Hkv;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int ctx = __ldg(a.context_lens + b);
  T* out = static_cast<T*>(a.out) + (size_t)blockIdx.x * D;
  if (ctx <= 0 || ctx > a.MBS * kBlockSize) {
    if (ctx != 0 && threadIdx.x == 0 && hq == 0) raise_error(a.err, kErrContext);
    if (threadIdx.x < D / 8) reinterpret_cast<uint4*>(out)[threadIdx.x] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int2 pr = a.ws_pair[b * a.Hkv + hq / G];
  if (pr.y < 2) return;   // the attention kernel wrote out
  const size_t row0 = (size_t)pr.x * G + hq % G;
  float M = kI4NoMax, L = 0.f, O[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) O[e] = 0.f;
  for (int p0 = warp * kI4MergeRows; p0 < pr.y; p0 += kI4Warps * kI4MergeRows) {
    float v[kI4MergeRows][EPL];
    float2 ml[kI4MergeRows];
#pragma unroll
    for (int u = 0; u < kI4MergeRows; ++u) {
      const bool in = p0 + u < pr.y;
      const size_t row = row0 + (size_t)(in ? p0 + u : p0) * G;
      ml[u] = a.ws_ml[row];
      if (!in) ml[u].y = 0.f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) v[u][e] = a.ws_o[row * D + lane * EPL + e];
    }
    float mx = M;
#pragma unroll
    for (int u = 0; u < kI4MergeRows; ++u)
      if (ml[u].y != 0.f) mx = fmaxf(mx, ml[u].x);
    const float r = exp2f(M - mx);
    M = mx;
    L *= r;
#pragma unroll
    for (int e = 0; e < EPL; ++e) O[e] *= r;
#pragma unroll
    for (int u = 0; u < kI4MergeRows; ++u) {
      if (ml[u].y == 0.f) continue;   // no key of that part, or not a part
      const float w = exp2f(ml[u].x - M);
      L = fmaf(w, ml[u].y, L);
#pragma unroll
      for (int e = 0; e < EPL; ++e) O[e] = fmaf(w, v[u][e], O[e]);
    }
  }
  if (lane == 0) {
    sm[warp] = M;
    sl[warp] = L;
  }
#pragma unroll
  for (int e = 0; e < EPL; ++e) so[warp][lane * EPL + e] = O[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float mx = sm[0];
#pragma unroll
    for (int w = 1; w < kI4Warps; ++w) mx = fmaxf(mx, sm[w]);
    float sum = 0.f, x = 0.f;
#pragma unroll
    for (int w = 0; w < kI4Warps; ++w) {
      const float k = exp2f(sm[w] - mx);
      sum = fmaf(k, sl[w], sum);
      x = fmaf(k, so[w][threadIdx.x], x);
    }
    out[threadIdx.x] = Elem<T>::narrow(sum > 0.f || sum != sum ? x / sum : 0.f);
  }
}

template <typename T, int D, bool kFull>
cudaError_t launch_int4(const DecodeInt4Args& a, cudaStream_t stream) {
  using C = I4Cfg<D>;
  auto kern = paged_decode_int4_kernel<T, D, kFull>;
  static std::atomic<int> ctas_per_sm[64];   // 0: not yet asked
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int per_sm = ctas_per_sm[dev].load(std::memory_order_relaxed);
  if (per_sm <= 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kI4Threads, C::kSmem);
    if (e != cudaSuccess) return e;
    if (per_sm <= 0) return cudaErrorInvalidConfiguration;
    ctas_per_sm[dev].store(per_sm, std::memory_order_relaxed);
  }
  // no more warps than the partials have slots for
  const int grid = std::min(per_sm * a.num_sms, a.max_warps / kI4Warps);
  if (a.ev_start) cudaEventRecord(a.ev_start, stream);
  e = launch_pdl(kern, dim3(grid), dim3(kI4Threads), C::kSmem, stream, a);
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged_decode_int4_merge_kernel<T, D>, dim3(a.B * a.Hq), dim3(kI4Threads), 0,
                 stream, a);
  if (e != cudaSuccess) return e;
  if (a.ev_stop) cudaEventRecord(a.ev_stop, stream);
  return cudaSuccess;
}

template <typename T>
cudaError_t launch_int4_t(const DecodeInt4Args& a, cudaStream_t stream) {
  const bool full = a.Hq / a.Hkv > 4;
  if (a.D == 64)
    return full ? launch_int4<T, 64, true>(a, stream) : launch_int4<T, 64, false>(a, stream);
  return full ? launch_int4<T, 128, true>(a, stream) : launch_int4<T, 128, false>(a, stream);
}

}  // namespace

cudaError_t launch_paged_decode_int4(const DecodeInt4Args& a, cudaStream_t stream) {
  return a.dtype == 1 ? launch_int4_t<__half>(a, stream) : launch_int4_t<__nv_bfloat16>(a, stream);
}

}  // namespace photon
