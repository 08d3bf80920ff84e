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
// fp16 ends at 2^-24, and what p_j step_j loses there the sums of p_j and p_j
// lo_j still count, so that many keys of little weight each (the tail behind a
// first key that holds nearly all) would pull the output towards their lo: by
// up to keys x 2^-25 of half a row's range, 1.5e-3 with 13900 keys at e^-17.
// So columns 4 .. 7 hold 2^14 times the residual, and with G = 8, where both
// go to the same sums, the weights fill fp16's upper end instead (kOne,
// kSlack): nothing above 2^-38 (G = 8: 2^-36) of the largest p_j step_j is lost.
//
// Work: a team of up to 8 neighbouring warps takes as many neighbouring KV
// heads, a warp each, through the same blocks, so that what it reads of a block
// is contiguous in the pool: 8 records are 8.7 KB, one is 1088 bytes.  The
// batch's (sequence, head group, block) triples in that order are one line,
// cut into equal runs, one per team; each (sequence, head group) counts
// kI4PairCost blocks more than it has, for what beginning and ending it costs.
// A warp has its own ring of cp.async stages and no barrier with any other
// warp.  A pair that lies in one run is written out directly, the others leave
// (m, l, o) partials, merged by a second kernel.  Runs are equal whatever the
// mix of lengths, without a queue or atomics, so results do not depend on
// timing.
//
// Measured (8 kv heads, d = 128, fp16; event times): 64 contexts of 128 .. 8192
// tokens 34.8 us = 4.0 TB/s of the codes and pairs, 59 % of the measured copy
// rate; a batch-256 mix at 32 q heads 65.0 us = 59 %; 4 short contexts 9.3 us.
// At 64 q heads (G = 8) contexts that take 32.8 us at 16 take 41.6: twice the P V
// products, and at d = 128 a few spilled registers.  Few long contexts: 4 of
// 65536 tokens 58 us = 4.9 TB/s, 8 of 131072 at 64 q heads 205 us = 5.6 TB/s.
// What bounds it: the first data comes 4 us after the call's start and the merge
// takes 3.5 us; between them 5.5 TB/s, the rate of the copies themselves: with
// no arithmetic at all the first version of this split took 34.5 us where it
// took 37.0.  The short contexts are two launches and a merge.  Other ways to
// bring the records in, at the same three: bulk copies per warp 33.7, 74.8, 9.5
// us; bulk copies into one ring a team 35.0, 74.3, 9.7; one warp per run of
// one KV head, without teams, 37.2, 69.5, 9.3.
#include <math.h>

#include <algorithm>

#include "int4_common.cuh"

namespace photon {
namespace {

constexpr int kI4Warps = kInt4CtaWarps;   // warps per CTA
constexpr int kI4Threads = 32 * kI4Warps;
// What beginning and ending a pair (its q rows, the sums over the warp, the
// output or a partial) costs a warp, in blocks of keys.  With 3, 4, 5, 6, 7, 8: a
// batch-256 mix 87.2, 83.8, 80.6, 79.4, 80.5, 80.1 us, 64 long contexts 33.7,
// 32.9, 32.8, 32.7, 33.2, 32.8, 256 of 128 .. 4096 tokens 66.7, 66.1, 65.2, 65.1,
// 66.8, 66.9.
constexpr int kI4PairCost = 6;
// Shortest run of a team on the line (4 contexts of up to 2048 tokens: 6 and
// 8: 9.0 and 9.6 us).
constexpr int kI4MinRun = 6;
// Running maximum before the first key: below the scores, and finite, so that
// no exponent is inf - inf.
constexpr float kI4NoMax = -3e38f;
constexpr int kI4StageUnits = 2;          // consecutive blocks of a pair in a stage
constexpr float kI4Rest = 16384.f;        // columns 4 .. 7: the residuals times this

template <int D>
struct I4Cfg {
  static constexpr int kRec = int4_record_bytes(D);
  static constexpr int kUnit = 2 * kRec;                 // K record, V record
  static constexpr int kStageBytes = kI4StageUnits * kUnit;
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr int kCtas = 2;                        // per SM (registers)
  static constexpr int kSmem = kI4Warps * kStages * kStageBytes;
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
// First product of a sum: D = A B.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// 2^(e - 127) from a biased exponent.
__device__ __forceinline__ float pow2_biased(int e) {
  return __uint_as_float((uint32_t)min(max(e, 1), 254) << 23);
}

// A team's place on the line: block `blk` of head group hg of sequence b, whose
// context has n blocks; block 0 is at `first` on the line.
struct I4Cursor {
  int b, hg, blk, n, ctx, first;
};

template <typename T, int D, bool kFull>
__global__ void __launch_bounds__(kI4Threads, I4Cfg<D>::kCtas)
    paged_decode_int4_kernel(const DecodeInt4Args a) {
  using C = I4Cfg<D>;
  constexpr int NW = D / 32;        // code words of a lane per row (or row pair)
  // Weights stay below 2^kSlack, V steps, once a power of two has brought the
  // largest below kOne, below kMost; their product is below 2^15 (G = 8), 2^11.
  constexpr float kSlack = kFull ? 2.f : 8.f;
  constexpr float kOne = kFull ? 4096.f : 1.f, kMost = kFull ? 8192.f : 8.f;
  extern __shared__ __align__(16) unsigned char i4_smem[];
  __shared__ int pre[kI4Threads];      // where a thread's sequences begin on the line
  __shared__ int ctx_first[kI4Threads];   // the lengths, when a thread has one sequence
  __shared__ int warp_sum[kI4Warps];

  {
    // while the kernel before runs out: the lengths, tables and q rows, spread
    // over the CTAs, into L2, a line a thread (hints; what that kernel still
    // writes is read after the wait)
    const size_t line = (size_t)blockIdx.x * kI4Threads + threadIdx.x, at = line * 128;
    if (at < (size_t)a.B * 4) prefetch_l2(reinterpret_cast<const char*>(a.context_lens) + at);
    if (at < (size_t)a.B * a.MBS * 4) prefetch_l2(reinterpret_cast<const char*>(a.block_tables) + at);
    if (at < (size_t)a.B * a.Hq * D * 2) prefetch_l2(static_cast<const char*>(a.q) + at);
  }
  pdl_wait_primary();
  pdl_launch_dependents();   // after the wait: the merge kernel reads the lengths ahead of its own
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int G = a.Hq / a.Hkv;
  const int span = a.MBS * kBlockSize;
  // the contexts' lengths; the merge kernel flags rejected ones
  const int per_thread = (a.B + kI4Threads - 1) / kI4Threads;
  auto load_ctx = [&](int b) -> int {
    const int c = __ldg(a.context_lens + b);
    return c > 0 && c <= span ? c : 0;
  };
  auto ctx_of = [&](int b) -> int { return per_thread == 1 ? ctx_first[b] : load_ctx(b); };
  auto blocks_of = [](int ctx) -> int { return (ctx + kBlockSize - 1) / kBlockSize; };
  auto pair_len = [](int blocks) -> int { return blocks ? blocks + kI4PairCost : 0; };

  // ---- the line: thread i sums sequences [i c, (i + 1) c)
  int mine = 0;
  for (int i = 0; i < per_thread; ++i) {
    const int b = tid * per_thread + i;
    const int ctx = b < a.B ? load_ctx(b) : 0;
    if (i == 0) ctx_first[tid] = ctx;
    mine += pair_len(blocks_of(ctx));
  }
  const int groups = a.Hkv / a.team;   // head groups
  mine *= groups;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kI4Warps; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  pre[tid] = before + incl - mine;
  __syncthreads();
  const int teams = (int)gridDim.x * kI4Warps / a.team;
  const int per = max((total + teams - 1) / teams, kI4MinRun);
  const int w_id = (int)blockIdx.x * kI4Warps + warp;
  const int team = w_id / a.team, member = w_id - team * a.team;
  if (total == 0 || team > (total - 1) / per) return;
  const int run_begin = team * per, run_end = min(run_begin + per, total);

  // ---- the run's first pair: the last thread whose sequences begin at or
  // before it, then a walk over that thread's sequences
  I4Cursor cur;
  {
    int owner = 0;
#pragma unroll
    for (int i = 0; i < kI4Warps; ++i) {
      const unsigned at = __ballot_sync(0xffffffffu, pre[i * 32 + lane] <= run_begin);
      if (at) owner = i * 32 + 31 - __clz(at);
    }
    int left = run_begin - pre[owner];
    cur.b = owner * per_thread;
    while (true) {   // ends inside the owner's sequences: run_begin < total
      cur.ctx = ctx_of(cur.b);
      cur.n = blocks_of(cur.ctx);
      const int len = pair_len(cur.n) * groups;
      if (left < len || cur.b + 1 >= a.B) break;
      left -= len;
      ++cur.b;
    }
    const int len = pair_len(cur.n);
    cur.hg = left / len;
    left -= cur.hg * len;
    cur.first = run_begin - left + kI4PairCost;
    cur.blk = max(0, left - kI4PairCost);
  }
  // blocks of the cursor's pair that are still in the run
  auto blocks_left = [&](const I4Cursor& c) -> int {
    return min(c.n, run_end - c.first) - c.blk;
  };
  // to the next pair; past the last sequence there is none
  auto next_pair = [&](I4Cursor& c) {
    c.blk = 0;
    c.first += c.n + kI4PairCost;
    if (++c.hg < groups) return;
    c.hg = 0;
    do {
      if (++c.b >= a.B) {
        c.n = 0;
        return;
      }
      c.ctx = ctx_of(c.b);
      c.n = blocks_of(c.ctx);
    } while (c.n == 0);
  };
  // the run may begin or end in what a pair costs beside its blocks
  if (blocks_left(cur) <= 0) return;

  // ---- the ring: a stage takes up to two consecutive blocks of one pair
  unsigned char* ring = i4_smem + warp * (C::kStages * C::kStageBytes);
  const uint32_t ring_addr = smem_addr(ring) + 16 * lane;
  // this lane's places in a record's codes, and in the pairs of a K record
  // (lanes 0 .. 3) and a V record (4 .. 7)
  const unsigned char* k_codes = static_cast<const unsigned char*>(a.k_cache) + 16 * lane;
  const unsigned char* v_codes = static_cast<const unsigned char*>(a.v_cache) + 16 * lane;
  const unsigned char* pairs = (lane < 4 ? k_codes : v_codes - 64) + 8 * D;
  const uint32_t pairs_to = lane < 4 ? 8 * D : C::kRec + 8 * D - 64;
  // The next 32 stages' records, one stage a lane: record numbers of its two
  // blocks; kGone for a block that is not in the pool, kNone for no block.
  I4Cursor fetch = cur;
  int stages_found = 0, issued = 0;
  bool more = true;   // blocks of the run are left to find
  constexpr uint32_t kGone = 0xfffffffeu, kNone = 0xffffffffu;
  uint32_t rec0 = kNone, rec1 = kNone;
  auto find = [&]() {
    int have = 0;
    rec0 = rec1 = kNone;
    while (have < 32 && more) {
      const int units = blocks_left(fetch);
      const int i = kI4StageUnits * (lane - have);
      const int32_t* entry = a.block_tables + (size_t)fetch.b * a.MBS + fetch.blk + i;
      const int kvh = fetch.hg * a.team + member;
      if (i >= 0 && i < units) {
        const int p0 = __ldg(entry), p1 = i + 1 < units ? __ldg(entry + 1) : 0;
        rec0 = (unsigned)p0 < (unsigned)a.NB ? (uint32_t)(p0 * a.Hkv + kvh) : kGone;
        if (i + 1 < units)
          rec1 = (unsigned)p1 < (unsigned)a.NB ? (uint32_t)(p1 * a.Hkv + kvh) : kGone;
        if (rec0 == kGone || rec1 == kGone) raise_error(a.err, kErrBlock);
      }
      const int taken = min(units, kI4StageUnits * (32 - have));
      have += (taken + kI4StageUnits - 1) / kI4StageUnits;
      fetch.blk += taken;
      if (taken == units) {
        next_pair(fetch);
        more = fetch.n > 0 && blocks_left(fetch) > 0;
      }
    }
    stages_found += have;
  };
  uint32_t absent = 0;   // bit 2 s + i: block i of stage s is not in the pool
  auto issue = [&](int s) {
    if ((issued & 31) == 0 && more) find();
    if (issued < stages_found) {
      const uint32_t dst = ring_addr + s * C::kStageBytes;
#pragma unroll
      for (int i = 0; i < kI4StageUnits; ++i) {
        const uint32_t rec = __shfl_sync(0xffffffffu, i ? rec1 : rec0, issued & 31);
        const uint32_t bit = 1u << (2 * s + i);
        if (rec < kGone) {
          const size_t off = (size_t)rec * C::kRec;
          const unsigned char* kp = k_codes + off;
          const unsigned char* vp = v_codes + off;
#pragma unroll
          for (int o = 0; o < 8 * D; o += 512) {
            cp_async16(dst + i * C::kUnit + o, kp + o);
            cp_async16(dst + i * C::kUnit + C::kRec + o, vp + o);
          }
          if (lane < 8) cp_async16(dst + i * C::kUnit + pairs_to, pairs + off);
          absent &= ~bit;
        } else {
          absent |= bit;
        }
      }
      ++issued;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) issue(s);

  // ---- a pair's state.  Columns (slots) 2t and 2t + 1 of the score fragment
  // are this lane's; with G <= 4 column 4 + s repeats slot s.
  uint32_t bq[NW][2][2];   // Q^T fragments: column g, products 2j and 2j + 1 of word j
  // score = (step f acc + lo c2) c1: c1 a power of two, f the rest of the scale, in
  // [1, 2).  So the maximum, scaled, is exact, and so is what the weights next to it
  // are taken from.  With c1 the whole factor the maximum would be rounded, from
  // 2^24 on by whole units, and a weight of 1 could be any power of two.  (Batch-256
  // mix 79.5 -> 81.2 us, others the same; differences of scores instead 81.2 too, a
  // branch for large scores only 80.5, but 64 long contexts 33.0 -> 33.4.)
  const float f = __uint_as_float((__float_as_uint(a.qscale) & 0x7fffffu) | 0x3f800000u);
  float c1[2], c2[2];
  float m[2], l[2], z[2];  // running max, sum of weights, sum of weights x lo of V
  float limit[2];          // (m + kSlack) / c1: what a score / c1 may reach before m moves
  float o[NW][2][4];       // O^T: dims (D / 8) g + 4j + 2h (rows g) and + 1 (rows g + 8)
  float vs = 0.f;          // power of two that the V steps are brought near kOne with
  auto begin_pair = [&]() {
    const int s = kFull ? g : g & 3;
    float x[NW * 8];
#pragma unroll
    for (int i = 0; i < NW * 8; ++i) x[i] = 0.f;
    if (s < G) {
      const T* row = static_cast<const T*>(a.q) +
                     ((size_t)cur.b * a.Hq + (size_t)(cur.hg * a.team + member) * G + s) * D + (D / 4) * t;
#pragma unroll
      for (int i = 0; i < NW; ++i) Elem<T>::widen(__ldg(reinterpret_cast<const uint4*>(row) + i), x + 8 * i);
    }
    float big = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < NW * 8; ++i) {
      big = fmaxf(big, fabsf(x[i]));
      sum = fmaf(x[i], 9.765625e-4f, sum);   // 2^-10 of it: a row of bf16's largest stays finite
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
      sum += __shfl_xor_sync(0xffffffffu, sum, off);
    }
    // the row's largest element is scaled by a power of two to [2^14, 2^15): fp16
    // then holds q and its 16th exactly down to 2^-24 of the largest, and what
    // is smaller to 2^-25, less than 2^-35 of it
    const int ex = (int)((__float_as_uint(big) >> 23) & 255u);
    const float up = pow2_biased(268 - ex);   // 2^(14 - (ex - 127))
    // with a negative scale q is turned round, so that the largest score is
    // the largest sum
    const float sc = a.qscale < 0.f ? -up : up;
    const float s16 = sc * 0.0625f;
#pragma unroll
    for (int j = 0; j < NW; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float* w = x + 8 * j + 2 * h;
        bq[j][h][0] = Mma<__half>::pack(w[0] * sc, w[4] * sc);
        bq[j][h][1] = Mma<__half>::pack(w[1] * s16, w[5] * s16);
      }
    // acc = 2^-24 sc (q . n), so lo enters as lo sum(q) 2^-24 sc; 1 / up is exact.
    // The factor stays positive and finite, whatever the scale and q: with a
    // zero scale or a zero row every weight is 1, but the -inf of a key that
    // is not there has to remain one (-inf x 0 is NaN), and so has a score of 0
    // (0 x inf).
    const float whole = __uint_as_float(__float_as_uint(a.qscale) & 0x7f800000u);   // |qscale| / f
    const float k1 = fminf(fmaxf((whole * 16777216.f) * (1.f / up), 1.8807910e-37f), 1.7014118e38f);
    const float k2 = sum * (sc * 6.1035156e-5f) * f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int col = 2 * t + i;
      c1[i] = __shfl_sync(0xffffffffu, k1, (kFull ? col : col & 3) * 4);
      c2[i] = __shfl_sync(0xffffffffu, k2, (kFull ? col : col & 3) * 4);
      m[i] = kI4NoMax;
      limit[i] = -INFINITY;
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

  // One stage: 32 keys, of which `keys` are in the context; bit i of `gone`:
  // block i is not there (both only matter to the last stage of a pair, or
  // with a bad table).
  auto attend = [&](const unsigned char* st, int keys, uint32_t gone) {
    float y[kI4StageUnits][4];   // score / c1 of keys g (0, 1) and g + 8 (2, 3), slots 2t, 2t + 1
    float step0[kI4StageUnits], step8[kI4StageUnits], low0[kI4StageUnits], low8[kI4StageUnits];
#pragma unroll
    for (int u = 0; u < kI4StageUnits; ++u) {
      const unsigned char* kr = st + u * C::kUnit;
      uint32_t k0[NW], k8[NW];   // K: rows g and g + 8
      words(kr + g * (D / 2) + t * (D / 8), k0);
      words(kr + (g + 8) * (D / 2) + t * (D / 8), k8);
      const uint32_t kp0 = *reinterpret_cast<const uint32_t*>(kr + 8 * D + 4 * g);
      const uint32_t kp8 = *reinterpret_cast<const uint32_t*>(kr + 8 * D + 4 * g + 32);
      const uint32_t vp0 = *reinterpret_cast<const uint32_t*>(kr + C::kRec + 8 * D + 4 * g);
      const uint32_t vp8 = *reinterpret_cast<const uint32_t*>(kr + C::kRec + 8 * D + 4 * g + 32);
      float acc[4];
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        const uint32_t x = k0[j], w = k8[j], x8 = x >> 8, w8 = w >> 8;
        const uint32_t f0[4] = {x & 0x000f000fu, w & 0x000f000fu, x & 0x00f000f0u,
                                w & 0x00f000f0u};
        const uint32_t f1[4] = {x8 & 0x000f000fu, w8 & 0x000f000fu, x8 & 0x00f000f0u,
                                w8 & 0x00f000f0u};
        if (j == 0)
          mma_first(acc, f0, bq[j][0][0], bq[j][0][1]);
        else
          Mma<__half>::run(acc, f0, bq[j][0][0], bq[j][0][1]);
        Mma<__half>::run(acc, f1, bq[j][1][0], bq[j][1][1]);
      }
      const float ks0 = Bits16<T>::to_f32(kp0 & 0xffffu) * f, kl0 = Bits16<T>::to_f32(kp0 >> 16);
      const float ks8 = Bits16<T>::to_f32(kp8 & 0xffffu) * f, kl8 = Bits16<T>::to_f32(kp8 >> 16);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y[u][i] = fmaf(i < 2 ? ks0 : ks8, acc[i], (i < 2 ? kl0 : kl8) * c2[i & 1]);
      step0[u] = Bits16<T>::to_f32(vp0 & 0xffffu);
      step8[u] = Bits16<T>::to_f32(vp8 & 0xffffu);
      low0[u] = Bits16<T>::to_f32(vp0 >> 16);
      low8[u] = Bits16<T>::to_f32(vp8 >> 16);
    }
    if (keys < 16 * kI4StageUnits || gone) {
      // what lies behind the context may hold anything
#pragma unroll
      for (int u = 0; u < kI4StageUnits; ++u) {
        const int valid = (gone >> u) & 1u ? 0 : keys - 16 * u;
        if (g >= valid) {
          y[u][0] = y[u][1] = -INFINITY;
          step0[u] = low0[u] = 0.f;
        }
        if (g + 8 >= valid) {
          y[u][2] = y[u][3] = -INFINITY;
          step8[u] = low8[u] = 0.f;
        }
      }
    }
    // The maximum only moves when a score passes it by more than kSlack (then
    // weights stay below 2^kSlack), the V steps' power of two when a step passes
    // kMost; what is summed so far is rescaled then.  Both cancel in O / l.
    const float y0 = fmaxf(fmaxf(y[0][0], y[0][2]), fmaxf(y[1][0], y[1][2]));
    const float y1 = fmaxf(fmaxf(y[0][1], y[0][3]), fmaxf(y[1][1], y[1][3]));
    const float top = fmaxf(fmaxf(step0[0], step8[0]), fmaxf(step0[1], step8[1]));
    if (__any_sync(0xffffffffu, y0 > limit[0] || y1 > limit[1] || top * vs > kMost)) {
      float n0 = fmaxf(m[0], y0 * c1[0]), n1 = fmaxf(m[1], y1 * c1[1]);
      float sm = top;
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, off));
        n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, off));
        sm = fmaxf(sm, __shfl_xor_sync(0xffffffffu, sm, off));
      }
      const float r0 = softmax_exp2(m[0] - n0), r1 = softmax_exp2(m[1] - n1);
      float up = 1.f;
      if (sm * vs > kOne) {
        // kOne x 2^-(exponent of sm + 1)
        const float next = pow2_biased(253 + (kFull ? 12 : 0) - (int)((__float_as_uint(sm) >> 23) & 255u));
        up = next * (1.f / vs);
        vs = next;
      }
      m[0] = n0;
      m[1] = n1;
      limit[0] = __fadd_rd(n0, kSlack) / c1[0];   // not above m + kSlack, however large m is
      limit[1] = __fadd_rd(n1, kSlack) / c1[1];
      l[0] *= r0, z[0] *= r0;
      l[1] *= r1, z[1] *= r1;
#pragma unroll
      for (int j = 0; j < NW; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][h][i] *= (i & 1 ? r1 : r0) * up;
    }
#pragma unroll
    for (int u = 0; u < kI4StageUnits; ++u) {
      const unsigned char* vr = st + u * C::kUnit + C::kRec;
      uint32_t v0[NW], v4[NW];   // V: row pairs t and t + 4
      words(vr + t * D + g * (D / 8), v0);
      words(vr + (t + 4) * D + g * (D / 8), v4);
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = softmax_exp2(fmaf(y[u][i], c1[i & 1], -m[i & 1]));   // 0 for masked rows
        l[i & 1] += p;
        z[i & 1] = fmaf(p, i < 2 ? low0[u] : low8[u], z[i & 1]);
        w[i] = p * ((i < 2 ? step0[u] : step8[u]) * vs);
      }
      // P^T fragments: the fp16 rounding, and its residual in columns 4 .. 7
      // (their scores repeat columns 0 .. 3) or, with eight slots, in a
      // second product
      uint32_t h01 = Mma<__half>::pack(w[0], w[1]), h23 = Mma<__half>::pack(w[2], w[3]);
      const float2 r01 = Mma<__half>::unpack(h01), r23 = Mma<__half>::unpack(h23);
      uint32_t b0, b1, d0 = 0u, d1 = 0u;
      if constexpr (kFull) {
        b0 = movmatrix_trans(h01);
        b1 = movmatrix_trans(h23);
        d0 = movmatrix_trans(Mma<__half>::pack(w[0] - r01.x, w[1] - r01.y));
        d1 = movmatrix_trans(Mma<__half>::pack(w[2] - r23.x, w[3] - r23.y));
      } else {
        const float mul = t >= 2 ? kI4Rest : 1.f, rest = t >= 2 ? -kI4Rest : 0.f;
        b0 = movmatrix_trans(
            Mma<__half>::pack(fmaf(rest, r01.x, w[0] * mul), fmaf(rest, r01.y, w[1] * mul)));
        b1 = movmatrix_trans(
            Mma<__half>::pack(fmaf(rest, r23.x, w[2] * mul), fmaf(rest, r23.y, w[3] * mul)));
      }
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        // rows g: nibble 0 (2) alone; rows g + 8: it and the next one, n + 16 n',
        // parted at the end: a mask less per word
        const uint32_t p = v0[j], q = v4[j];
        const uint32_t p8 = __byte_perm(p, 0u, 0x4341), q8 = __byte_perm(q, 0u, 0x4341);
        const uint32_t f0[4] = {p & 0x000f000fu, p & 0x00ff00ffu, q & 0x000f000fu,
                                q & 0x00ff00ffu};
        const uint32_t f1[4] = {p8 & 0x000f000fu, p8, q8 & 0x000f000fu, q8};
        Mma<__half>::run(o[j][0], f0, b0, b1);
        Mma<__half>::run(o[j][1], f1, b0, b1);
        if constexpr (kFull) {
          Mma<__half>::run(o[j][0], f0, d0, d1);
          Mma<__half>::run(o[j][1], f1, d0, d1);
        }
      }
    }
  };

  // the pair's sums over the warp; then out, or a partial
  auto end_pair = [&]() {
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
          if constexpr (!kFull) {
            const float other = __shfl_xor_sync(0xffffffffu, o[j][h][i], 2);
            o[j][h][i] = fmaf(other, 1.f / kI4Rest, o[j][h][i]);   // lanes t < 2 go on with it
          }
        }
#pragma unroll
    for (int j = 0; j < NW; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // rows g + 8 hold the even dim's sum and 16 times the odd one's
          const float even = o[j][h][i], odd = o[j][h][2 + i] - even;
          o[j][h][i] = fmaf(even * 16777216.f, unscale, z[i]);
          o[j][h][2 + i] = fmaf(odd * 1048576.f, unscale, z[i]);
        }
    // the pair's partials: one for each team whose run touches it; along the
    // line either the team or the pair moves on, so their sum numbers them
    const int kvh = cur.hg * a.team + member, pair = cur.b * groups + cur.hg;
    const int t_first = cur.first / per, t_last = (cur.first + cur.n - 1) / per;
    if (team == t_first && lane == 0)
      a.ws_pair[cur.b * a.Hkv + kvh] =
          make_int2((t_first + pair) * a.team + member, t_last - t_first + 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = 2 * t + i;
      if (s >= G || (!kFull && t >= 2)) continue;
      if (t_first == t_last) {
        const float inv = l[i] > 0.f || l[i] != l[i] ? 1.f / l[i] : 0.f;
        T* dst = static_cast<T*>(a.out) + ((size_t)cur.b * a.Hq + (size_t)kvh * G + s) * D + (D / 8) * g;
#pragma unroll
        for (int j = 0; j < NW; j += 2)
          *reinterpret_cast<uint4*>(dst + 4 * j) =
              make_uint4(Mma<T>::pack(o[j][0][i] * inv, o[j][0][2 + i] * inv),
                         Mma<T>::pack(o[j][1][i] * inv, o[j][1][2 + i] * inv),
                         Mma<T>::pack(o[j + 1][0][i] * inv, o[j + 1][0][2 + i] * inv),
                         Mma<T>::pack(o[j + 1][1][i] * inv, o[j + 1][1][2 + i] * inv));
      } else {
        const size_t row = ((size_t)(team + pair) * a.team + member) * G + s;
        if (g == 0) a.ws_ml[row] = make_float2(m[i], l[i]);
        float4* dst = reinterpret_cast<float4*>(a.ws_o + row * D + (D / 8) * g);
#pragma unroll
        for (int j = 0; j < NW; ++j)
          dst[j] = make_float4(o[j][0][i], o[j][0][2 + i], o[j][1][i], o[j][1][2 + i]);
      }
    }
  };

  int stage = 0;
  while (true) {   // pairs
    begin_pair();
    int units = blocks_left(cur);
    int keys = min(cur.ctx - cur.blk * kBlockSize, units * kBlockSize);
    for (; units > 0; units -= kI4StageUnits, keys -= kI4StageUnits * kBlockSize) {
      cp_async_wait<C::kStages - 2>();
      __syncwarp();
      attend(ring + stage * C::kStageBytes, keys, (absent >> (2 * stage)) & 3u);
      __syncwarp();   // every lane has read the stage before it is filled again
      issue(stage == 0 ? C::kStages - 1 : stage - 1);
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
    }
    end_pair();
    next_pair(cur);
    if (cur.n == 0 || blocks_left(cur) <= 0) break;
  }
  cp_async_wait<0>();
}

// out = sum_p w_p o_p / sum_p w_p l_p with w_p = 2^(m_p - max m) over the
// partials of a (sequence, q head), and the zero rows of empty sequences.
// kSplit warps take an item, each every kSplit-th group of 8 partials, loaded
// at once.  4 when the items are few (their partials are then many: up to 32
// cost one round trip), 1 when they fill the device (batch-256 mix, 8192
// items, most of them written by the attention kernel).
constexpr int kI4MergeRows = 8, kI4MergeWarps = 4;

template <typename T, int D, int kSplit>
__global__ void __launch_bounds__(32 * kI4MergeWarps)
    paged_decode_int4_merge_kernel(const DecodeInt4Args a) {
  constexpr int EPL = D / 32;
  __shared__ float sm[kI4MergeWarps], sl[kI4MergeWarps], so[kSplit > 1 ? kI4MergeWarps : 1][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = warp % kSplit;
  const int item = (int)blockIdx.x * (kI4MergeWarps / kSplit) + warp / kSplit;
  if (item >= a.B * a.Hq) return;   // (kSplit == 1, or the whole CTA)
  const int b = item / a.Hq, hq = item - b * a.Hq;
  const int G = a.Hq / a.Hkv;
  pdl_launch_dependents();
  // the attention kernel has passed its own wait: the lengths are there
  const int ctx = __ldg(a.context_lens + b);
  pdl_wait_primary();
  T* out = static_cast<T*>(a.out) + (size_t)item * D;
  if (ctx <= 0 || ctx > a.MBS * kBlockSize) {
    if (ctx != 0 && lane == 0 && part == 0 && hq == 0) raise_error(a.err, kErrContext);
    if (part == 0 && lane < D / 8) reinterpret_cast<uint4*>(out)[lane] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int2 pr = a.ws_pair[b * a.Hkv + hq / G];
  if (pr.y < 2) return;   // the attention kernel wrote out
  const size_t row0 = (size_t)pr.x * G + hq % G;
  float M = kI4NoMax, L = 0.f, O[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) O[e] = 0.f;
  for (int p0 = part * kI4MergeRows; p0 < pr.y; p0 += kSplit * kI4MergeRows) {
    float v[kI4MergeRows][EPL];
    float2 ml[kI4MergeRows];
#pragma unroll
    for (int u = 0; u < kI4MergeRows; ++u) {
      const bool in = p0 + u < pr.y;
      const size_t row = row0 + (size_t)(in ? p0 + u : p0) * G * a.team;
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
  if constexpr (kSplit == 1) {
    const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
#pragma unroll
    for (int e = 0; e < EPL; e += 2)
      *reinterpret_cast<uint32_t*>(out + lane * EPL + e) = Mma<T>::pack(O[e] * inv, O[e + 1] * inv);
  } else {
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
      for (int w = 1; w < kI4MergeWarps; ++w) mx = fmaxf(mx, sm[w]);
      float sum = 0.f, x = 0.f;
#pragma unroll
      for (int w = 0; w < kI4MergeWarps; ++w) {
        const float k = exp2f(sm[w] - mx);
        sum = fmaf(k, sl[w], sum);
        x = fmaf(k, so[w][threadIdx.x], x);
      }
      out[threadIdx.x] = Elem<T>::narrow(sum > 0.f || sum != sum ? x / sum : 0.f);
    }
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
  // from 16 items an SM (2432) on, a warp an item.  A warp against four: 1024 items of
  // 64 long contexts 35.4, 32.7 us; 2048 of a mix 31.4, 28.9, of long contexts 54.5,
  // 55.3; 2560 of a mix 34.2, 33.3; 4096 of a mix 47.8, 49.3, of long contexts 65.2,
  // 69.9; 8192 of a mix 79.4, 85.2, of short contexts 18.4, 24.4
  const int items = a.B * a.Hq;
  e = items >= 16 * a.num_sms
          ? launch_pdl(paged_decode_int4_merge_kernel<T, D, 1>,
                       dim3((items + kI4MergeWarps - 1) / kI4MergeWarps), dim3(32 * kI4MergeWarps),
                       0, stream, a)
          : launch_pdl(paged_decode_int4_merge_kernel<T, D, kI4MergeWarps>, dim3(items),
                       dim3(32 * kI4MergeWarps), 0, stream, a);
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
