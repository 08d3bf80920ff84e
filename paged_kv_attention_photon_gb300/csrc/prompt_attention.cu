// prompt_attention.cu -- causal attention of packed whole prompts over their
// own K and V rows, on the fifth-generation tensor cores.
//
// PhotonInfer README, "Roadmap": FlashAttention-2 style IO-aware attention for
// long sequences.
//
// For token i and q head h of a prompt, out = sum_{j <= i} softmax_j(scale
// q . k_j) v_j: S = Q K^T, P = 2^(S - m), O += P V per chunk of 128 keys with
// a running maximum m and sum l, so scores never leave the SM.  4 Hq d
// sum n (n + 1) / 2 flops against 2 n (Hq + Hkv) d elements: the tensor cores
// bound it.  So P enters the second product rounded to the storage type, in one
// product (with a residual, as the decode has it, there would be half again as
// many); sums and statistics are fp32.  Against 64 bits the output's error is
// 1.25 (fp16) to 1.35 times (bf16) that of one rounding at the end.
//
// A persistent CTA per SM takes items of 256 query rows of one (prompt, KV
// head) -- row r is (token r / G, head r % G), so one K/V chunk serves the
// whole group -- as two tiles of 128 rows, and runs 15 warps in fixed roles:
//   warps 0-3, 4-7  softmax of tile 0, 1: thread r owns TMEM lane r
//   warp 8, 9       tensor-map copies of Q and K, of V (128-byte swizzle)
//   warp 10, 11     issue S of tile 0, 1
//   warp 12, 13     issue P V of tile 0, 1
//   warp 14         finds the items
// Per tile, TMEM holds S (128 columns) and O (D columns).  S, softmax and P V
// go by halves of 64 keys, each half with its own barriers: P of a half lies
// over its S as 16-bit pairs and is read from there as the A operand, so the
// softmax of one half runs while S or P V of the other does.  (With S of all 128
// keys at once the tensor cores reach their rate on it, but a chunk is one long
// chain: 1 x 16384 tokens 0.73 ms against 0.64 ms by halves (a few calls in a row).  At d = 64 TMEM has
// room for a P apart from S; by halves that is slower, 4 x 4096 tokens 0.356 ms
// against 0.30 to 0.33 ms.)  An issuing warp is held up for hundreds of clocks by
// each of its commits, hence four of them; issued from inside one elected
// lane's branch a product costs 50 clocks, predicated in the whole warp 75 to
// 95.  Copies run ahead across items, and the next item's first S products
// overlap this one's epilogue.
//
// Measured (16 q, 8 kv heads, d = 128): 1 x 16384 tokens, bf16, 0.64 ms = 1718
// TFLOP/s over 20 calls, 91 % of the measured dense burst rate; over 1000 calls
// the power limit lowers the clock (2070 to about 1800 MHz) and it is 0.69 ms =
// 1594 TFLOP/s, 94 % of the sustained rate; whether the inputs change makes no
// difference.  16 x 1024, fp16, 64 us = 1080 TFLOP/s.  At d = 64 (32 q, 8 kv heads, fp16) 4 x 4096 tokens take 0.30 to
// 0.33 ms = 840 to 920 TFLOP/s: the products are half as long for the same
// softmax, which bounds it.  In short prompts the items do: ending one and
// starting the next costs a tile about 3000 clocks (the last P V 120, the
// output's four turns of 430, the next item and its first S 750), when a chunk
// of 128 keys takes about 2200.  Asking for the next item's Q ahead of time (a
// prefetch into L2) made 16 x 1024 slower, 66.5 against 64.9 us; coalesced
// stores from shared memory in place of the output's tensor copies 66.9 against
// 63.7 us.
//
// Items are numbered tile by tile from the prompts' far ends (the longest key
// ranges) to their beginnings, and dealt to the CTAs forwards and backwards in
// turn, so that all finish close together; each CTA finds its items from the
// lengths alone (pa_locate), without a queue.
//
// Barriers complete once per use; use i has parity i & 1:
//   k_full, v_full[st]   a chunk landed      k_free, v_free[st]  both tiles are done with it
//   q_full[t]            Q tile landed       q_free[t]           the item's last S product is done
//   s_full[t][h]         S of 64 keys        p_full[t][h]        their P written
//   o_done[t][h]         O += P V of 64 keys done; the next chunk's S may overwrite P
//   item_full, item_free[i]  an item is known; every role has read it
// Where a wait runs out the CTA gives up, and what it has in flight still lands
// first: copies write its shared memory, products its tensor memory, and both
// arrive on its barriers.  Each warp waits (bounded) for its own: the copying
// ones on the barriers of their last copies, the issuing ones on
//   drained[i]           every product that the warp has issued is done
#include <math.h>

#include <algorithm>

#include "prompt_attention.cuh"
#include "tc_common.cuh"

namespace photon {
namespace {

constexpr int kPaRows = 128;            // query rows of a tile = TMEM lanes
constexpr int kPaKeys = 128;            // keys of a chunk
constexpr int kPaHalf = 64;             // keys of an S product, of a softmax step and of a P V product
constexpr int kPaTiles = 2;
constexpr int kPaItemRows = kPaTiles * kPaRows;
constexpr int kPaThreads = 512;        // four warpgroups; warp 15 has no role
// Registers a thread: 512 x 128 at launch, dealt anew to the softmax
// warpgroups and the other two (160 + 160 + 96 + 96 = 4 x 128).
constexpr int kPaSoftmaxRegs = 160, kPaOtherRegs = 96;
constexpr uint32_t kPaTmemO = 256;      // S of tile t: columns [128 t, 128 t + 128); then the O's
constexpr float kPaRescaleLog2 = 8.f;
// Weights are 2^(score - maximum + lift).  fp16 ends at 2^-24, and a weight that
// it loses the sum l still counts: the many keys of little weight behind one that
// holds nearly all would be lost together, 2^-25 of the largest |v| each.  The lift
// uses the upper end of its range (2^7 x 2^8 < 65504) and cancels in O / l.
template <typename T>
constexpr float kPaLift = std::is_same<T, __half>::value ? 7.f : 0.f;
constexpr float kPaNoMax = -3e38f;      // before the first key; finite, so that no exponent is inf - inf
// The weights' exponents are one operation on the scores, qm s + base.  base holds
// the scaled maximum, rounded, which is the same for all of a row's weights; but
// from this on (2^23) it is rounded by half a unit and more, and weights would leave
// fp16.  There fp32 scores are whole units of the exponent apart, so qm is the scale's
// power of two alone, with which the scaled maximum and the differences are exact.
constexpr float kPaFar = 8388608.f;
constexpr int kPaItems = 4;             // items found ahead
constexpr int kPaRoles = 14;            // warps that work on an item

template <int D>
struct PaCfg {
  static constexpr int kKStages = D == 128 ? 2 : 3;
  static constexpr int kVStages = D == 128 ? 2 : 3;
  static constexpr int kQBytes = kPaRows * D * 2;
  static constexpr int kKvBytes = kPaKeys * D * 2;
  static constexpr int kOffK = kPaTiles * kQBytes;
  static constexpr int kOffV = kOffK + kKStages * kKvBytes;
  static constexpr int kOffO = kOffV + kVStages * kKvBytes;   // a softmax warp's 2 x 2 KB: 32 rows x 32
  static constexpr int kSmem = kOffO + kPaTiles * 4 * 4096 + 1024;   // + alignment to a swizzle atom
};

// MN-major V operand (sw128_desc walked along N): 64-element blocks of N are
// kPaKeys rows of 128 bytes apart (leading offset), groups of 8 keys 1 KB.
__device__ __forceinline__ uint64_t pa_v_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)((kPaKeys * 128) >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void tma_load_box3(uint32_t dst, const CUtensorMap* map, int x, int y,
                                              int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// Tensor copy of a box from shared memory to global memory, in a bulk group of
// its own.
__device__ __forceinline__ void tma_store_box3(const CUtensorMap* map, int x, int y, int z,
                                               uint32_t src) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(z), "r"(src)
      : "memory");
}
// This thread's bulk stores, all but the N newest, have read their shared memory.
template <int N>
__device__ __forceinline__ void bulk_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Bounded wait for a barrier phase, by a whole warp; false after kWaitLimitNs,
// or once any other warp of the CTA has given up.
__device__ __forceinline__ bool pa_wait(uint64_t* bar, uint32_t parity, volatile int* gave_up) {
  bool ok = mbar_try_wait(bar, parity);
  if (!__all_sync(0xffffffffu, ok)) {
    const unsigned long long t0 = global_timer_ns();
    while (!ok) {
#pragma unroll 1
      for (int i = 0; i < 32 && !ok; ++i) ok = mbar_try_wait(bar, parity);
      if (ok || *gave_up) break;
      if (global_timer_ns() - t0 > kWaitLimitNs) *gave_up = 1;
    }
    ok = __all_sync(0xffffffffu, ok);
  }
  return ok;
}

struct PaItem {
  int q0;      // the prompt's first token
  int n;       // its tokens
  int kvh;
  int row0;    // first row of the item, counted from the prompt's first
};

// Items of prompt b: tiles of 256 rows; 0 for an empty or a rejected one.
__device__ __forceinline__ int pa_tiles_of(const PromptArgs& a, int G, int b) {
  if (b >= a.B) return 0;
  const int q0 = __ldg(a.query_start + b), q1 = __ldg(a.query_start + b + 1);
  if (q0 < 0 || q1 <= q0 || q1 > a.num_tokens || q1 - q0 > a.max_query_len) return 0;
  return ((q1 - q0) * G + kPaItemRows - 1) / kPaItemRows;
}

// Where a warp that looks for items in rising order stands.  Item L is KV head
// L % Hkv of the (L / Hkv)-th (prompt, tile), taken from the highest tile index
// of any prompt down, prompts in order within one index.  F(x), the number of
// (prompt, tile) with tile index >= x, falls with x: the tile index is the
// largest x with F(x) > L / Hkv.  Both x and the place among x's prompts only
// move one way, so all items of a CTA together cost a few passes over the
// lengths for each tile index that it meets.  4096 prompts of 8 .. 32 tokens
// (16 q, 8 kv heads, d = 128): 0.70 ms; with each item found anew it was 5.7, or
// 18 under a max_query_len of 16384, growing with the square of the prompts.
struct PaFinder {
  int x;                 // tile index
  uint32_t f, f_above;   // F(x), F(x + 1)
  uint32_t total;        // F(0)
  int b0;                // prompts from here on have not been looked at for x ..
  uint32_t before;       // .. and so many before them have a tile x
};

// `first` holds pa_tiles_of(lane).
__device__ __forceinline__ PaFinder pa_finder(const PromptArgs& a, int G, int first, int lane) {
  int s = first, longest = first;
  for (int b0 = 32; b0 < a.B; b0 += 32) {
    const int t = pa_tiles_of(a, G, b0 + lane);
    s += t;
    longest = max(longest, t);
  }
  PaFinder p;
  p.x = __reduce_max_sync(0xffffffffu, longest);
  p.total = __reduce_add_sync(0xffffffffu, (unsigned)s);
  p.f = p.f_above = p.before = 0;
  p.b0 = 0;
  return p;
}

// Item L, not below the last one asked for, by a whole warp; false past the last one.
__device__ __forceinline__ bool pa_locate(const PromptArgs& a, int G, uint32_t L, int first,
                                          int lane, PaFinder& p, PaItem& it) {
  auto tiles = [&](int b0) { return b0 == 0 ? first : pa_tiles_of(a, G, b0 + lane); };
  const uint32_t i = L / (uint32_t)a.Hkv;
  if (i >= p.total) return false;
  if (i >= p.f) {   // a lower tile index, the largest x with F(x) > i
    int lo = 0, hi = p.x;
    uint32_t f_lo = p.total, f_hi = p.f;
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      int s = 0;
      for (int b0 = 0; b0 < a.B; b0 += 32) s += max(0, tiles(b0) - mid);
      const uint32_t f = __reduce_add_sync(0xffffffffu, (unsigned)s);
      if (f > i) {
        lo = mid;
        f_lo = f;
      } else {
        hi = mid;
        f_hi = f;
      }
    }
    p.x = lo;
    p.f = f_lo;
    p.f_above = f_hi;
    p.b0 = 0;
    p.before = 0;
  }
  const uint32_t rank = i - p.f_above;   // among the prompts with a tile x
  int b = 0;
  for (; p.b0 < a.B; p.b0 += 32) {
    const bool in = tiles(p.b0) > p.x;
    const unsigned mask = __ballot_sync(0xffffffffu, in);
    const uint32_t n = __popc(mask);
    if (rank < p.before + n) {
      const bool me = in && p.before + __popc(mask & ((1u << lane) - 1)) == rank;
      b = p.b0 + __ffs(__ballot_sync(0xffffffffu, me)) - 1;
      break;
    }
    p.before += n;
  }
  it.q0 = __ldg(a.query_start + b);
  it.n = __ldg(a.query_start + b + 1) - it.q0;
  it.kvh = (int)(L - i * a.Hkv);
  it.row0 = p.x * kPaItemRows;
  return true;
}

// Rows, keys and chunks of tile t of an item (rows 0: the prompt ends before it).
struct PaTile {
  int rows, kend, chunks;
};
__device__ __forceinline__ PaTile pa_tile(const PaItem& it, int g2, int t) {   // g2 = log2(G)
  PaTile p;
  const int first = it.row0 + t * kPaRows;
  p.rows = min(kPaRows, (it.n << g2) - first);
  if (p.rows <= 0) {
    p.rows = p.kend = p.chunks = 0;
  } else {
    p.kend = ((first + p.rows - 1) >> g2) + 1;
    p.chunks = (p.kend + kPaKeys - 1) / kPaKeys;
  }
  return p;
}

template <typename T, int D>
__global__ void __launch_bounds__(kPaThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap tm_q,
                            const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v,
                            const __grid_constant__ CUtensorMap tm_o, const PromptArgs a) {
  using C = PaCfg<D>;
  constexpr int SK = C::kKStages, SV = C::kVStages;
  extern __shared__ unsigned char pa_smem_raw[];
  __shared__ __align__(8) uint64_t k_full[SK], k_free[SK], v_full[SV], v_free[SV],
      q_full[kPaTiles], q_free[kPaTiles], s_full[kPaTiles][2], p_full[kPaTiles][2], o_done[kPaTiles][2],
      v_tail, item_full[kPaItems], item_free[kPaItems], drained[2 * kPaTiles];
  __shared__ int4 items[kPaItems];   // (first token, tokens, KV head, first row); tokens 0: the end
  __shared__ uint32_t tmem_slot;
  __shared__ int gave_up_word;
  volatile int* gave_up = &gave_up_word;
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(pa_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sQ = smem_addr(smem), sK = sQ + C::kOffK, sV = sQ + C::kOffV;
  // uniform() tells the compiler that a value is the same in all lanes, so that
  // what the products take (descriptors, addresses) is kept and computed in
  // uniform registers
  auto uniform = [](uint32_t x) -> uint32_t { return __shfl_sync(0xffffffffu, x, 0); };
  const int tid = threadIdx.x, warp = (int)uniform(tid >> 5), lane = tid & 31;
  const int G = a.Hq / a.Hkv, g2 = __ffs(G) - 1;   // a power of two

  if (tid == 0) {
    gave_up_word = 0;
    for (int i = 0; i < SK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_free[i], kPaTiles);
    }
    for (int i = 0; i < SV; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_free[i], kPaTiles);
    }
    for (int t = 0; t < kPaTiles; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_free[t], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&s_full[t][h], 1);
        mbar_init(&p_full[t][h], 4);   // one arrival per softmax warp
        mbar_init(&o_done[t][h], 1);
      }
    }
    mbar_init(&v_tail, 1);
    for (int i = 0; i < 2 * kPaTiles; ++i) mbar_init(&drained[i], 1);
    for (int i = 0; i < kPaItems; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_free[i], kPaRoles);
    }
    mbar_init_fence();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 32 * 8) {
    prefetch_tensor_map(&tm_q);
    prefetch_tensor_map(&tm_k);
  }
  if (tid == 32 * 9) prefetch_tensor_map(&tm_v);
  pdl_launch_dependents();
  pdl_wait_primary();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(tmem_slot);

  if (blockIdx.x == 0 && warp == 0) {
    // rejected prompts
    for (int b = lane; b < a.B; b += 32) {
      const int q0 = __ldg(a.query_start + b), q1 = __ldg(a.query_start + b + 1);
      if (q0 < 0 || q1 < q0 || q1 > a.num_tokens || q1 - q0 > a.max_query_len)
        raise_error(a.err, kErrQuery);
    }
  }
  bool ok = true;
  PaItem it;
  // the CTA's m-th item, from the warp that finds them; false past the last one
  auto take = [&](uint32_t m, PaItem& to) -> bool {
    const int slot = m % kPaItems;
    ok = pa_wait(&item_full[slot], (m / kPaItems) & 1, gave_up);
    if (!ok) return false;
    const int4 v = items[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_free[slot]);
    to.q0 = v.x;
    to.n = v.y;
    to.kvh = v.z;
    to.row0 = v.w;
    return to.n > 0;
  };
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPaSoftmaxRegs));
    // ================================================================ softmax rows
    const int t = warp >> 2;
    const int trow = (warp & 3) * 32 + lane;   // row inside the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_base + t * kPaKeys;
    const uint32_t t_o = tmem + lane_base + kPaTmemO + t * D;
    unsigned char* stage = smem + C::kOffO + warp * 4096;
    const float qscale = a.qscale;
    // a zero scale as a tiny one: every weight is 1 and -inf stays -inf
    const float qmul = fmaxf(fabsf(qscale), 1e-37f);
    uint32_t done = 0;                                // chunks of this tile so far
    PaItem next;
    bool have = take(0, next);
    for (uint32_t m = 1; ok && have; ++m) {
      it = next;
      const PaTile mine = pa_tile(it, g2, t);
      if (mine.rows == 0) {
        have = take(m, next);
        continue;
      }
      const int first_row = it.row0 + t * kPaRows;
      const int my_pos = (first_row + min(trow, mine.rows - 1)) >> g2;
      const int warp_row = (warp & 3) * 32;
      const int pos_min = (first_row + min(warp_row, mine.rows - 1)) >> g2;
      const int pos_max = (first_row + min(warp_row + 31, mine.rows - 1)) >> g2;
      float m_run = kPaNoMax, l_run = 0.f;   // running maximum, unscaled; sum of weights
      float qm = qmul, base = 0.f;
      for (int c = 0; c < mine.chunks; ++c, ++done) {
        const int key0 = c * kPaKeys;
        const bool second = key0 + kPaHalf <= pos_max;   // a row of the warp sees the second half
        // Half a chunk at a time: scores, maximum, weights.  One instance of
        // the code (unrolled twice it no longer stays in the instruction
        // cache, and the rarely taken masks then cost thousands of clocks).
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          ok = pa_wait(&s_full[t][half], done & 1, gave_up);
          if (!ok) break;
          tc_fence_after();
          const uint32_t t_h = t_s + kPaHalf * half;
          if (half == 0 || second) {
            const int k0 = key0 + kPaHalf * half;
            float s[64];
            tmem_ld64(t_h, s);
            if (k0 + kPaHalf - 1 > pos_min) {
              const int lim = my_pos - k0;   // the row's last key of these
#pragma unroll
              for (int j = 0; j < 64; ++j) s[j] = j > lim ? -INFINITY : s[j];
            }
            float m8[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) m8[k] = fmaxf(s[k], s[8 + k]);
#pragma unroll
            for (int j = 16; j < 64; j += 16)
#pragma unroll
              for (int k = 0; k < 8; ++k) m8[k] = fmax3(m8[k], s[j + k], s[j + 8 + k]);
            const float mx = fmaxf(fmax3(m8[0], m8[1], m8[2]),
                                   fmax3(fmaxf(m8[3], m8[4]), fmaxf(m8[5], m8[6]), m8[7]));
            // The running maximum only moves when a score passes it by more
            // than 2^8, and only then is O rescaled: weights stay below 2^8
            // times the lift, and the stale maximum cancels in O / l.
            const bool moved = (mx - m_run) * qmul > kPaRescaleLog2;
            if (__any_sync(0xffffffffu, moved)) {
              const float corr = moved ? softmax_exp2((m_run - mx) * qmul) : 1.f;   // of nothing, at first
              l_run *= corr;
              if (moved) {
                m_run = mx;
                qm = fabsf(qmul * mx) < kPaFar ? qmul : __uint_as_float(__float_as_uint(qmul) & 0x7f800000u);
                base = __fmaf_rd(-qm, mx, kPaLift<T>);   // lifted no further, however large
              }
              if (c > 0 || half > 0) {
                // the product of the half before still adds to O
                ok = pa_wait(&o_done[t][1 - half], (half ? done : done - 1) & 1, gave_up);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int col = 0; col < D; col += 32) {
                  float o[32];
                  tmem_ld32(t_o + col, o);
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] *= corr;
                  tmem_st32(t_o + col, o);
                }
              }
            }
            // weights as 16-bit pairs, over scores that are read
            float w[32], sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              float x0, x1;
              fma_f32x2(x0, x1, s[2 * j], s[2 * j + 1], qm, base);
              const float p0 = softmax_exp2(x0), p1 = softmax_exp2(x1);
              add_f32x2(sum[(j & 1) * 2], sum[(j & 1) * 2 + 1], p0, p1);
              w[j] = __uint_as_float(Mma<T>::pack(p0, p1));
            }
            tmem_st32(t_h, w);
            l_run += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          } else if (mine.kend - key0 > kPaHalf) {   // another warp's rows see keys there
            float zero[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) zero[j] = 0.f;
            tmem_st32(t_h, zero);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[t][half]);
        }
        if (!ok) break;
      }
      if (!ok) break;
      have = take(m, next);   // while the last product runs
      if (!ok) break;
      // ---- O / l
      ok = pa_wait(&o_done[t][1], (done - 1) & 1, gave_up);
      if (!ok) break;
      tc_fence_after();
      // Through shared memory in the copies' swizzled layout.  A warp whose 32
      // rows all belong to the prompt hands them to tensor copies, which run
      // on while the next item begins; at a prompt's end 4 lanes write 64
      // bytes of a row (rows past it belong to others).  32 columns a turn:
      // the loop is short enough that its code is fetched once, and a buffer
      // is filled while the other one's copy reads.
      const float inv = 1.f / l_run;
      const bool whole = warp_row + 32 <= mine.rows;
      T* dst = static_cast<T*>(a.out) + (int64_t)it.q0 * a.out_stride + (int64_t)it.kvh * G * D;
#pragma unroll 1
      for (int col = 0; col < D; col += 32) {
        // 32 rows x 32 elements in one of the warp's two buffers
        float o[32];
        tmem_ld32(t_o + col, o);
        unsigned char* buf = stage + (col & 32) * 64;
        if (lane == 0) {   // the buffer's last copy has read it
          if (whole)
            bulk_store_wait_read<1>();
          else
            bulk_store_wait_read<0>();   // no copies of this item's to count
        }
        __syncwarp();
#pragma unroll
        for (int ch = 0; ch < 4; ++ch)
          *reinterpret_cast<uint4*>(buf + lane * 64 + ((ch ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(Mma<T>::pack(o[ch * 8] * inv, o[ch * 8 + 1] * inv),
                         Mma<T>::pack(o[ch * 8 + 2] * inv, o[ch * 8 + 3] * inv),
                         Mma<T>::pack(o[ch * 8 + 4] * inv, o[ch * 8 + 5] * inv),
                         Mma<T>::pack(o[ch * 8 + 6] * inv, o[ch * 8 + 7] * inv));
        if (whole) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0)
            tma_store_box3(&tm_o, col, it.kvh * G, it.q0 + ((first_row + warp_row) >> g2),
                           smem_addr(buf));
        } else {
          __syncwarp();
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2), ch = lane & 3;
            const uint4 v =
                *reinterpret_cast<const uint4*>(buf + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
            const int row = first_row + warp_row + r;
            if (warp_row + r < mine.rows)
              *reinterpret_cast<uint4*>(dst + (int64_t)(row >> g2) * a.out_stride +
                                        (row & (G - 1)) * D + col + ch * 8) = v;
          }
          __syncwarp();
        }
      }
      tc_fence_before();   // O is read before the next item's products (p_full orders them)
    }
    if (lane == 0) bulk_store_wait_read<0>();   // before the CTA's shared memory goes
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPaOtherRegs));
    if (warp == 8) {
      // ================================================================ Q and K copies
      uint32_t kc = 0;                      // chunks so far
      uint32_t q_count[kPaTiles] = {0, 0};   // Q tiles asked for so far
      for (uint32_t m = 0; ok && take(m, it); ++m) {
        const PaTile t0 = pa_tile(it, g2, 0), t1 = pa_tile(it, g2, 1);
        const int chunks = max(t0.chunks, t1.chunks);
        for (int c = 0; c < chunks && ok; ++c, ++kc) {
          const int st = kc % SK;
          if (kc >= SK) ok = pa_wait(&k_free[st], ((kc / SK) - 1) & 1, gave_up);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&k_full[st], C::kKvBytes);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_box(sK + st * C::kKvBytes + h * (kPaKeys * 128), &tm_k, it.kvh * D + h * 64,
                           it.q0 + c * kPaKeys, &k_full[st]);
          }
          __syncwarp();
          if (c > 0) continue;
          // the Q tiles, after the first chunk is on its way
          for (int t = 0; t < kPaTiles && ok; ++t) {
            if (m > 0) ok = pa_wait(&q_free[t], (m - 1) & 1, gave_up);
            if (!ok) break;
            ++q_count[t];
            if (lane != 0) continue;
            if ((t == 0 ? t0.rows : t1.rows) == 0) {
              mbar_arrive(&q_full[t]);
              continue;
            }
            mbar_arrive_expect_tx(&q_full[t], C::kQBytes);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_box3(sQ + t * C::kQBytes + h * (kPaRows * 128), &tm_q, h * 64, it.kvh * G,
                            it.q0 + ((it.row0 + t * kPaRows) >> g2), &q_full[t]);
          }
          __syncwarp();
        }
      }
      if (!ok) {
        // what is in flight lands before the CTA ends
        for (uint32_t c = kc > SK ? kc - SK : 0; c < kc; ++c)
          (void)mbar_wait_bounded(&k_full[c % SK], (c / SK) & 1);
        for (int t = 0; t < kPaTiles; ++t)
          if (q_count[t] > 0) (void)mbar_wait_bounded(&q_full[t], (q_count[t] - 1) & 1);
      }
    } else if (warp == 9) {
      // ================================================================ V copies
      uint32_t vc = 0, tails = 0;
      for (uint32_t m = 0; ok && take(m, it); ++m) {
        const PaTile t0 = pa_tile(it, g2, 0), t1 = pa_tile(it, g2, 1);
        const int chunks = max(t0.chunks, t1.chunks), kend = max(t0.kend, t1.kend);
        for (int c = 0; c < chunks && ok; ++c, ++vc) {
          const int st = vc % SV;
          if (vc >= SV) ok = pa_wait(&v_free[st], ((vc / SV) - 1) & 1, gave_up);
          if (!ok) break;
          // The products read whole groups of 16 keys.  Rows past the last key
          // meet zero weights, but 0 x NaN would not vanish: the last chunk
          // lands on a barrier of its own and its group is filled up with zeros
          // before the stage is handed over.
          const int valid = min(kPaKeys, kend - c * kPaKeys);
          const bool fill = valid % 16 != 0;
          uint64_t* land = fill ? &v_tail : &v_full[st];
          if (lane == 0) {
            mbar_arrive_expect_tx(land, C::kKvBytes);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_box(sV + st * C::kKvBytes + h * (kPaKeys * 128), &tm_v, it.kvh * D + h * 64,
                           it.q0 + c * kPaKeys, land);
          }
          __syncwarp();
          if (fill) {
            ok = pa_wait(&v_tail, tails & 1, gave_up);
            if (!ok) {
              (void)mbar_wait_bounded(&v_tail, tails & 1);   // its copy, in flight
              break;
            }
            ++tails;
            unsigned char* rows = smem + C::kOffV + st * C::kKvBytes;
            for (int i = lane; i < (16 - valid % 16) * (D / 8); i += 32) {
              const int r = valid + i / (D / 8), ch = i % (D / 8);
              *reinterpret_cast<uint4*>(rows + (ch >> 3) * (kPaKeys * 128) + r * 128 +
                                        (((ch & 7) ^ (r & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_full[st]);
          }
        }
      }
      if (!ok) {
        for (uint32_t c = vc > SV ? vc - SV : 0; c < vc; ++c)
          (void)mbar_wait_bounded(&v_full[c % SV], (c / SV) & 1);
      }
    } else if (warp == 14) {
      // ================================================================ items
      const int first = pa_tiles_of(a, G, lane);
      PaFinder finder = pa_finder(a, G, first, lane);
      const uint32_t N = gridDim.x;
      for (uint32_t m = 0, run = 0;; ++m, run += N) {
        const int slot = m % kPaItems;
        if (m >= kPaItems) ok = pa_wait(&item_free[slot], ((m / kPaItems) - 1) & 1, gave_up);
        if (!ok) break;
        // one item from each run of N, forwards and backwards in turn
        const bool found =
            pa_locate(a, G, run + (m & 1 ? N - 1 - blockIdx.x : blockIdx.x), first, lane, finder, it);
        if (lane == 0) {
          items[slot] = found ? make_int4(it.q0, it.n, it.kvh, it.row0) : make_int4(0, 0, 0, 0);
          mbar_arrive(&item_full[slot]);
        }
        __syncwarp();
        if (!found) break;
      }
    } else if (warp >= 10 && warp < 14) {
      // ================================================================ products
      // Per tile one warp issues S and one P V: an issuing warp is held up for
      // hundreds of clocks by each of its commits, so the two streams are kept
      // apart and commit nothing that another barrier already tells (a K stage
      // goes back once S is seen, a V stage once O is, by plain arrivals).
      const int t = (warp - 10) & 1;
      const uint32_t t_s = tmem + t * kPaKeys, t_o = tmem + kPaTmemO + t * D;
      // a descriptor's start address is address >> 4 in its low 14 bits; every
      // operand lies below 256 KB, so offsets are added to the base's descriptor
      uint32_t chunk0 = 0, done = 0;   // the item's first chunk; chunks of this tile so far
      const bool leader = elect_one();
      if (warp < 12) {
        // with a negative scale the product is negated (A's sign bit of the
        // descriptor), so that the maximum is always the largest score
        const uint32_t id_s = f16_idesc<T>(kPaRows, kPaHalf) | (a.qscale < 0.f ? 1u << 13 : 0u);
        const uint64_t q_desc = sw128_desc(sQ + t * C::kQBytes), k_desc = sw128_desc(sK);
        for (uint32_t m = 0; ok && take(m, it); ++m) {
          const PaTile mine = pa_tile(it, g2, t), other = pa_tile(it, g2, 1 - t);
          const int chunks = max(mine.chunks, other.chunks);
          ok = pa_wait(&q_full[t], m & 1, gave_up);
          if (!ok) break;
          if (mine.chunks == 0 && lane == 0) mbar_arrive(&q_free[t]);
          for (int c = 0; c < chunks; ++c) {
            const uint32_t kc = chunk0 + c;
            ok = pa_wait(&k_full[kc % SK], (kc / SK) & 1, gave_up);
            if (ok && c < mine.chunks) {
              const uint64_t kb = k_desc + (uint64_t)(((kc % SK) * C::kKvBytes) >> 4);
              for (int h = 0; h < 2; ++h) {
                // P of the last chunk's half, which lies over S, is used
                if (done > 0) ok = pa_wait(&o_done[t][h], (done - 1) & 1, gave_up);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                  for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t at = (kk & 3) * 32;
                    tc_mma(t_s + h * kPaHalf,
                           q_desc + (uint64_t)(((kk >> 2) * (kPaRows * 128) + at) >> 4),
                           kb + (uint64_t)(((kk >> 2) * (kPaKeys * 128) + h * (kPaHalf * 128) + at) >> 4),
                           id_s, kk > 0);
                  }
                  tc_commit(&s_full[t][h]);
                  if (h == 1 && c + 1 == mine.chunks) tc_commit(&q_free[t]);
                }
                __syncwarp();
              }
              if (!ok) break;
              ++done;
              ok = pa_wait(&s_full[t][1], (done - 1) & 1, gave_up);
            }
            if (!ok) break;
            if (lane == 0) mbar_arrive(&k_free[kc % SK]);
          }
          chunk0 = uniform(chunk0 + chunks);
        }
      } else {
        const uint32_t id_o = f16_idesc<T>(kPaRows, D) | (1u << 16);   // B (V) MN-major
        const uint64_t v_desc = pa_v_desc(sV);
        constexpr uint32_t kNothing = ~0u;
        uint32_t held = kNothing;   // the chunk whose V stage is to be handed back
        for (uint32_t m = 0; ok && take(m, it); ++m) {
          const PaTile mine = pa_tile(it, g2, t), other = pa_tile(it, g2, 1 - t);
          const int chunks = max(mine.chunks, other.chunks);
          for (int c = 0; c < chunks; ++c) {
            const uint32_t vc = chunk0 + c;
            if (held != kNothing) {
              ok = pa_wait(&o_done[t][1], (done - 1) & 1, gave_up);
              if (!ok) break;
              if (lane == 0) mbar_arrive(&v_free[held % SV]);
              held = kNothing;
            }
            ok = pa_wait(&v_full[vc % SV], (vc / SV) & 1, gave_up);
            if (!ok) break;
            if (c >= mine.chunks) {   // a chunk of the other tile only
              if (lane == 0) mbar_arrive(&v_free[vc % SV]);
              continue;
            }
            const uint64_t vb = v_desc + (uint64_t)(((vc % SV) * C::kKvBytes) >> 4);
            const int steps = (min(kPaKeys, mine.kend - c * kPaKeys) + 15) / 16;
            // 64 keys at a time, as their weights become ready; a half without
            // keys has nothing to add, only its barrier to complete
            for (int h = 0; h < 2; ++h) {
              ok = pa_wait(&p_full[t][h], done & 1, gave_up);
              if (!ok) break;
              tc_fence_after();
              auto product = [&](int kk) {
                tc_mma_ts(t_o, t_s + h * kPaHalf + kk * 8,
                          vb + (uint64_t)((h * (kPaHalf * 128) + kk * 2048) >> 4), id_o,
                          c > 0 || h > 0 || kk > 0 ? 1u : 0u);
              };
              if (leader) {
                if (steps >= 4 * h + 4) {
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk) product(kk);
                } else {
#pragma unroll 1
                  for (int kk = 0; kk < steps - 4 * h; ++kk) product(kk);
                }
                tc_commit(&o_done[t][h]);
              }
              __syncwarp();
            }
            if (!ok) break;
            held = vc;
            ++done;
          }
          chunk0 = uniform(chunk0 + chunks);
        }
      }
      if (!ok) {
        if (leader) tc_commit(&drained[warp - 10]);
        __syncwarp();
        (void)mbar_wait_bounded(&drained[warp - 10], 0);
      }
    }
  }
  if (!ok && lane == 0) raise_error(a.err, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
}

template <typename T, int D>
cudaError_t launch_t(const PromptArgs& a, cudaStream_t stream) {
  using C = PaCfg<D>;
  auto kern = prompt_attention_kernel<T, D>;
  static std::atomic<bool> configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    configured[dev].store(true, std::memory_order_relaxed);
  }
  const CUtensorMapDataType type =
      a.dtype == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint64_t T_ = (cuuint64_t)a.num_tokens;
  const cuuint32_t G = (cuuint32_t)(a.Hq / a.Hkv);
  CUtensorMap tq, tk, tv, to;
  // q as [token][head][element], a box of 128 / G tokens x G heads x 64 elements
  const cuuint64_t qd[3] = {(cuuint64_t)D, (cuuint64_t)a.Hq, T_};
  const cuuint64_t qs[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.q_stride * 2};
  const cuuint32_t qb[3] = {64, G, (cuuint32_t)kPaRows / G};
  e = encode_tensor_map(&tq, type, 3, a.q, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  // k and v as [token][head and element], boxes of 128 tokens x 64 elements
  const cuuint64_t kd[2] = {(cuuint64_t)a.Hkv * D, T_};
  const cuuint32_t kb[2] = {64, kPaKeys};
  const cuuint64_t ks[1] = {(cuuint64_t)a.k_stride * 2}, vs[1] = {(cuuint64_t)a.v_stride * 2};
  e = encode_tensor_map(&tk, type, 2, a.k, kd, ks, kb, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  e = encode_tensor_map(&tv, type, 2, a.v, kd, vs, kb, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  // out as q, a box of a warp's 32 rows
  const cuuint64_t os[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.out_stride * 2};
  const cuuint32_t ob[3] = {32, G, 32u / G};
  e = encode_tensor_map(&to, type, 3, a.out, qd, os, ob, CU_TENSOR_MAP_SWIZZLE_64B);
  if (e != cudaSuccess) return e;
  // at most this many items exist
  const int64_t most = ((int64_t)a.num_tokens * (int)G / kPaItemRows + a.B) * a.Hkv;
  if (most > INT32_MAX) return cudaErrorInvalidValue;
  const int grid = (int)std::min<int64_t>(a.num_sms, most);
  return launch_pdl(kern, dim3(grid), dim3(kPaThreads), C::kSmem, stream, tq, tk, tv, to, a);
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t stream) {
  if (a.dtype == 1)
    return a.D == 64 ? launch_t<__half, 64>(a, stream) : launch_t<__half, 128>(a, stream);
  return a.D == 64 ? launch_t<__nv_bfloat16, 64>(a, stream)
                   : launch_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace photon
