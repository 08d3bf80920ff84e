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
// bound it, with the exponentials close behind (16384 of them per 128 x 128
// tile at 16 a clock take about as long as the tile's two products).
//
// A persistent CTA per SM takes items of 256 query rows of one (prompt, KV
// head) -- row r is (token r / G, head r % G), so one K/V chunk serves the
// whole group -- as two tiles of 128 rows, and runs 12 warps in fixed roles:
//   warps 0-3, 4-7  softmax of tile 0, 1: thread r owns TMEM lane r
//   warp 8, 9       tensor-map copies of Q and K, of V (128-byte swizzle)
//   warp 10, 11     issue the products of tile 0, 1
// The two tiles run in antiphase: while one's softmax is on, the other's
// products are.  Per tile, TMEM holds S (128 columns) and O (D columns); P
// overwrites the second half of S as 16-bit pairs and is read from there as
// the A operand.  S products have N = 128 keys: with N = 64 the operand reads of Q
// from shared memory hold the tensor cores to two thirds of their rate.
// Copies run ahead across items, and the next item's first S product overlaps
// this one's epilogue.
//
// Items are numbered tile by tile from the prompts' far ends (the longest key
// ranges) to their beginnings, and dealt to the CTAs forwards and backwards in
// turn, so that all finish close together; every warp finds its next item from
// the lengths alone (pa_locate), without a queue.
//
// Barriers complete once per use; use i has parity i & 1:
//   k_full, v_full[st]   a chunk landed      k_free, v_free[st]  both tiles are done with it
//   q_full[t]            Q tile landed       q_free[t]           the item's last S product is done
//   s_full[t]            S written           p_full[t]           P written, S read
//   o_done[t]            O += P V done; the tile's next S may overwrite P
#include <math.h>

#include <algorithm>

#include "prompt_attention.cuh"
#include "tc_common.cuh"

namespace photon {
namespace {

constexpr int kPaRows = 128;            // query rows of a tile = TMEM lanes
constexpr int kPaKeys = 128;            // keys of a chunk
constexpr int kPaTiles = 2;
constexpr int kPaItemRows = kPaTiles * kPaRows;
constexpr int kPaThreads = 384;
constexpr uint32_t kPaTmemP = 64;       // P of a tile: the second half of its S columns
constexpr uint32_t kPaTmemO = 256;      // S of tile t: columns [128 t, 128 t + 128); then the O's
constexpr float kPaRescaleLog2 = 8.f;

template <int D>
struct PaCfg {
  static constexpr int kKStages = 3;
  static constexpr int kVStages = D == 128 ? 2 : 3;
  static constexpr int kQBytes = kPaRows * D * 2;
  static constexpr int kKvBytes = kPaKeys * D * 2;
  static constexpr int kOffK = kPaTiles * kQBytes;
  static constexpr int kOffV = kOffK + kKStages * kKvBytes;
  static constexpr int kSmem = kOffV + kVStages * kKvBytes + 1024;   // + alignment to a swizzle atom
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

// The L-th item, by a whole warp; false past the last one.  Item L is KV head
// L % Hkv of the (L / Hkv)-th (prompt, tile), taken from the highest tile
// index of any prompt down, prompts in order within one index.  F(x), the
// number of (prompt, tile) with tile index >= x, falls with x: the tile index
// is the largest x with F(x) > L / Hkv.  `first` holds pa_tiles_of(lane).
__device__ __forceinline__ bool pa_locate(const PromptArgs& a, int G, long long L, int first,
                                          int lane, PaItem& it) {
  auto tiles = [&](int b0) { return b0 == 0 ? first : pa_tiles_of(a, G, b0 + lane); };
  auto above = [&](int x) -> int {   // F(x)
    int s = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) s += max(0, tiles(b0) - x);
    return (int)__reduce_add_sync(0xffffffffu, (unsigned)s);
  };
  const long long i = L / a.Hkv;
  if (i >= above(0)) return false;
  int lo = 0, hi = (a.max_query_len * G + kPaItemRows - 1) / kPaItemRows, f_hi = 0;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2, f = above(mid);
    if (f > i) {
      lo = mid;
    } else {
      hi = mid;
      f_hi = f;
    }
  }
  int r = (int)i - f_hi, b = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const bool in = tiles(b0) > lo;
    const unsigned mask = __ballot_sync(0xffffffffu, in);
    const int c = __popc(mask);
    if (r < c) {
      const bool me = in && __popc(mask & ((1u << lane) - 1)) == r;
      b = b0 + __ffs(__ballot_sync(0xffffffffu, me)) - 1;
      break;
    }
    r -= c;
  }
  it.q0 = __ldg(a.query_start + b);
  it.n = __ldg(a.query_start + b + 1) - it.q0;
  it.kvh = (int)(L % a.Hkv);
  it.row0 = lo * kPaItemRows;
  return true;
}

// Rows, keys and chunks of tile t of an item (rows 0: the prompt ends before it).
struct PaTile {
  int rows, kend, chunks;
};
__device__ __forceinline__ PaTile pa_tile(const PaItem& it, int G, int t) {
  PaTile p;
  const int first = it.row0 + t * kPaRows;
  p.rows = min(kPaRows, it.n * G - first);
  if (p.rows <= 0) {
    p.rows = p.kend = p.chunks = 0;
  } else {
    p.kend = (first + p.rows - 1) / G + 1;
    p.chunks = (p.kend + kPaKeys - 1) / kPaKeys;
  }
  return p;
}

template <typename T, int D>
__global__ void __launch_bounds__(kPaThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap tm_q,
                            const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const PromptArgs a) {
  using C = PaCfg<D>;
  constexpr int SK = C::kKStages, SV = C::kVStages;
  extern __shared__ unsigned char pa_smem_raw[];
  __shared__ __align__(8) uint64_t k_full[SK], k_free[SK], v_full[SV], v_free[SV],
      q_full[kPaTiles], q_free[kPaTiles], s_full[kPaTiles], p_full[kPaTiles], o_done[kPaTiles],
      v_tail;
  __shared__ uint32_t tmem_slot;
  __shared__ int gave_up_word;
  volatile int* gave_up = &gave_up_word;
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(pa_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sQ = smem_addr(smem), sK = sQ + C::kOffK, sV = sQ + C::kOffV;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;

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
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);   // one arrival per softmax warp
      mbar_init(&o_done[t], 1);
    }
    mbar_init(&v_tail, 1);
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
  const uint32_t tmem = tmem_slot;

  if (blockIdx.x == 0 && warp == 0) {
    // rejected prompts
    for (int b = lane; b < a.B; b += 32) {
      const int q0 = __ldg(a.query_start + b), q1 = __ldg(a.query_start + b + 1);
      if (q0 < 0 || q1 < q0 || q1 > a.num_tokens || q1 - q0 > a.max_query_len)
        raise_error(a.err, kErrQuery);
    }
  }
  const int first = pa_tiles_of(a, G, lane);
  const long long N = gridDim.x;
  // the CTA's items: one from each run of N, forwards and backwards in turn
  auto item_of = [&](long long round) -> long long {
    return round * N + (round & 1 ? N - 1 - blockIdx.x : blockIdx.x);
  };
  bool ok = true;
  PaItem it;

  if (warp == 8) {
    // ================================================================ Q and K copies
    uint32_t kc = 0;                      // chunks so far
    uint32_t q_count[kPaTiles] = {0, 0};   // Q tiles asked for so far
    for (long long m = 0; ok && pa_locate(a, G, item_of(m), first, lane, it); ++m) {
      const PaTile t0 = pa_tile(it, G, 0), t1 = pa_tile(it, G, 1);
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
                          it.q0 + (it.row0 + t * kPaRows) / G, &q_full[t]);
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
    for (long long m = 0; ok && pa_locate(a, G, item_of(m), first, lane, it); ++m) {
      const PaTile t0 = pa_tile(it, G, 0), t1 = pa_tile(it, G, 1);
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
          ++tails;
          if (!ok) break;
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
  } else if (warp >= 10) {
    // ================================================================ products
    const int t = warp - 10;
    const uint32_t id_s = f16_idesc<T>(kPaRows, kPaKeys);
    const uint32_t id_o = f16_idesc<T>(kPaRows, D) | (1u << 16);   // B (V) MN-major
    // a descriptor's start address is address >> 4 in its low 14 bits; every
    // operand lies below 256 KB, so offsets are added to the base's descriptor
    const uint64_t q_desc = sw128_desc(sQ + t * C::kQBytes);
    const uint64_t k_desc = sw128_desc(sK), v_desc = pa_v_desc(sV);
    const uint32_t t_s = tmem + t * kPaKeys, t_o = tmem + kPaTmemO + t * D;
    uint32_t kc = 0, vc = 0, done = 0;   // K and V chunks so far; chunks of this tile
    for (long long m = 0; ok && pa_locate(a, G, item_of(m), first, lane, it); ++m) {
      const PaTile mine = pa_tile(it, G, t), other = pa_tile(it, G, 1 - t);
      const int chunks = max(mine.chunks, other.chunks);
      ok = pa_wait(&q_full[t], m & 1, gave_up);
      if (!ok) break;
      if (mine.chunks == 0 && lane == 0) mbar_arrive(&q_free[t]);
      for (int c = 0; c <= chunks; ++c) {
        if (c > 0) {
          // O += P V of chunk c - 1
          const int st = vc % SV;
          ok = pa_wait(&v_full[st], (vc / SV) & 1, gave_up);
          if (!ok) break;
          if (c - 1 < mine.chunks) {
            ok = pa_wait(&p_full[t], done & 1, gave_up);
            if (!ok) break;
            tc_fence_after();
            const int steps = (min(kPaKeys, mine.kend - (c - 1) * kPaKeys) + 15) / 16;
            const uint64_t vb = v_desc + (uint64_t)((st * C::kKvBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < kPaKeys / 16; ++kk)
              tc_mma_ts_warp(t_o, t_s + kPaTmemP + kk * 8, vb + (uint64_t)((kk * 2048) >> 4), id_o,
                             (c > 1 || kk > 0) ? 1u : 0u, lane == 0 && kk < steps);
            if (lane == 0) {
              tc_commit(&o_done[t]);
              tc_commit(&v_free[st]);
            }
            ++done;
          } else if (lane == 0) {
            mbar_arrive(&v_free[st]);
          }
          ++vc;
        }
        if (c < chunks) {
          // S = Q K^T of chunk c, over the P of the tile's previous chunk
          const int st = kc % SK;
          ok = pa_wait(&k_full[st], (kc / SK) & 1, gave_up);
          if (!ok) break;
          if (c < mine.chunks) {
            if (done > 0) ok = pa_wait(&o_done[t], (done - 1) & 1, gave_up);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kb = k_desc + (uint64_t)((st * C::kKvBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * (kPaKeys * 128) + (kk & 3) * 32;
              tc_mma_warp(t_s, q_desc + (uint64_t)(off >> 4), kb + (uint64_t)(off >> 4), id_s,
                          kk > 0, lane == 0);
            }
            if (lane == 0) {
              tc_commit(&s_full[t]);
              tc_commit(&k_free[st]);
              if (c + 1 == mine.chunks) tc_commit(&q_free[t]);
            }
          } else if (lane == 0) {
            mbar_arrive(&k_free[st]);
          }
          ++kc;
        }
      }
    }
  } else {
    // ================================================================ softmax rows
    const int t = warp >> 2;
    const int trow = (warp & 3) * 32 + lane;   // row inside the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_base + t * kPaKeys;
    const uint32_t t_o = tmem + lane_base + kPaTmemO + t * D;
    const float qscale = a.qscale;
    const float qmul = qscale > 0.f ? qscale : 1.f;   // multiplier left for the exponent
    uint32_t done = 0;                                // chunks of this tile so far
    for (long long m = 0; ok && pa_locate(a, G, item_of(m), first, lane, it); ++m) {
      const PaTile mine = pa_tile(it, G, t);
      if (mine.rows == 0) continue;
      const int first_row = it.row0 + t * kPaRows;
      const int my_pos = (first_row + min(trow, mine.rows - 1)) / G;
      const int warp_row = (warp & 3) * 32;
      const int pos_min = (first_row + min(warp_row, mine.rows - 1)) / G;
      const int pos_max = (first_row + min(warp_row + 31, mine.rows - 1)) / G;
      float m_run = -INFINITY, l_run = 0.f;
      for (int c = 0; c < mine.chunks; ++c, ++done) {
        ok = pa_wait(&s_full[t], done & 1, gave_up);
        if (!ok) break;
        tc_fence_after();
        const int key0 = c * kPaKeys;
        // scores of 64 of the chunk's keys, -inf where they lie past the row
        auto scores = [&](int half, float (&s)[64]) {
          tmem_ld64(t_s + 64 * half, s);
          const int k0 = key0 + 64 * half;
          if (k0 + 63 > pos_min) {
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (k0 + j > my_pos) s[j] = -INFINITY;
          }
          if (!(qscale > 0.f)) {
            // a negative (or zero) scale turns the order of the scores around
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (k0 + j <= my_pos) s[j] *= qscale;
          }
        };
        auto maximum = [&](const float (&s)[64]) -> float {
          float m8[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) m8[k] = fmaxf(s[k], s[8 + k]);
#pragma unroll
          for (int j = 16; j < 64; j += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k) m8[k] = fmax3(m8[k], s[j + k], s[j + 8 + k]);
          return fmaxf(fmax3(m8[0], m8[1], m8[2]),
                       fmax3(fmaxf(m8[3], m8[4]), fmaxf(m8[5], m8[6]), m8[7]));
        };
        // The second half's scores stay in registers while the maximum is
        // settled; the first half's are read again after them (128 scores a
        // thread would spill).  P takes the columns of the second half, so
        // what is still to be read is not overwritten.
        const bool second = key0 + 64 <= pos_max;   // a row of the warp sees keys there
        float s[64];
        scores(0, s);
        float mx = maximum(s);
        if (second) {
          scores(1, s);
          mx = fmaxf(mx, maximum(s));
        }
        mx *= qmul;
        // The running maximum only moves when a score passes it by more than
        // 2^8, and only then is O rescaled: weights stay below 2^8, and the
        // stale maximum cancels in O / l.
        const bool moved = mx > m_run + kPaRescaleLog2;
        const float corr = moved ? softmax_exp2(m_run - mx) : 1.f;   // 0 on the first chunk
        l_run *= corr;
        if (moved) m_run = mx;
        if (c > 0 && __any_sync(0xffffffffu, moved)) {
          // the product of chunk c - 1 still adds to O
          ok = pa_wait(&o_done[t], (done - 1) & 1, gave_up);
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
          tc_fence_before();
        }
        // weights, as 16-bit pairs
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        auto weights = [&](int half) {
          float w[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float x0, x1;
            fma_f32x2(x0, x1, s[2 * j], s[2 * j + 1], qmul, -m_run);
            const float p0 = softmax_exp2(x0), p1 = softmax_exp2(x1);
            add_f32x2(sum[(j & 1) * 2], sum[(j & 1) * 2 + 1], p0, p1);
            w[j] = __uint_as_float(Mma<T>::pack(p0, p1));
          }
          tmem_st32(t_s + kPaTmemP + 32 * half, w);
        };
        if (second) {
          weights(1);
          scores(0, s);
        } else {
          float zero[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) zero[j] = 0.f;
          tmem_st32(t_s + kPaTmemP + 32, zero);
        }
        weights(0);
        l_run += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      if (!ok) break;
      // ---- O / l
      ok = pa_wait(&o_done[t], (done - 1) & 1, gave_up);
      if (!ok) break;
      tc_fence_after();
      T* dst = static_cast<T*>(a.out) + (int64_t)(it.q0 + my_pos) * a.out_stride +
               (int64_t)(it.kvh * G + (first_row + trow) % G) * D;
      const float inv = 1.f / l_run;
#pragma unroll 1
      for (int col = 0; col < D; col += 32) {
        float o[32];
        tmem_ld32(t_o + col, o);   // warp-wide: every lane
        if (trow >= mine.rows) continue;
#pragma unroll
        for (int ch = 0; ch < 4; ++ch)
          *reinterpret_cast<uint4*>(dst + col + ch * 8) =
              make_uint4(Mma<T>::pack(o[ch * 8] * inv, o[ch * 8 + 1] * inv),
                         Mma<T>::pack(o[ch * 8 + 2] * inv, o[ch * 8 + 3] * inv),
                         Mma<T>::pack(o[ch * 8 + 4] * inv, o[ch * 8 + 5] * inv),
                         Mma<T>::pack(o[ch * 8 + 6] * inv, o[ch * 8 + 7] * inv));
      }
      tc_fence_before();   // O is read before the next item's products (p_full orders them)
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
  CUtensorMap tq, tk, tv;
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
  // at most this many items exist
  const int64_t most = ((int64_t)a.num_tokens * (int)G / kPaItemRows + a.B) * a.Hkv;
  const int grid = (int)std::min<int64_t>(a.num_sms, most);
  return launch_pdl(kern, dim3(grid), dim3(kPaThreads), C::kSmem, stream, tq, tk, tv, a);
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t stream) {
  if (a.dtype == 1)
    return a.D == 64 ? launch_t<__half, 64>(a, stream) : launch_t<__half, 128>(a, stream);
  return a.D == 64 ? launch_t<__nv_bfloat16, 64>(a, stream)
                   : launch_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace photon
