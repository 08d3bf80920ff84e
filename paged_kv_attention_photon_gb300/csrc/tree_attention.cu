// tree_attention.cu -- attention of each sequence's drafted tree over its paged
// cache, on the fifth-generation tensor cores.
//
// PhotonInfer README, "Technical details / Paged attention" (block-wise KV cache,
// per-sequence offsets); "Roadmap" (speculative decoding; FlashAttention-2 style
// attention for long sequences).
//
// Node i of a tree of n nodes, whose rows are the last n of a context, attends to
// the context before the tree, to its ancestors and to itself:
// out = sum_j softmax_j(scale q . k_j) v_j over those keys.  A row of K and V is
// read once for all n G query rows (node, head of the group) of its KV head: 2 n G
// flops a byte at 16 bits, so memory bounds it up to about 280 rows and the tensor
// cores above.  mma.sync would do for 8 rows or so (photon_paged_multi_query's
// few-token mode); from 16 on only tcgen05 keeps up with memory, and as memory
// bounds it the rows of a 128-row product that a small tree leaves empty cost nothing.
//
// A persistent CTA per SM takes runs of 128-key chunks of (sequence, KV head, group
// of 256 rows).  Two tiles of 128 rows each have scores S and sums O in tensor
// memory.  With more than 128 rows each tile has its own rows and sees every chunk;
// with up to 128 both tiles have the same rows and take every other chunk, so that
// one tile's softmax runs beside the other's products, and their sums meet at the end
// through shared memory, or, up to kOneTile chunks, one tile takes the item and the other
// the next one.  S, softmax and P V go by halves of 64 keys; P of a half lies over its S
// as 16-bit pairs.  16 warps in fixed roles:
//   warps 0-3, 4-7  softmax of tile 0, 1: thread r owns TMEM lane r
//   warp 8, 9       tensor-map copies of Q and K, of V: 16-row boxes through the table
//   warp 10, 11     issue S of tile 0, 1
//   warp 12, 13     issue P V of tile 0, 1
//   warp 14         finds the items
//   warp 15         finds the ancestors of each node; rejected sequences
//
// Which keys a node sees of its tree is a bit mask of its ancestors, found by
// doubling (node i takes its ancestor's mask and the ancestor's ancestor, until all
// have reached the root) when an item holds the tree's keys.  Only the chunks that
// hold some are masked, 64 bits a row and half.
//
// The chunks of all (sequence, KV head, group) triples lie on one line, each triple
// counting kTreePairCost more than it has for what beginning and ending it costs;
// the line is cut into equal runs, one per CTA: no queue and no atomics, so results
// do not depend on timing.  A triple within one run is written out at once, the
// others (one at most at each end of a run) leave partial sums, joined by a second
// kernel.
//
// Numerics: products of the stored values, sums and statistics in fp32; weights P
// enter the second product rounded to the storage type, as in
// photon_paged_multi_query and photon_prompt_attention: a product with their
// rounding errors besides would be half again as many.  fp16 weights are lifted to
// the upper end of fp16's range (kLift), so that what they lose lies below 2^-32 of
// the largest.  A zero weight times an infinity would not vanish: a CTA that ends with a row
// that is not finite goes through its items again, with what of the nodes' V is not finite
// kept out of the product and added to the rows that see it.  (Taken out always, and in a
// second pass: 128 contexts of 100 .. 400 tokens x 16 nodes, 16 q / 16 kv heads x 128, 96 and 88
// us, a batch-256 mix 190 and 187, 4 short contexts 11.5 and 11.6: the look at V lies between its
// copy and its product, and its code drives the softmax's out of the instruction cache, with
// four rows a turn in the mix 220.)
//
// Measured (event times of calls in a row): 64 contexts of 128 .. 8192 tokens x 16 nodes,
// 16 q / 8 kv heads x 128, fp16: 96 us = 5.5 TB/s, 81 % of the measured copy rate; a
// batch-256 mix x 1 .. 32 nodes, 32 / 8 x 64, bf16: 189 us, 82 %; 4 short contexts 12.0
// us.  In long contexts a chunk takes the time of its bytes: 1.51 us for 64 KB (d = 128,
// up to 128 rows), 0.75 us for 32 KB (d = 64, up to 64 rows; 0.80 with 128): 6.5 TB/s over
// all SMs.  With 256 rows at d = 64 it takes 1.38 us, the softmax's latency on two warps
// a scheduler: 32 contexts x 64 nodes 58 us.  A call begins and ends in 7.1 us (launch,
// lengths, table, first data), 8.2 with the join's launch, 11 where pairs are split; an
// item of its own costs 1.4 us (one tile's) to 2 or 3.  On the way there (64 contexts /
// the mix / 4 short ones / 32 x 64): the first right version 101 / 230 / 18.6 / 64 us; block
// ids a chunk ahead and not four 101 / 215 / 12.9 / 59; items of up to 4 chunks on both
// tiles, too, - / 229 / 12.3 / 60.
// Measured and left out: stages of 64 keys, twice as many (135 / 316 / 13.2 / 63); up to
// 64 rows in the upper lanes for tile 1, so that the two tiles' softmax warps are on
// different quarters of the SM (94 / 224 / 12.5 / 60); Q in both places for that (96 / 221).
//
// Barriers complete once per use; use i has parity i & 1:
//   k_full, v_full[st]   a chunk landed      k_free, v_free[st]  both tiles are done with it
//   q_full[i]            a Q tile landed     q_free[i]           the item's last S is done
//   s_full[t][h]         S of 64 keys        p_full[t][h]        their P written
//   o_done[t][h]         O += P V of 64 keys done; the next chunk's S may overwrite P
//   item_full, item_free[i]  an item is known; every role has read it
//   mask_full, mask_free     the ancestors of a tree's nodes; no softmax warp uses them any more
//   meet_full, meet_free[w]  32 columns of one tile's O are in shared memory; the other has taken them
// Where a wait runs out the CTA gives up, and what it has in flight still lands
// first: the copying warps wait (bounded) for their last copies, the issuing ones on
//   drained[i]           every product that the warp has issued is done
#include <math.h>

#include <algorithm>

#include "speculate.cuh"
#include "tc_common.cuh"

namespace photon {
namespace {

constexpr int kRows = 128;              // query rows of a tile = TMEM lanes
constexpr int kKeys = kTreeChunk;       // keys of a chunk
constexpr int kHalf = 64;               // keys of an S product, of a softmax step and of a P V product
constexpr int kChunkBlocks = kKeys / kBlockSize;
constexpr int kTiles = 2;
constexpr int kThreads = 512;           // four warpgroups
// Registers a thread: 512 x 128 at launch, dealt anew to the softmax warpgroups and
// the other two (160 + 160 + 96 + 96 = 4 x 128).
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 160, kOtherRegs = 96;
constexpr uint32_t kTmemO = 256;        // S of tile t: columns [128 t, 128 t + 128); then the O's
constexpr float kRescale = 8.f;         // the running maximum moves by 2^8 or not at all
// Weights are 2^(score - maximum + lift): see the top.
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 7.f : 0.f;
constexpr float kNoMax = -3e38f;        // before the first key; finite, so that no exponent is inf - inf
// From here on (2^23) fp32 scores are whole units of the exponent apart, and the
// scaled maximum, rounded, would move all weights by half a unit and more: the
// exponents then take the scale's power of two alone, which is exact.
constexpr float kFar = 8388608.f;
constexpr int kItems = 4;               // items found ahead
constexpr int kRoles = 15;              // warps that an item is told
constexpr int kMaskWords = kTreeNodes / 32, kMaskStride = kMaskWords + 1;
// Items of up to so many chunks (and 128 rows) go to one tile, the next one to the other,
// where a CTA has several (a.one_tile is 1 otherwise).  With 1, 2, 4, 6, 12: a batch-256
// mix 210, 200, 193, 194, 194 us, 152 x 1024 tokens (32 q, 8 kv heads x 64, 16 nodes) 73.7,
// 73.6, 73.9, 73.6, 78.7; 4 short contexts, an item a CTA, 11.7, 12.1, 12.2, 12.1, 12.1.
constexpr int kOneTile = 4;
// Where no context can have more than kWholePairs chunks, and whole pairs leave a CTA no
// more than kWholeIdle2 / 2 of their time unused on average, pairs are not split, and no
// second kernel joins them.  What contexts can have is the table's width, all that the host
// knows: with a table of more than 64 blocks pairs are split, however short the contexts are.
// Whole and split: 4 contexts of 300 tokens x 16 nodes (16 q, 8 kv heads x 128) 9.9, 11.9 us; 16
// of 1000 15.8, 22.2; 64 of 1000 (32 q, 8 kv heads x 64) 39.0, 40.7; but 24 of 1000 (192 pairs, a
// second round for 40 of them) 28.1, 25.9, 1 of 1000 13.8, 10.8, and 40 of 2000 72.8, 63.6.
constexpr int kWholePairs = 8, kWholeIdle2 = 11;
// Chunks whose missing blocks are remembered.  Softmax reads a chunk's entry when its S
// is done, which is not when its stage is handed back: until the softmax has gone on, its
// tile's issuer still passes over what the other tile takes, kOneTile + 1 chunks at most
// (the last one of an item on both tiles, and an item on one), and hands back those
// stages too.  So copies run ahead of the softmax by up to that and the stages.
constexpr int kGoneRing = 16;

template <int D>
struct Cfg {
  static constexpr int kKStages = D == 128 ? 2 : 4;
  static constexpr int kVStages = D == 128 ? 2 : 4;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kKvBytes = kKeys * D * 2;
  static constexpr int kOffK = kTiles * kQBytes;
  static constexpr int kOffV = kOffK + kKStages * kKvBytes;
  static constexpr int kOffMeet = kOffV + kVStages * kKvBytes;   // 4 warps x 32 columns x 32 rows
  static constexpr int kOffMask = kOffMeet + 4 * 4096;
  static constexpr int kSmem = kOffMask + kTreeNodes * kMaskStride * 4 + 1024;   // + alignment to a swizzle atom
  static_assert(kGoneRing > kKStages + kOneTile + 1, "the ring of K's missing blocks");
  static_assert(kGoneRing > kVStages, "V's are read before the stage is handed back");
};

// MN-major V operand (sw128_desc walked along N): 64-element blocks of N are kKeys
// rows of 128 bytes apart (leading offset), groups of 8 keys 1 KB.
__device__ __forceinline__ uint64_t v_operand(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)((kKeys * 128) >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// 8 elements with 0 in the place of infinities and NaN.
template <typename T>
__device__ __forceinline__ uint4 finite8(uint4 x) {
  auto two = [](uint32_t v) -> uint32_t {
    constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
    constexpr uint32_t kOne = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
    const uint32_t full = ((v & kExp) + kOne) & 0x80008000u;   // bits 15 and 31: all of an exponent is set
    return v & ~((full >> 15) * 0xffffu);
  };
  return make_uint4(two(x.x), two(x.y), two(x.z), two(x.w));
}
__device__ __forceinline__ void mbar_inval(uint64_t* bar) {
  asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// sum += 0 x: NaN from an infinity or NaN on.
__device__ __forceinline__ void add_zero_times(float2& sum, float x, float y) {
  asm("{\n.reg .b64 s, v, z;\nmov.b64 s, {%0, %1};\nmov.b64 v, {%2, %3};\nmov.b64 z, {%4, %4};\n"
      "fma.rn.f32x2 s, v, z, s;\nmov.b64 {%0, %1}, s;\n}"
      : "+f"(sum.x), "+f"(sum.y)
      : "f"(x), "f"(y), "f"(0.f));
}

// A sequence's tree and context; n == 0: empty or rejected.
struct Seq {
  int q0, n, ctx;
};
__device__ __forceinline__ Seq seq_of(const TreeArgs& a, int b) {
  Seq s{0, 0, 0};
  if (b >= a.B) return s;
  const int q0 = __ldg(a.query_start + b), q1 = __ldg(a.query_start + b + 1);
  const int ctx = __ldg(a.context_lens + b);
  if (q0 < 0 || q1 <= q0 || q1 > a.num_tokens || q1 - q0 > a.max_query_len || ctx < q1 - q0 ||
      ctx > a.MBS * kBlockSize)
    return s;
  s.q0 = q0;
  s.n = q1 - q0;
  s.ctx = ctx;
  return s;
}
__device__ __forceinline__ int chunks_of(int ctx) { return (ctx + kKeys - 1) / kKeys; }
__host__ __device__ __forceinline__ int groups_of(int n, int G) { return (n * G + kTreeRows - 1) / kTreeRows; }
// Units of a sequence on the line.
__device__ __forceinline__ int units_of(const TreeArgs& a, const Seq& s, int G) {
  return s.n == 0 ? 0 : a.Hkv * groups_of(s.n, G) * (chunks_of(s.ctx) + kTreePairCost);
}

// Chunks [c0, c1) of row group g of (sequence b, KV head kvh).
struct Item {
  int b, kvh, g, c0;
  int c1, q0, n, ctx;
  int place;   // where the sums go: 0 out, 1 the rows' own partials, 2 the CTA's
  int tree;    // which of the trees' masks it needs, counted up; -1: holds no key of a tree
  int one_tile;
  __device__ __forceinline__ int rows(int g2) const { return min(kTreeRows, (n << g2) - g * kTreeRows); }
  __device__ __forceinline__ int chunks() const { return c1 - c0; }
  // both tiles have rows of their own
  __device__ __forceinline__ bool apart(int g2) const { return rows(g2) > kRows; }
  // both tiles have the same rows, and every other chunk each
  __device__ __forceinline__ bool shared(int g2) const { return !apart(g2) && chunks() > one_tile; }
  // the place of tile t's Q: items of one tile's rows take the two places in turn
  __device__ __forceinline__ int place_of(int g2, uint32_t m, int t) const {
    return apart(g2) ? t : (int)(m & 1);
  }
  // whether tile t takes the lc-th chunk of the CTA's m-th item
  __device__ __forceinline__ bool takes(int g2, uint32_t m, int lc, int t) const {
    return apart(g2) || (((int)m + (chunks() > one_tile ? lc : 0)) & 1) == t;
  }
};

template <int D>
struct Shared {
  uint64_t k_full[Cfg<D>::kKStages], k_free[Cfg<D>::kKStages], v_full[Cfg<D>::kVStages], v_free[Cfg<D>::kVStages],
      q_full[kTiles], q_free[kTiles], s_full[kTiles][2], p_full[kTiles][2], o_done[kTiles][2], item_full[kItems],
      item_free[kItems], mask_full, mask_free, meet_full[4], meet_free[4], drained[2 * kTiles];
  int4 items[kItems][3];
  float2 meet_ml[4][32];
  uint8_t k_gone[kGoneRing], v_gone[kGoneRing];   // blocks of a chunk that are not there
  int up[kTreeNodes];
  uint32_t tmem_slot;
  int gave_up, odd;   // a wait ran out; some row is not finite

  template <typename F>
  __device__ __forceinline__ void barriers(F one) {   // one(barrier, arrivals)
      for (int i = 0; i < Cfg<D>::kKStages; ++i) {
        one(&k_full[i], 1);
        one(&k_free[i], kTiles);
      }
      for (int i = 0; i < Cfg<D>::kVStages; ++i) {
        one(&v_full[i], 1);
        one(&v_free[i], kTiles);
      }
      for (int t = 0; t < kTiles; ++t) {
        one(&q_full[t], 1);
        one(&q_free[t], kTiles);
        for (int h = 0; h < 2; ++h) {
          one(&s_full[t][h], 1);
          one(&p_full[t][h], 4);   // one arrival per softmax warp
          one(&o_done[t][h], 1);
        }
      }
      for (int i = 0; i < kItems; ++i) {
        one(&item_full[i], 1);
        one(&item_free[i], kRoles);
      }
      one(&mask_full, 1);
      one(&mask_free, 8);
      for (int i = 0; i < 4; ++i) {
        one(&meet_full[i], 1);
        one(&meet_free[i], 1);
      }
      for (int i = 0; i < 2 * kTiles; ++i) one(&drained[i], 1);
  }
};

// All of a CTA's items, by warps in their roles.  kCareful: with an eye to V that is not
// finite.
template <typename T, int D, bool kCareful>
__device__ __forceinline__ void attend_items(Shared<D>& sh, const TreeArgs& a, const CUtensorMap* tm_q,
                                             const CUtensorMap* tm_k, const CUtensorMap* tm_v) {
  using C = Cfg<D>;
  constexpr int SK = C::kKStages, SV = C::kVStages;
  auto &k_full = sh.k_full, &k_free = sh.k_free;
  auto &v_full = sh.v_full, &v_free = sh.v_free;
  auto &q_full = sh.q_full, &q_free = sh.q_free;
  auto &s_full = sh.s_full, &p_full = sh.p_full, &o_done = sh.o_done;
  auto &item_full = sh.item_full, &item_free = sh.item_free;
  auto &mask_full = sh.mask_full, &mask_free = sh.mask_free;
  auto &meet_full = sh.meet_full, &meet_free = sh.meet_free;
  auto& drained = sh.drained;
  auto& items = sh.items;
  auto& meet_ml = sh.meet_ml;
  auto &k_gone = sh.k_gone, &v_gone = sh.v_gone;
  auto& up = sh.up;
  volatile int* gave_up = &sh.gave_up;
  extern __shared__ unsigned char tree_smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(tree_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sQ = smem_addr(smem), sK = sQ + C::kOffK, sV = sQ + C::kOffV;
  uint32_t* masks = reinterpret_cast<uint32_t*>(smem + C::kOffMask);
  auto uniform = [](uint32_t x) -> uint32_t { return __shfl_sync(0xffffffffu, x, 0); };
  const uint32_t tmem = uniform(sh.tmem_slot);
  const int tid = threadIdx.x, warp = (int)uniform(tid >> 5), lane = tid & 31;
  const int G = a.Hq / a.Hkv, g2 = __ffs(G) - 1;   // a power of two

  bool ok = true;
  Item it;
  // the CTA's m-th item, from the warp that finds them; false past the last one
  auto take = [&](uint32_t m, Item& to) -> bool {
    const int slot = m % kItems;
    ok = cta_wait(&item_full[slot], (m / kItems) & 1, gave_up);
    if (!ok) return false;
    const int4 x = items[slot][0], y = items[slot][1];
    to.place = items[slot][2].x;
    to.tree = items[slot][2].y;
    to.one_tile = a.one_tile;
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_free[slot]);
    to.b = x.x, to.kvh = x.y, to.g = x.z, to.c0 = x.w;
    to.c1 = y.x, to.q0 = y.y, to.n = y.z, to.ctx = y.w;
    return to.n > 0;
  };

  if (warp < 8) {
    more_registers<kSoftmaxRegs>();
    // ================================================================ softmax rows
    const int t = warp >> 2, w4 = warp & 3;
    const int trow = w4 * 32 + lane;           // row inside the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)(w4 * 32) << 16;
    const uint32_t t_s = tmem + lane_base + t * kKeys;
    const uint32_t t_o = tmem + lane_base + kTmemO + t * D;
    const float qscale = a.qscale;
    // a zero scale as a tiny one: every weight is 1 and -inf stays -inf
    const float qmul = fmaxf(fabsf(qscale), 1e-37f);
    uint32_t done = 0, chunk0 = 0, met = 0;   // this tile's chunks, the CTA's, exchanges
    int held = -1;                            // the masks that this warp may still use ..
    bool mask_there = false;                  // .. and whether it has waited for them
    Item next;
    bool have = take(0, next);
    for (uint32_t m = 0; ok && have; ++m) {
      it = next;
      const int rows = it.rows(g2), n_chunks = it.chunks();
      const bool apart = it.apart(g2), both = it.shared(g2);
      const int main = m & 1;                          // the tile that ends an item of one tile's rows
      const int my_rows = apart && t == 1 ? rows - kRows : min(rows, kRows);
      const bool active = w4 * 32 < my_rows;           // a row of the warp is there
      const int group_row = apart ? t * kRows + trow : trow;
      const int row = it.g * kTreeRows + min(group_row, rows - 1);   // (node, head) of the sequence
      const int tree0 = it.ctx - it.n;
      const uint32_t* mask = masks + (row >> g2) * kMaskStride;
      if (it.tree >= 0 && it.tree != held) {
        // the last ones go back; no phase of the barrier is passed over
        if (held >= 0 && !mask_there) ok = cta_wait(&mask_full, held & 1, gave_up);
        if (!ok) break;
        __syncwarp();
        if (held >= 0 && lane == 0) mbar_arrive(&mask_free);
        held = it.tree;
        mask_there = false;
      }
      float m_run = kNoMax, l_run = 0.f;   // running maximum, unscaled; sum of weights
      float qm = qmul, base = 0.f;
      bool begun = false;
      for (int lc = 0; lc < n_chunks; ++lc) {
        if (!it.takes(g2, m, lc, t)) continue;
        const int key0 = (it.c0 + lc) * kKeys;
        const int valid = min(kKeys, it.ctx - key0);
        uint32_t gone = 0;
        // Half a chunk at a time: scores, maximum, weights.  One instance of the
        // code, so that it stays in the instruction cache.
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          ok = cta_wait(&s_full[t][half], done & 1, gave_up);
          if (!ok) break;
          tc_fence_after();
          const uint32_t t_h = t_s + kHalf * half;
          if (active && (half == 0 || valid > kHalf)) {
            if (half == 0) gone = k_gone[(chunk0 + lc) % kGoneRing];
            const int k0 = key0 + kHalf * half;
            float s[64];
            tmem_ld64(t_h, s);
            const uint32_t gone4 = (gone >> (4 * half)) & 15u;
            if (k0 + kHalf > tree0 || gone4) {
              // which of the 64 keys the row sees
              if (it.tree >= 0 && !mask_there) {
                ok = cta_wait(&mask_full, it.tree & 1, gave_up);
                if (!ok) break;
                mask_there = true;
              }
              const int rel = k0 - tree0;   // first key, counted from the tree's
              uint64_t see = ~0ull;
              if (rel > -kHalf) {
                auto word = [&](int i) -> uint64_t { return i < kMaskWords ? mask[i] : 0u; };
                if (rel < 0) {
                  see = ((word(0) | word(1) << 32) << -rel) | ((1ull << -rel) - 1);
                } else {
                  const int i = rel >> 5, by = rel & 31;
                  see = (word(i) | word(i + 1) << 32) >> by;
                  if (by) see |= word(i + 2) << (64 - by);
                }
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if ((gone4 >> i) & 1u) see &= ~(0xffffull << (16 * i));
              const uint32_t lo = (uint32_t)see, hi = (uint32_t)(see >> 32);
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                s[j] = (lo >> j) & 1u ? s[j] : -INFINITY;
                s[32 + j] = (hi >> j) & 1u ? s[32 + j] : -INFINITY;
              }
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
            // The running maximum only moves when a score passes it by more than
            // 2^8, and only then is O rescaled: weights stay below 2^8 times the
            // lift, and the stale maximum cancels in O / l.
            const bool moved = (mx - m_run) * qmul > kRescale;
            if (__any_sync(0xffffffffu, moved)) {
              const float corr = moved ? softmax_exp2((m_run - mx) * qmul) : 1.f;   // of nothing, at first
              l_run *= corr;
              if (moved) {
                m_run = mx;
                qm = fabsf(qmul * mx) < kFar ? qmul : __uint_as_float(__float_as_uint(qmul) & 0x7f800000u);
                base = __fmaf_rd(-qm, mx, kLift<T>);   // lifted no further, however large
              }
              __syncwarp();
              if (begun) {
                // the product of the half before still adds to O
                ok = cta_wait(&o_done[t][1 - half], (half ? done : done - 1) & 1, gave_up);
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
            begun = true;
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
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[t][half]);
        }
        if (!ok) break;
        ++done;
      }
      if (!ok) break;
      chunk0 += n_chunks;
      have = take(m + 1, next);   // while the last product runs
      if (!ok) break;
      // ---- the item's end: O / l, or what a partial holds
      if (!active || (!apart && t != main && !both)) continue;
      ok = cta_wait(&o_done[t][1], (done - 1) & 1, gave_up);
      if (!ok) break;
      tc_fence_after();
      // what the weights' exponents exceed (score - maximum) by: the lift, and what
      // the scaled maximum was rounded by
      float factor = softmax_exp2(-fmaf(qm, m_run, base));
      if (m_run == kNoMax) factor = 0.f;   // no key
      float* meet = reinterpret_cast<float*>(smem + C::kOffMeet + w4 * 4096);
      if (both && t != main) {
        // to the other tile's warp of the same rows, 32 columns a turn
        for (int col = 0; ok && col < D; col += 32, ++met) {
          float o[32];
          tmem_ld32(t_o + col, o);
          if (met > 0) ok = cta_wait(&meet_free[w4], (met - 1) & 1, gave_up);
          if (!ok) break;
          if (col == 0) meet_ml[w4][lane] = make_float2(m_run, l_run * factor);
#pragma unroll
          for (int i = 0; i < 32; ++i) meet[i * 32 + lane] = o[i] * factor;
          __syncwarp();
          if (lane == 0) mbar_arrive(&meet_full[w4]);
        }
        if (!ok) break;
        tc_fence_before();
        continue;
      }
      float other = 0.f;
      float2 zero = make_float2(0.f, 0.f);   // NaN if a sum is not finite
      const bool store = group_row < rows;
      const int64_t head = (int64_t)(it.q0 + (row >> g2)) * a.Hq + it.kvh * G + (row & (G - 1));
      const int64_t part = it.place == 2
                               ? (int64_t)a.num_tokens * a.Hq + (int64_t)blockIdx.x * kTreeRows + group_row
                               : head;
      for (int col = 0; ok && col < D; col += 32) {
        __syncwarp();   // lanes without a row skip the stores below
        float o[32];
        tmem_ld32(t_o + col, o);
        if (both) {
          ok = cta_wait(&meet_full[w4], met & 1, gave_up);
          if (!ok) break;
          if (col == 0) {
            const float2 ml = meet_ml[w4][lane];
            const float top = fmaxf(m_run, ml.x);
            other = softmax_exp2((ml.x - top) * qmul);
            factor *= softmax_exp2((m_run - top) * qmul);
            l_run = fmaf(ml.y, other, l_run * factor);
            m_run = top;
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = fmaf(meet[i * 32 + lane], other, o[i] * factor);
          __syncwarp();
          if (lane == 0) mbar_arrive(&meet_free[w4]);
          ++met;
        } else {
          if (col == 0) l_run *= factor;
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= factor;
        }
        if (!store) continue;
#pragma unroll
        for (int i = 0; i < 32; i += 2) add_zero_times(zero, o[i], o[i + 1]);
        if (it.place == 0) {
          const float inv = l_run > 0.f || l_run != l_run ? 1.f / l_run : 0.f;
          T* dst = static_cast<T*>(a.out) + head * D + col;
#pragma unroll
          for (int ch = 0; ch < 4; ++ch)
            *reinterpret_cast<uint4*>(dst + ch * 8) =
                make_uint4(Mma<T>::pack(o[ch * 8] * inv, o[ch * 8 + 1] * inv),
                           Mma<T>::pack(o[ch * 8 + 2] * inv, o[ch * 8 + 3] * inv),
                           Mma<T>::pack(o[ch * 8 + 4] * inv, o[ch * 8 + 5] * inv),
                           Mma<T>::pack(o[ch * 8 + 6] * inv, o[ch * 8 + 7] * inv));
        } else {
          if (col == 0) a.ws_ml[part] = make_float2(m_run, l_run);
          float* dst = a.ws_o + part * D + col;
#pragma unroll
          for (int ch = 0; ch < 8; ++ch)
            *reinterpret_cast<float4*>(dst + ch * 4) =
                make_float4(o[ch * 4], o[ch * 4 + 1], o[ch * 4 + 2], o[ch * 4 + 3]);
        }
      }
      if (!ok) break;
      if (it.tree >= 0 && !(zero.x + zero.y == 0.f)) sh.odd = 1;
      __syncwarp();
      if (kCareful && it.tree >= 0) {
        // what of the item's V is not finite, to the rows that see it, whatever its weight
        if (!mask_there) {
          ok = cta_wait(&mask_full, it.tree & 1, gave_up);
          if (!ok) break;
          mask_there = true;
        }
        const int j0 = max(0, it.c0 * kKeys - tree0), j1 = min(it.n, it.c1 * kKeys - tree0);
#pragma unroll 1
        for (int j = store ? j0 : j1; j < j1; ++j) {
          if (!((mask[j >> 5] >> (j & 31)) & 1u)) continue;
          const int key = tree0 + j;
          const int id = __ldg(a.block_tables + (int64_t)it.b * a.MBS + key / kBlockSize);
          if (id < 0 || id >= a.NB) continue;
          const T* v = static_cast<const T*>(a.v_cache) +
                       (((int64_t)id * a.Hkv + it.kvh) * kBlockSize + key % kBlockSize) * D;
#pragma unroll 1
          for (int e = 0; e < D; ++e) {
            const float x = Elem<T>::to_f32(v[e]);
            if (fabsf(x) < INFINITY) continue;
            if (it.place == 0) {
              T* dst = static_cast<T*>(a.out) + head * D + e;
              *dst = Elem<T>::narrow(Elem<T>::to_f32(*dst) + x);
            } else {
              a.ws_o[part * D + e] += x;
            }
          }
        }
      }
      tc_fence_before();   // O is read before the next item's products (p_full orders them)
    }
  } else {
    fewer_registers<kOtherRegs>();
    if (warp == 8 || warp == 9) {
      // ================================================================ copies
      // warp 8: Q and K, warp 9: V.  Lane i < 8 copies block i of a chunk.
      const bool is_v = warp == 9;
      const int S = is_v ? SV : SK;
      uint64_t* full = is_v ? v_full : k_full;
      uint64_t* freed = is_v ? v_free : k_free;
      uint8_t* missing = is_v ? v_gone : k_gone;
      const CUtensorMap* map = is_v ? tm_v : tm_k;
      const uint32_t ring = is_v ? sV : sK;
      uint32_t kc = 0, q_uses[kTiles] = {0, 0};   // chunks, Q tiles of each place asked for so far
      // Block ids come for four chunks at a time (a lane each), asked for a group ahead,
      // across items too.  -1: past the context; -2: outside the pool.
      constexpr int kGroup = 32 / kChunkBlocks;
      auto blocks_of = [&](const Item& i, int c) -> int {
        const int k = c * kChunkBlocks + lane;
        if (k >= i.c1 * kChunkBlocks || k * kBlockSize >= i.ctx) return -1;
        const int id = __ldg(a.block_tables + (int64_t)i.b * a.MBS + k);
        return id >= 0 && id < a.NB ? id : -2;
      };
      Item next;
      bool have = take(0, next);
      int ids = 0, ahead = have ? blocks_of(next, next.c0) : -1;
      for (uint32_t m = 0; ok && have; ++m) {
        it = next;
        for (int c = it.c0; c < it.c1 && ok; ++c) {
          const int st = kc % S, in_group = (c - it.c0) % kGroup;
          if (in_group == 0) ids = ahead;
          const int mine = __shfl_sync(0xffffffffu, ids, in_group * kChunkBlocks + lane % kChunkBlocks);
          const int id = lane < kChunkBlocks ? mine : -1;
          if (kc >= (uint32_t)S) ok = cta_wait(&freed[st], ((kc / S) - 1) & 1, gave_up);
          if (!ok) break;
          const unsigned present = __ballot_sync(0xffffffffu, id >= 0);
          const unsigned bad = __ballot_sync(0xffffffffu, id == -2);
          if (lane == 0) {
            missing[kc % kGoneRing] = (uint8_t)bad;   // published by the arrival below
            if (bad && !is_v) raise_error(a.err, kErrBlock);
            mbar_arrive_expect_tx(&full[st], __popc(present) * (kBlockSize * D * 2));
          }
          __syncwarp();
          if (id >= 0) {
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_box(ring + st * C::kKvBytes + h * (kKeys * 128) + lane * (kBlockSize * 128),
                           map, h * 64, (id * a.Hkv + it.kvh) * kBlockSize, &full[st]);
          }
          __syncwarp();
          ++kc;
          if (!is_v && c == it.c0) {
            // the Q tiles, after the first chunk is on its way
            for (int i = 0; ok && i < kTiles; ++i) {
              if (it.place_of(g2, m, i) != i) continue;
              if (q_uses[i] > 0) ok = cta_wait(&q_free[i], (q_uses[i] - 1) & 1, gave_up);
              if (!ok) break;
              ++q_uses[i];
              if (lane != 0) continue;
              const int first = it.g * kTreeRows + (it.apart(g2) ? i * kRows : 0);
              mbar_arrive_expect_tx(&q_full[i], C::kQBytes);
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                tma_load_box3(sQ + i * C::kQBytes + h * (kRows * 128), tm_q, h * 64, it.kvh * G,
                              it.q0 + (first >> g2), &q_full[i]);
            }
            __syncwarp();
            if (!ok) break;
          }
          if (in_group == 0) {
            if (c + kGroup < it.c1) {
              ahead = blocks_of(it, c + kGroup);
            } else {
              have = take(m + 1, next);
              if (ok && have) ahead = blocks_of(next, next.c0);
            }
          }
        }
      }
      if (!ok) {
        // what is in flight lands before the CTA ends
        for (uint32_t c = kc > (uint32_t)S ? kc - S : 0; c < kc; ++c)
          (void)mbar_wait_bounded(&full[c % S], (c / S) & 1);
        for (int i = 0; i < kTiles; ++i)
          if (q_uses[i] > 0) (void)mbar_wait_bounded(&q_full[i], (q_uses[i] - 1) & 1);
      }
    } else if (warp == 14) {
      // ================================================================ items
      // where the CTA's run lies on the line
      const Seq first = seq_of(a, lane);   // most batches need no more loads
      auto seqs = [&](int b0) { return b0 == 0 ? first : seq_of(a, b0 + lane); };
      int64_t total = 0;
      for (int b0 = 0; b0 < a.B; b0 += 32)
        total += __reduce_add_sync(0xffffffffu, (unsigned)units_of(a, seqs(b0), G));
      const int per = (int)((total + gridDim.x - 1) / gridDim.x);
      const int u0 = (int)min(total, (int64_t)blockIdx.x * per), u1 = (int)min(total, (int64_t)u0 + per);
      uint32_t m = 0;
      int trees = 0, masked_b = -1;   // masks asked for so far, and the last one's sequence
      bool told = false;
      // whose partials lie with this CTA: the pair that its run begins in the midst of
      auto tell = [&](const Item& i, int t_first, int t_last) {
        if (!told && lane == 0) {
          a.ws_split[2 * blockIdx.x] = make_int4(i.q0, i.n, i.kvh, i.g);
          a.ws_split[2 * blockIdx.x + 1] = make_int4(t_first, t_last, 0, 0);
        }
        told = true;
      };
      auto publish = [&](const Item& i) {
        const int slot = m % kItems;
        if (m >= kItems) ok = cta_wait(&item_free[slot], ((m / kItems) - 1) & 1, gave_up);
        if (!ok) return;
        if (lane == 0) {
          items[slot][0] = make_int4(i.b, i.kvh, i.g, i.c0);
          items[slot][1] = make_int4(i.c1, i.q0, i.n, i.ctx);
          items[slot][2].x = i.place;
          items[slot][2].y = i.tree;
          mbar_arrive(&item_full[slot]);
        }
        __syncwarp();
        ++m;
      };
      it = Item{};
      int u = 0;   // units before sequence b0 + ..
      for (int b0 = 0; ok && b0 < a.B && u < u1; b0 += 32) {
        const Seq here = seqs(b0);
        const int mine = units_of(a, here, G);
        int sum = mine;   // inclusive prefix
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += y;
        }
        unsigned in = __ballot_sync(0xffffffffu, mine > 0 && u + sum > u0 && u + sum - mine < u1);
        while (ok && in) {
          const int k = __ffs(in) - 1;
          in &= in - 1;
          const int start = u + __shfl_sync(0xffffffffu, sum - mine, k);
          it.b = b0 + k;
          it.q0 = __shfl_sync(0xffffffffu, here.q0, k);
          it.n = __shfl_sync(0xffffffffu, here.n, k);
          it.ctx = __shfl_sync(0xffffffffu, here.ctx, k);
          const int chunks = chunks_of(it.ctx), groups = groups_of(it.n, G), each = chunks + kTreePairCost;
          for (int p = max(0, u0 - start) / each; ok && p < a.Hkv * groups; ++p) {
            const int at = start + p * each + kTreePairCost;   // the pair's first chunk on the line
            if (at - kTreePairCost >= u1) break;
            it.kvh = p / groups;
            it.g = p - it.kvh * groups;
            int t_first = at / per, t_last = (at + chunks - 1) / per;
            if (a.split) {
              it.c0 = max(0, u0 - at);
              it.c1 = min(chunks, u1 - at);
            } else {   // all of it, where it begins
              it.c0 = 0;
              it.c1 = at - kTreePairCost >= u0 ? chunks : 0;
              t_first = t_last = blockIdx.x;
            }
            if (it.c1 <= it.c0) continue;
            it.place = t_first == t_last ? 0 : (int)blockIdx.x == t_first ? 1 : 2;
            tell(it, t_first, it.place == 2 ? t_last : -1);
            const bool tree = it.c1 * kKeys > it.ctx - it.n, fresh = tree && it.b != masked_b;
            trees += fresh;
            it.tree = tree ? trees - 1 : -1;
            if (tree) masked_b = it.b;
            publish(it);
          }
        }
        u += __shfl_sync(0xffffffffu, sum, 31);
      }
      it.n = 0;
      tell(it, 0, -1);
      if (ok) publish(it);
    } else if (warp == 15) {
      // ================================================================ the nodes' ancestors
      // One set of masks at a time, for all items of a sequence in a row; a softmax warp
      // gives them back on the first item with others.
      int made = -1;
      for (uint32_t m = 0; ok && take(m, it); ++m) {
        if (it.tree <= made) continue;
        made = it.tree;
        if (made > 0) ok = cta_wait(&mask_free, (made - 1) & 1, gave_up);
        if (!ok) break;
        const int words = (it.n + 31) >> 5;
        bool wrong = false;
        for (int i = lane; i < it.n; i += 32) {
          int x = __ldg(a.parents + it.q0 + i);
          if (x < -1 || x >= i) {
            wrong = true;
            x = -1;
          }
          up[i] = x;
#pragma unroll
          for (int w = 0; w < kMaskWords; ++w)
            masks[i * kMaskStride + w] = w == i >> 5 ? 1u << (i & 31) : 0u;
        }
        if (wrong) raise_error(a.err, kErrTree);
        __syncwarp();
        // node i's mask holds it and its ancestors down to, not with, up[i]
        bool more = true;
        while (more) {
          more = false;
          for (int i0 = 0; i0 < it.n; i0 += 32) {
            const int i = i0 + lane;
            const int x = i < it.n ? up[i] : -1;
            int y = -1;
            uint32_t add[kMaskWords];
            if (x >= 0) {
              y = up[x];
#pragma unroll
              for (int w = 0; w < kMaskWords; ++w) add[w] = w < words ? masks[x * kMaskStride + w] : 0u;
            }
            __syncwarp();   // a node's mask and its up change together
            if (x >= 0) {
              up[i] = y;
#pragma unroll
              for (int w = 0; w < kMaskWords; ++w)
                if (w < words) masks[i * kMaskStride + w] |= add[w];
            }
            __syncwarp();
            more |= __any_sync(0xffffffffu, y >= 0);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&mask_full);
      }
      // ---- rejected sequences: their error, and zero rows where they have rows
      for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (seq_of(a, b).n > 0) continue;
        const int q0 = __ldg(a.query_start + b), n = __ldg(a.query_start + b + 1) - q0;
        const bool outside = q0 < 0 || n < 0 || q0 + n > a.num_tokens;
        if (n == 0 && !outside) continue;
        if (lane == 0) raise_error(a.err, outside || n > a.max_query_len ? kErrQuery : kErrContext);
        if (outside) continue;
        const int64_t chunks = (int64_t)min(n, a.max_query_len) * a.Hq * (D / 8);
        uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + (int64_t)q0 * a.Hq * D);
        for (int64_t i = lane; i < chunks; i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
      }
    } else if (warp >= 10 && warp < 14) {
      // ================================================================ products
      const int t = (warp - 10) & 1;
      const uint32_t t_s = tmem + t * kKeys, t_o = tmem + kTmemO + t * D;
      // a descriptor's start address is address >> 4 in its low 14 bits; every
      // operand lies below 256 KB, so offsets are added to the base's descriptor
      uint32_t chunk0 = 0, done = 0;   // the item's first chunk; chunks of this tile so far
      const bool leader = elect_one();
      if (warp < 12) {
        // with a negative scale the product is negated (A's sign bit of the
        // descriptor), so that the maximum is always the largest score
        const uint32_t id_s = f16_idesc<T>(kRows, kHalf) | (a.qscale < 0.f ? 1u << 13 : 0u);
        const uint64_t q_desc0 = sw128_desc(sQ), k_desc = sw128_desc(sK);
        uint32_t q_uses0 = 0, q_uses1 = 0;   // of each place so far
        for (uint32_t m = 0; ok && take(m, it); ++m) {
          const int n_chunks = it.chunks(), place = it.place_of(g2, m, t);
          const uint64_t q_desc = q_desc0 + (uint64_t)((place * C::kQBytes) >> 4);
          ok = cta_wait(&q_full[place], (place ? q_uses1 : q_uses0) & 1, gave_up);
          // An item with rows of both tiles hands both places back.  Without this wait a
          // warp that had nothing to do in the item before could hand the other place back
          // twice in one phase, while the other tile's products still read it.
          if (ok && it.apart(g2)) ok = cta_wait(&q_full[1 - place], (place ? q_uses0 : q_uses1) & 1, gave_up);
          if (!ok) break;
          for (int lc = 0; lc < n_chunks; ++lc) {
            const uint32_t kc = chunk0 + lc;
            ok = cta_wait(&k_full[kc % SK], (kc / SK) & 1, gave_up);
            if (ok && it.takes(g2, m, lc, t)) {
              const uint64_t kb = k_desc + (uint64_t)(((kc % SK) * C::kKvBytes) >> 4);
              for (int h = 0; h < 2; ++h) {
                // P of the last chunk's half, which lies over S, is used
                if (done > 0) ok = cta_wait(&o_done[t][h], (done - 1) & 1, gave_up);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                  for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t at = (kk & 3) * 32;
                    tc_mma(t_s + h * kHalf, q_desc + (uint64_t)(((kk >> 2) * (kRows * 128) + at) >> 4),
                           kb + (uint64_t)(((kk >> 2) * (kKeys * 128) + h * (kHalf * 128) + at) >> 4),
                           id_s, kk > 0);
                  }
                  tc_commit(&s_full[t][h]);
                }
                __syncwarp();
              }
              if (!ok) break;
              ++done;
              ok = cta_wait(&s_full[t][1], (done - 1) & 1, gave_up);
            }
            if (!ok) break;
            if (lane == 0) mbar_arrive(&k_free[kc % SK]);
          }
          if (!ok) break;
          // the item's S are done
          if (it.place_of(g2, m, 0) == 0) {
            ++q_uses0;
            if (lane == 0) mbar_arrive(&q_free[0]);
          }
          if (it.place_of(g2, m, 1) == 1) {
            ++q_uses1;
            if (lane == 0) mbar_arrive(&q_free[1]);
          }
          chunk0 = uniform(chunk0 + n_chunks);
        }
      } else {
        const uint32_t id_o = f16_idesc<T>(kRows, D) | (1u << 16);   // B (V) MN-major
        const uint64_t v_desc = v_operand(sV);
        constexpr uint32_t kNothing = ~0u;
        uint32_t held = kNothing;   // the chunk whose V stage is to be handed back
        for (uint32_t m = 0; ok && take(m, it); ++m) {
          const int n_chunks = it.chunks();
          bool begun = false;
          for (int lc = 0; lc < n_chunks; ++lc) {
            const uint32_t vc = chunk0 + lc;
            if (held != kNothing) {
              ok = cta_wait(&o_done[t][1], (done - 1) & 1, gave_up);
              if (!ok) break;
              if (lane == 0) mbar_arrive(&v_free[held % SV]);
              held = kNothing;
            }
            ok = cta_wait(&v_full[vc % SV], (vc / SV) & 1, gave_up);
            if (!ok) break;
            if (!it.takes(g2, m, lc, t)) {   // a chunk of the other tile
              if (lane == 0) mbar_arrive(&v_free[vc % SV]);
              continue;
            }
            const int valid = min(kKeys, it.ctx - (it.c0 + lc) * kKeys);
            const int steps = (valid + 15) / 16;
            // The products read whole groups of 16 keys.  Rows past the last key,
            // and of blocks that are not there, meet zero weights, but 0 x NaN would
            // not vanish: they are filled up with zeros.  (Where both tiles see the
            // chunk both do it: the same zeros, before their own products.)
            const uint32_t gone = v_gone[vc % kGoneRing];
            if (gone || (valid & 15)) {
              unsigned char* rows = smem + C::kOffV + (vc % SV) * C::kKvBytes;
              for (int i = lane; i < steps * 16 * (D / 8); i += 32) {
                const int r = i / (D / 8), ch = i % (D / 8);
                if (r >= valid || (gone >> (r >> 4)) & 1u)
                  *reinterpret_cast<uint4*>(rows + (ch >> 3) * (kKeys * 128) + r * 128 + ((ch & 7) << 4)) =
                      make_uint4(0u, 0u, 0u, 0u);
              }
              fence_async_smem();
              __syncwarp();
            }
            // A node's V meets zero weights, too, of the rows that do not see it: here what
            // of it is not finite is taken out, and added at the item's end to the rows that
            // do.  (Where both tiles see the chunk both do it, as above.)
            const int tree_row = max(0, it.ctx - it.n - (it.c0 + lc) * kKeys);   // the chunk's first
            if (kCareful && tree_row < valid) {
              unsigned char* rows = smem + C::kOffV + (vc % SV) * C::kKvBytes;
              __syncwarp();   // filled up above
#pragma unroll 1
              for (int i = lane; i < (valid - tree_row) * (D / 8); i += 32) {
                const int r = tree_row + i / (D / 8), ch = i % (D / 8);
                uint4* at = reinterpret_cast<uint4*>(rows + (ch >> 3) * (kKeys * 128) + r * 128 + ((ch & 7) << 4));
                *at = finite8<T>(*at);
              }
              fence_async_smem();
              __syncwarp();
            }
            const uint64_t vb = v_desc + (uint64_t)(((vc % SV) * C::kKvBytes) >> 4);
            // 64 keys at a time, as their weights become ready; a half without keys
            // has nothing to add, only its barrier to complete
            for (int h = 0; h < 2; ++h) {
              ok = cta_wait(&p_full[t][h], done & 1, gave_up);
              if (!ok) break;
              tc_fence_after();
              auto product = [&](int kk) {
                tc_mma_ts(t_o, t_s + h * kHalf + kk * 8,
                          vb + (uint64_t)((h * (kHalf * 128) + kk * 2048) >> 4), id_o,
                          begun || h > 0 || kk > 0 ? 1u : 0u);
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
            begun = true;
            held = vc;
            ++done;
          }
          chunk0 = uniform(chunk0 + n_chunks);
        }
      }
      if (!ok) {
        if (leader) tc_commit(&drained[warp - 10]);
        __syncwarp();
        (void)mbar_wait_bounded(&drained[warp - 10], 0);
      }
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const TreeArgs a) {
  __shared__ __align__(16) Shared<D> sh;
  const int tid = threadIdx.x, warp = (int)__shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    sh.gave_up = sh.odd = 0;
    sh.barriers([](uint64_t* bar, int n) { mbar_init(bar, n); });
    mbar_init_fence();
  }
  if (warp == 0) tmem_alloc(&sh.tmem_slot, 512);
  if (tid == 32 * 8) {
    prefetch_tensor_map(&tm_q);
    prefetch_tensor_map(&tm_k);
  }
  if (tid == 32 * 9) prefetch_tensor_map(&tm_v);
  pdl_wait_primary();
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  attend_items<T, D, false>(sh, a, &tm_q, &tm_k, &tm_v);
  tc_fence_before();
  __syncthreads();
  if (sh.odd && !sh.gave_up) {
    // Some row is not finite, which may have come from a node that it does not see: all
    // of the CTA's items once more.  Everything that was in flight is done.
    if (warp < 8)
      fewer_registers<kLaunchRegs>();
    else
      more_registers<kLaunchRegs>();
    if (tid == 0) {
      sh.barriers([](uint64_t* bar, int) { mbar_inval(bar); });
      sh.barriers([](uint64_t* bar, int n) { mbar_init(bar, n); });
      mbar_init_fence();
    }
    __syncthreads();
    tc_fence_after();
    attend_items<T, D, true>(sh, a, &tm_q, &tm_k, &tm_v);
    tc_fence_before();
    __syncthreads();
  }
  if (tid == 0 && sh.gave_up) raise_error(a.err, kErrTimeout);
  if (warp == 0) tmem_dealloc(sh.tmem_slot, 512);
}

// The weighted sums of some partials of a row: l, and four elements of o, against the
// largest of their maxima m; w_p = 2^(scale (m_p - m)).
struct Joined {
  float m = kNoMax, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void raise(float to, float qmul) {
    const float r = softmax_exp2((m - to) * qmul);
    m = to;
    l *= r;
    o.x *= r, o.y *= r, o.z *= r, o.w *= r;
  }
  __device__ __forceinline__ void add(float2 ml, float4 v, float qmul) {   // ml.x <= m
    const float w = softmax_exp2((ml.x - m) * qmul);
    l = fmaf(w, ml.y, l);
    o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y), o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
  }
};

// out = sum_p w_p o_p / sum_p w_p l_p over the partials of a row.  A pair's partials lie
// with consecutive CTAs, and the second one's index names the pair here.  A CTA takes a
// slice of its rows; D / 4 lanes a row and each of kSplit parts of its partials, all
// asked for at once: one round trip for up to 16 partials (kSplit > 1), or for two rows'
// 4 (kSplit == 1).
constexpr int kMergeThreads = 256;
template <int D, int kSplit>
constexpr int kMergeRows = kMergeThreads / (D / 4 * kSplit) * (kSplit == 1 ? 2 : 1);

template <typename T, int D, int kSplit>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const TreeArgs a) {
  constexpr int kLanes = D / 4, kAtOnce = kMergeThreads / (kLanes * kSplit);
  constexpr int kAhead = kSplit == 1 ? 4 : 16 / kSplit;
  constexpr int kInFlight = kSplit == 1 ? 2 : 1;
  __shared__ Joined parts_of[kSplit > 1 ? kMergeThreads : 1];
  pdl_launch_dependents();
  pdl_wait_primary();
  const int4 at = a.ws_split[2 * (blockIdx.y + 1)], of = a.ws_split[2 * (blockIdx.y + 1) + 1];
  if (of.y < 0 || of.x != (int)blockIdx.y) return;   // nothing, or another one's pair
  const int lane = threadIdx.x % kLanes, part = threadIdx.x / kLanes % kSplit;
  const int G = a.Hq / a.Hkv, g2 = __ffs(G) - 1;
  const int q0 = at.x, n = at.y, kvh = at.z, g = at.w, parts = of.y - of.x + 1;
  const int rows = min(n << g2, (g + 1) * kTreeRows);
  const int row0 = g * kTreeRows + (int)blockIdx.x * (kAtOnce * kInFlight) + threadIdx.x / (kLanes * kSplit);
  if (g * kTreeRows + (int)blockIdx.x * (kAtOnce * kInFlight) >= rows) return;
  const float qmul = fmaxf(fabsf(a.qscale), 1e-37f);
  Joined sum[kInFlight];
  for (int p0 = part; p0 < parts; p0 += kSplit * kAhead) {
    float4 v[kInFlight][kAhead];
    float2 ml[kInFlight][kAhead];
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      const int r = min(row0 + k * kAtOnce, rows - 1);
      // the first partial lies with the row, the others with their CTAs
      const int64_t head = (int64_t)(q0 + (r >> g2)) * a.Hq + kvh * G + (r & (G - 1));
      const int64_t later = (int64_t)a.num_tokens * a.Hq + (int64_t)of.x * kTreeRows + (r - g * kTreeRows);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int p = p0 + i * kSplit;
        ml[k][i] = make_float2(kNoMax, 0.f);
        v[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p < parts) {
          const int64_t row = p == 0 ? head : later + (int64_t)p * kTreeRows;
          ml[k][i] = a.ws_ml[row];
          v[k][i] = reinterpret_cast<const float4*>(a.ws_o + row * D)[lane];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      float top = sum[k].m;
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (ml[k][i].y != 0.f) top = fmaxf(top, ml[k][i].x);
      sum[k].raise(top, qmul);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (ml[k][i].y != 0.f) sum[k].add(ml[k][i], v[k][i], qmul);   // else no key of that part, or none
    }
  }
  if constexpr (kSplit > 1) {
    parts_of[threadIdx.x] = sum[0];
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int i = 1; i < kSplit; ++i) {
      const Joined x = parts_of[threadIdx.x + i * kLanes];
      if (x.l == 0.f) continue;
      sum[0].raise(fmaxf(sum[0].m, x.m), qmul);
      sum[0].add(make_float2(x.m, x.l), x.o, qmul);
    }
  }
#pragma unroll
  for (int k = 0; k < kInFlight; ++k) {
    const int r = row0 + k * kAtOnce;
    if (r >= rows) continue;
    const float l = sum[k].l, inv = l > 0.f || l != l ? 1.f / l : 0.f;
    const int64_t head = (int64_t)(q0 + (r >> g2)) * a.Hq + kvh * G + (r & (G - 1));
    const float4 o = sum[k].o;
    reinterpret_cast<uint2*>(static_cast<T*>(a.out) + head * D)[lane] =
        make_uint2(Mma<T>::pack(o.x * inv, o.y * inv), Mma<T>::pack(o.z * inv, o.w * inv));
  }
}

template <typename T, int D>
cudaError_t launch_t(TreeArgs a, cudaStream_t stream) {
  using C = Cfg<D>;
  auto kern = tree_attention_kernel<T, D>;
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
  CUtensorMap tq, tk, tv;
  // q as [token][head][element], a box of 128 / G tokens x G heads x 64 elements
  const cuuint32_t G = (cuuint32_t)(a.Hq / a.Hkv);
  const cuuint64_t qd[3] = {(cuuint64_t)D, (cuuint64_t)a.Hq, (cuuint64_t)a.num_tokens};
  const cuuint64_t qs[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.Hq * D * 2};
  const cuuint32_t qb[3] = {64, G, (cuuint32_t)kRows / G};
  e = encode_tensor_map(&tq, a.dtype == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        3, a.q, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  if ((e = make_pool_map(&tk, a.k_cache, a.dtype, a.NB, a.Hkv, a.D)) != cudaSuccess) return e;
  if ((e = make_pool_map(&tv, a.v_cache, a.dtype, a.NB, a.Hkv, a.D)) != cudaSuccess) return e;
  const int64_t pairs = (int64_t)a.B * a.Hkv * groups_of(a.max_query_len, (int)G);
  const int chunks = (a.MBS * kBlockSize + kKeys - 1) / kKeys;   // of the longest context there can be
  const int grid = (int)std::min<int64_t>(std::min(a.num_sms, kTreeMaxCtas), pairs * (chunks + kTreePairCost));
  const int64_t spare = (pairs + grid - 1) / grid * grid - pairs;   // places that whole pairs leave empty
  a.split = grid > 1 && (chunks > kWholePairs || 2 * chunks * spare > kWholeIdle2 * grid);
  a.one_tile = pairs > grid ? kOneTile : 1;
  e = launch_pdl(kern, dim3(grid), dim3(kThreads), C::kSmem, stream, tq, tk, tv, a);
  if (e != cudaSuccess) return e;
  if (!a.split) return cudaSuccess;
  // With fewer pairs than CTAs each pair has several partials; with more, two or so.
  const int rows = std::min(a.max_query_len * (int)G, kTreeRows);
  auto slices = [&](int each) { return dim3((rows + each - 1) / each, grid - 1); };
  if (pairs < grid)
    return launch_pdl(tree_merge_kernel<T, D, 256 / D>, slices(kMergeRows<D, 256 / D>),
                      dim3(kMergeThreads), 0, stream, a);
  return launch_pdl(tree_merge_kernel<T, D, 1>, slices(kMergeRows<D, 1>), dim3(kMergeThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_tree_attention(const TreeArgs& a, cudaStream_t stream) {
  if (a.dtype == 1)
    return a.D == 64 ? launch_t<__half, 64>(a, stream) : launch_t<__half, 128>(a, stream);
  return a.D == 64 ? launch_t<__nv_bfloat16, 64>(a, stream) : launch_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace photon
