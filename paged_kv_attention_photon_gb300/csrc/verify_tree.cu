// verify_tree.cu -- rejection sampling of drafted trees against the target's
// probabilities, from given random numbers.
//
// PhotonInfer README, "Key features / GPU-optimized kernels" (zero-copy GPU
// sampling); "Roadmap" (speculative decoding).
//
// At node c with the target's p and the draft's q, r = p and Z = 1; a child x is
// accepted if r(x) > u Z q(x), else r <- max(0, r / Z - q), Z <- sum r.  Up to a
// factor, which neither the test nor the sampling needs, r is (p - L q)+ with L = 0,
// and with F = 1, then F = sum (p - L q)+, in the place of Z a rejection is L <- L +
// F: one number stands for the whole row, and a rejection costs one pass over two
// rows for F, none if no sibling follows (the sampling pass finds the sum itself).
// Without q a child is a point mass: Z loses r(x), and the row needs no pass at all.
//
// (p - L q)+ loses what p and L q have in common: where F is a millionth of L, the rest of
// the tree is verified as the definition says it, in double: each element's r from p and
// the row sums so far, a pass over the rows for each of them.  Children that the draft
// drew get there once in a million times.  (Never mind the time: 8 sequences with 255
// rejections each over 128256 tokens 20 ms, 320 where hardly an element drops out.)
//
// What it answers are whole numbers, so what they hang on is held to about 48 bits:
// L, F and the row sums are pairs of floats whose rounding errors are carried along
// (two-sum), two elements an instruction; a test is made in single precision, and
// where that leaves it open in double.  Doubles throughout are too slow here, the rows
// by their rate, the walk by their latency.
//
// A cluster of CTAs takes a sequence.  All of them walk the tree, each for itself,
// from the nodes' probabilities in shared memory; a pass over a row is cut into one
// run per CTA and warp, the sums meet through distributed shared memory, and the
// warp in whose run the sampled sum is passed goes through it once more (L2).  So
// a step is one launch, and even one sequence has several SMs to read with.
//
// Measured: 4 chains of 5 over 32000 tokens 7.2 us (4.8 for one node and 1000 tokens: the
// launch, three dependent loads, the sums' way over the cluster and the search); 64 x 1
// node over 128256 tokens 12.9 us, 64 chains of 16 24; 32 x 1 .. 48 chosen nodes over 99991
// 12.3 us; 64 x 16 drawn nodes over 128256 56 to 70 us, as the draws fall, which is up to seven passes one
// after another in the slowest sequence, 5 to 7 us each: all sequences' first ones share
// the memory, the last one's are its cluster's latency.  The first version, A and B in
// doubles for every thread and sums of single elements, took 12.8 us for the 4 chains,
// 18.9 for the chosen nodes and 111 for the drawn ones.  Measured and left out: clusters of
// 16 (19.1 us for 64 x 1 node, 53 to 62), loads of four chunks ahead of their sums (12.8, 55
// to 66), a pass's next loads before its sums (17.9, 67).
#include <math.h>

#include <algorithm>

#include "speculate.cuh"

namespace photon {
namespace {

constexpr int kVerifyResident = 1024;   // threads per SM: 64 registers each
constexpr int kVerifyCluster = 8;   // most CTAs of a cluster
// What is left of 1 (of L) so far below it that 48 bits of that are few of its own.
constexpr float kLittle = 1.f / (1 << 20);
constexpr int kVerifyRun = kVerifyVocab / kVerifyCluster;   // most tokens of a CTA's run

// Two floats in one register pair, and the paired instructions.
typedef unsigned long long Pair;
__device__ __forceinline__ Pair pair(float x, float y) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ float2 parts(Pair p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
  return f;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ Pair sub2(Pair a, Pair b) {   // a - b, rounded once
  return fma2(b, pair(-1.f, -1.f), a);
}

// A sum held in two floats.  a + b and b + a are the same bits (what hi rounds off is
// exact in either order, and is added to lo + rest), so that lanes which exchange their
// sums hold the same one: all of a warp walks the tree, and has to go one way.
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x, float rest) {
    const float s = hi + x, b = s - hi;
    lo = (lo + rest) + ((hi - (s - b)) + (x - b));
    hi = s;
  }
  // lo no more than half a step of hi
  __device__ __forceinline__ void settle() {
    const float s = hi + lo, b = s - hi;
    lo = (hi - (s - b)) + (lo - b);
    hi = s;
  }
  __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
  __device__ __forceinline__ bool positive() const { return hi + lo > 0.f; }
  __device__ __forceinline__ bool above(const Sum2& t) const { return (hi - t.hi) + (lo - t.lo) > 0.f; }
  // the sum over `lanes` neighbouring lanes, in all of them
  __device__ __forceinline__ void over(int lanes) {
    for (int o = 1; o < lanes; o <<= 1) {
      const float x = __shfl_xor_sync(0xffffffffu, hi, o), y = __shfl_xor_sync(0xffffffffu, lo, o);
      add(x, y);
    }
  }
};
// Two such sums side by side.
struct Sums2 {
  Pair hi = 0, lo = 0;
  __device__ __forceinline__ void add(Pair x, Pair rest) {
    const Pair s = add2(hi, x), b = sub2(s, hi);
    const Pair off = add2(sub2(hi, sub2(s, b)), sub2(x, b));
    lo = add2(lo, add2(off, rest));
    hi = s;
  }
  __device__ __forceinline__ Sum2 both() const {
    const float2 h = parts(hi), l = parts(lo);
    Sum2 s;
    s.hi = h.x;
    s.lo = l.x;
    s.add(h.y, l.y);
    return s;
  }
};
// before, and x of the lanes up to each one's: prefix sums over a warp.
__device__ __forceinline__ Sum2 prefix(const Sum2& before, Sum2 x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float h = __shfl_up_sync(0xffffffffu, x.hi, o), l = __shfl_up_sync(0xffffffffu, x.lo, o);
    if (lane >= o) x.add(h, l);
  }
  x.add(before.hi, before.lo);
  return x;
}
__device__ __forceinline__ Sum2 of_lane(const Sum2& x, int lane) {
  Sum2 s;
  s.hi = __shfl_sync(0xffffffffu, x.hi, lane);
  s.lo = __shfl_sync(0xffffffffu, x.lo, lane);
  return s;
}
// x > y for x = max(0, p - L q), y = u F q, L settled: in single precision where that is
// clear (each side is off by a few 2^-24 of what goes into it), else in double.
__device__ __forceinline__ bool passes(float p, float q, const Sum2& L, float u, const Sum2& F) {
  const float lq = L.hi * q, x = fmaxf(p - lq, 0.f), y = u * (F.hi + F.lo) * q;
  if (fabsf(x - y) > 1e-5f * (p + lq + y)) return x > y;
  return fmax((double)p - L.value() * (double)q, 0.0) > (double)u * F.value() * (double)q;
}

// An entry as a probability: NaN and negative ones are 0, ones above 1 are 1.
__device__ __forceinline__ float as_prob(float x) { return __saturatef(x); }

// r = (p - L q)+ of two elements as r + rest, L = hi + lo.  What is left may be a small
// part of p, next to L q: whether anything is hangs on all of L q, and r takes what rest
// has of it, so that sums are as exact as what they add up.
__device__ __forceinline__ void left_of(float2 p, float2 q, float hi, float lo, Pair& r, Pair& rest) {
  const Pair h = pair(hi, hi), qq = pair(q.x, q.y), pp = pair(p.x, p.y);
  const Pair y = mul2(h, qq);
  // what rounding y has cost, and L's second part
  const Pair yl = fma2(pair(lo, lo), qq, fma2(h, qq, sub2(0, y)));
  const Pair d = sub2(pp, y);
  // (p - d) - y is exact: p > y or so near to it that d is
  const Pair e = sub2(sub2(sub2(pp, d), y), yl);
  const Pair s = add2(d, e);
  const float2 df = parts(d), ylf = parts(yl), sf = parts(s), ef = parts(sub2(e, sub2(s, d)));
  const bool x = df.x > ylf.x, z = df.y > ylf.y;
  r = pair(x ? sf.x : 0.f, z ? sf.y : 0.f);
  rest = pair(x ? ef.x : 0.f, z ? ef.y : 0.f);
}

// 16 bytes of a row from element e on; what lies behind its end is 0.
template <typename T, bool kVec>
__device__ __forceinline__ uint4 load_chunk(const T* row, int e, int vocab) {
  constexpr int N = 16 / sizeof(T);
  if (kVec && e + N <= vocab) return __ldg(reinterpret_cast<const uint4*>(row + e));
  union {
    uint4 all;
    T one[N];
  } c;
  c.all = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (e + i < vocab) c.one[i] = row[e + i];
  return c.all;
}

__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();   // the aligned form is for warps whose lanes have met
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();   // the aligned form is for warps whose lanes have met
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores into the same place of another CTA's shared memory.
__device__ __forceinline__ void store_peer(float2* p, int rank, float2 v) {
  asm volatile(
      "{\n.reg .b32 at;\nmapa.shared::cluster.u32 at, %0, %1;\n"
      "st.shared::cluster.v2.f32 [at], {%2, %3};\n}" ::"r"(smem_addr(p)),
      "r"(rank), "f"(v.x), "f"(v.y)
      : "memory");
}

// What of a sequence's verification is in shared memory.
template <int kWarps>
struct VerifyTree {
  int parent[kTreeNodes], token[kTreeNodes], path[kTreeNodes];
  float prob[kTreeNodes], draft[kTreeNodes], number[kTreeNodes];
  double inverse[kTreeNodes];   // 1 / Z of each rejection
  float2 sums_of[2][kVerifyCluster * kWarps];
};

// The rest of a walk from `node`, the len-th of the path, by its definition and in double:
// r after some rejections is p through r <- max(0, r / Z - q) for each of them.  Slow, for
// where little is left; every thread of the cluster goes the same way, by itself.
template <typename T, int kWarps>
__device__ __noinline__ void finish_in_double(const VerifyArgs& a, VerifyTree<kWarps>& s, int b, int ranks,
                                              int node, int len, int round) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x % ranks;
  const int q0 = __ldg(a.query_start + b), n = __ldg(a.query_start + b + 1) - q0, V = a.vocab;
  const int each = (V + ranks * kWarps - 1) / (ranks * kWarps);
  const int run0 = min(V, (rank * kWarps + warp) * each), run1 = min(V, run0 + each);
  int times = 0;
  auto left = [&](float p, float q) -> double {
    double r = p;
    for (int j = 0; j < times && r > 0.0; ++j) r = fma(r, s.inverse[j], -(double)q);
    return fmax(r, 0.0);
  };
  auto of_row = [&](int e) -> double {
    const int64_t row = q0 + node;
    return left(as_prob(Elem<T>::to_f32(static_cast<const T*>(a.target)[row * a.target_stride + e])),
                as_prob(Elem<T>::to_f32(static_cast<const T*>(a.draft)[row * a.draft_stride + e])));
  };
  auto share = [&](int k) -> double {   // of the last sum, warp k's of the cluster
    const float2 x = s.sums_of[(round - 1) & 1][k];
    return __hiloint2double(__float_as_int(x.y), __float_as_int(x.x));
  };
  auto sum = [&]() -> double {
    double mine = 0.0;
    for (int e = run0 + lane; e < run1; e += 32) mine += of_row(e);
    __syncwarp();
    for (int o = 1; o < 32; o <<= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    const int parity = round++ & 1;
    if (lane < ranks)
      store_peer(&s.sums_of[parity][rank * kWarps + warp], lane,
                 make_float2(__int_as_float(__double2loint(mine)), __int_as_float(__double2hiint(mine))));
    cluster_arrive();
    cluster_wait();
    double all = 0.0;
    for (int k = 0; k < ranks * kWarps; ++k) all += share(k);
    return all;
  };
  double Z = 1.0;
  for (int j = node + 1; j < n; ++j) {
    if (s.parent[j] != node || s.token[j] < 0) continue;
    if (left(s.prob[j], s.draft[j]) > (double)s.number[j] * Z * (double)s.draft[j]) {
      if (tid == 0) s.path[len] = j;
      ++len;
      node = j;
      times = 0;
      Z = 1.0;
      continue;   // its children come after it
    }
    __syncthreads();   // nobody reads the list
    if (tid == 0) s.inverse[times] = Z > 0.0 ? 1.0 / Z : 1.0;
    __syncthreads();
    ++times;
    if (Z > 0.0) Z = sum();   // else nothing will be left again
  }
  double all = sum();
  if (!(all > 0.0) && times > 0) {   // the target's own row
    times = 0;
    all = sum();
  }
  __syncthreads();   // the path is written
  if (rank == 0) {
    for (int i = tid; i < n; i += 32 * kWarps) a.path[q0 + i] = i < len ? s.path[i] : -1;
    if (tid == 0) a.path_len[b] = len;
    if (tid == 0 && !(all > 0.0)) a.next[b] = -1;
  }
  if (!(all > 0.0)) return;
  const double t = (double)__ldg(a.sample + b) * all;
  // the warp in whose run t is passed, or the last that holds anything
  double before = 0.0, up_to = 0.0;
  int owner = 0;
  for (int k = 0; k < ranks * kWarps; ++k) {
    const double x = share(k);
    if (x > 0.0) {
      owner = k;
      before = up_to;
    }
    up_to += x;
    if (x > 0.0 && up_to > t) break;
  }
  if (owner != rank * kWarps + warp) return;
  int answer = -1;
  for (int e0 = run0; e0 < run1; e0 += 32) {
    const double x = e0 + lane < run1 ? of_row(e0 + lane) : 0.0;
    __syncwarp();
    double y = x;
    for (int o = 1; o < 32; o <<= 1) {
      const double z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    y += before;
    const unsigned held = __ballot_sync(0xffffffffu, x > 0.0);
    const unsigned hit = __ballot_sync(0xffffffffu, x > 0.0 && y > t);
    if (held) answer = e0 + (hit ? __ffs(hit) - 1 : 31 - __clz(held));
    if (hit) break;
    before = __shfl_sync(0xffffffffu, y, 31);
  }
  if (lane == 0) a.next[b] = answer;
}

// kVec: rows begin on 16-byte boundaries.
template <typename T, bool kVec, int kThreads>
__global__ void __launch_bounds__(kThreads, kVerifyResident / kThreads)
    verify_tree_kernel(const __grid_constant__ VerifyArgs a, int ranks) {
  constexpr int kWarps = kThreads / 32, N = 16 / sizeof(T), kTile = 32 * N, kDepth = 8 / N;   // elements of a lane, of a warp; loads ahead
  __shared__ VerifyTree<kWarps> tree;
  auto &parent = tree.parent, &token = tree.token, &path = tree.path;
  auto &prob = tree.prob, &draft = tree.draft, &number = tree.number;
  auto& sums_of = tree.sums_of;
  __shared__ float2 threshold, owner_before;
  __shared__ float2 state_less;   // L
  __shared__ int state_node, state_len, state_sweep, state_out, row_left, owner_warp;
  enum { kNone, kSome, kLittleLeft };   // of a row; kSome of a walk: a pass is wanted
  extern __shared__ uint32_t out[];   // a bit for each token of the CTA's run
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / ranks, rank = blockIdx.x % ranks;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int q0 = __ldg(a.query_start + b), q1 = __ldg(a.query_start + b + 1);
  const bool good = q0 >= 0 && q1 >= q0 && q1 <= a.num_tokens && q1 - q0 <= a.max_query_len;
  const int n = q1 - q0;
  if (!good || n == 0) {   // alike in all of the cluster
    if (rank == 0 && tid == 0) {
      if (!good) raise_error(a.err, kErrQuery);
      a.path_len[b] = 0;
      a.next[b] = -1;
    }
    return;
  }
  cluster_arrive();   // this CTA has begun: its shared memory may be written to
  const T* target = static_cast<const T*>(a.target) + (int64_t)q0 * a.target_stride;
  const T* drafts = a.draft ? static_cast<const T*>(a.draft) + (int64_t)q0 * a.draft_stride : nullptr;
  const int V = a.vocab;
  // each warp's run, in whole tiles
  const int per_warp = ((V + ranks * kWarps - 1) / (ranks * kWarps) + kTile - 1) / kTile * kTile;
  const int64_t cta_begin = (int64_t)rank * kWarps * per_warp;
  const int run0 = (int)min((int64_t)V, cta_begin + (int64_t)warp * per_warp);
  const int run1 = (int)min((int64_t)V, cta_begin + (int64_t)(warp + 1) * per_warp);

  for (int i = tid; i < n; i += kThreads) {
    int up = __ldg(a.parents + q0 + i);
    int x = __ldg(a.tokens + q0 + i);
    if (up < -1 || up >= i || (x >= V && i > 0)) {   // (node 0's token is not used)
      if (rank == 0) raise_error(a.err, kErrTree);
      if (up < -1 || up >= i) up = -1;
    }
    if (x >= V || x < 0) x = -1;   // never accepted
    parent[i] = up;
    token[i] = x;
    number[i] = __ldg(a.accept + q0 + i);
    float p = 0.f, q = 1.f;
    if (up >= 0 && x >= 0) {
      p = as_prob(Elem<T>::to_f32(target[(int64_t)up * a.target_stride + x]));
      if (drafts) q = as_prob(Elem<T>::to_f32(drafts[(int64_t)up * a.draft_stride + x]));
    }
    prob[i] = p;
    draft[i] = q;
  }
  if (tid == 0) path[0] = 0;
  cluster_wait();   // and so have the others
  __syncthreads();
  if (!drafts) {
    // a sibling before it has the same token: nothing is left for it
    for (int i = tid; i < n; i += kThreads) {
      bool same = false;
      for (int j = 0; j < i; ++j) same |= parent[j] == parent[i] && token[j] == token[i];
      if (same) prob[i] = 0.f;
    }
    __syncthreads();
  }

  float2 less = make_float2(0.f, 0.f);   // L
  const T* prow = target;
  const T* qrow = drafts;
  bool marked = false;   // some tokens of the run are out

  // adds r of the N elements from e on, of chunks p and q
  auto add_left = [&](int e, uint4 pc, uint4 qc, Sums2& sum) {
    float p[N], q[N];
    Elem<T>::widen(pc, p);
    Elem<T>::widen(qc, q);
    if (marked && e < run1) {
      const uint32_t at = (uint32_t)(e - cta_begin);
      const uint32_t gone = out[at >> 5] >> (at & 31);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((gone >> i) & 1u) p[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 pp = make_float2(as_prob(p[i]), as_prob(p[i + 1]));
      Pair r = pair(pp.x, pp.y), l = 0;
      if (less.x != 0.f) left_of(pp, make_float2(as_prob(q[i]), as_prob(q[i + 1])), less.x, less.y, r, l);
      sum.add(r, l);
    }
  };
  auto load = [&](int e, uint4& p, uint4& q) {
    p = q = make_uint4(0u, 0u, 0u, 0u);
    if (e < run1) {
      p = load_chunk<T, kVec>(prow, e, V);
      if (less.x != 0.f) q = load_chunk<T, kVec>(qrow, e, V);
    }
  };
  int round = 0;
  Sum2 row;   // warp 0's
  // The sum of r over the row, into warp 0's `row`; the warps' sums are in sums_of[parity].
  auto sweep = [&]() {
    Sums2 sums;
    for (int e0 = run0 + lane * N; e0 < run1; e0 += kDepth * kTile) {
      uint4 p[kDepth], q[kDepth];
#pragma unroll
      for (int k = 0; k < kDepth; ++k) load(e0 + k * kTile, p[k], q[k]);
#pragma unroll
      for (int k = 0; k < kDepth; ++k) add_left(e0 + k * kTile, p[k], q[k], sums);
    }
    Sum2 sum = sums.both();
    sum.over(32);
    const int parity = round++ & 1;
    // every warp's sum to every CTA of the cluster
    if (lane < ranks) store_peer(&sums_of[parity][rank * kWarps + warp], lane, make_float2(sum.hi, sum.lo));
    cluster_arrive();
    cluster_wait();
    if (warp == 0) {
      Sum2 all;
      for (int k = lane; k < ranks * kWarps; k += 32) {
        const float2 s = sums_of[parity][k];
        all.add(s.x, s.y);
      }
      all.over(32);
      row = all;
      // L q and p have nearly all of their bits in common (never where L is 0)
      if (lane == 0) row_left = all.hi < kLittle * less.x ? kLittleLeft : all.positive() ? kSome : kNone;
    }
  };
  // ---- the walk: warp 0, up to the next pass that it needs.  Doubles are for one
  // warp at a time: at their rate the whole CTA's would take longer than a pass.
  int node = 0, last = 0, len = 1;
  Sum2 L, F;
  F.hi = 1.f;   // < 0: not known yet
  while (true) {
    if (warp == 0) {
      bool some = false;
      int want = kNone;
      while (true) {
        int taken = -1;
        some = false;   // a child of the node was rejected
        if (drafts) {
          // one child after another
          int j = n;
          for (int i0 = (last + 1) & ~31; i0 < n && j == n; i0 += 32) {
            const int i = i0 + lane;
            const unsigned hit = __ballot_sync(
                0xffffffffu, i > last && i < n && parent[i] == node && token[i] >= 0);
            if (hit) j = i0 + __ffs(hit) - 1;
          }
          if (j == n) break;
          if (F.hi < 0.f) {
            want = kSome;
            break;
          }
          if (F.hi < kLittle * L.hi) {
            want = kLittleLeft;
            break;
          }
          last = j;
          if (passes(prob[j], draft[j], L, number[j], F)) {
            taken = j;
          } else {
            L.add(F.hi, F.lo);
            L.settle();
            F.hi = -1.f;
            F.lo = 0.f;
            continue;
          }
        } else {
          // all children at once: before each, Z has lost what those before it had
          Sum2 lost, one;
          one.hi = 1.f;
          for (int i0 = (node + 1) & ~31; i0 < n && taken < 0; i0 += 32) {
            const int i = i0 + lane;
            const bool child = i > node && i < n && parent[i] == node && token[i] >= 0;
            if (!__any_sync(0xffffffffu, child)) continue;
            Sum2 mine;
            if (child) mine.hi = prob[i];
            const Sum2 up_to = prefix(lost, mine, lane);
            Sum2 z = one;   // 1 - what those before it had
            z.add(-up_to.hi, -up_to.lo);
            z.add(mine.hi, 0.f);
            if (!z.positive()) z = Sum2{};
            bool pass = child && passes(mine.hi, 1.f, Sum2{}, number[i], z);
            if (child && z.hi + z.lo < kLittle) {
              // of 48 bits few are left: in double, one after another
              double Z = 1.0;
              for (int j = node + 1; j < i; ++j)
                if (parent[j] == node && token[j] >= 0) Z = fmax(0.0, Z - (double)prob[j]);
              pass = (double)mine.hi > (double)number[i] * Z;
            }
            __syncwarp();
            const unsigned yes = __ballot_sync(0xffffffffu, pass);
            if (yes) taken = i0 + __ffs(yes) - 1;
            some = true;
            lost = of_lane(up_to, 31);
          }
          if (taken < 0) break;
        }
        if (lane == 0) path[len] = taken;
        ++len;
        node = last = taken;
        L = F = Sum2{};
        F.hi = 1.f;
      }
      if (lane == 0) {
        state_node = node;
        state_len = len;
        state_sweep = want;
        state_out = some;
        state_less = make_float2(L.hi, L.lo);
      }
    }
    __syncthreads();
    prow = target + (int64_t)state_node * a.target_stride;
    qrow = drafts + (int64_t)state_node * a.draft_stride;
    less = state_less;
    if (state_sweep == kNone) break;
    if (state_sweep == kLittleLeft) {
      finish_in_double<T, kWarps>(a, tree, b, ranks, state_node, state_len, round);
      return;
    }
    sweep();
    if (warp == 0) F = row;
  }

  // ---- the token that follows
  if (state_out) {
    // all of the node's children are out: mark them in the CTA's run
    const int words = (kWarps * per_warp + 31) / 32;
    for (int i = tid; i < words; i += kThreads) out[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const int64_t at = (int64_t)token[i] - cta_begin;
      if (parent[i] == state_node && token[i] >= 0 && at >= 0 &&
          at < (int64_t)kWarps * per_warp)
        atomicOr(&out[at >> 5], 1u << (at & 31));
    }
    __syncthreads();
    marked = true;
  }
  sweep();
  __syncthreads();
  if (row_left == kLittleLeft) {
    finish_in_double<T, kWarps>(a, tree, b, ranks, state_node, state_len, round);
    return;
  }
  if (!row_left && (marked || less.x != 0.f)) {   // nothing is left: the target's own row
    marked = false;
    less = make_float2(0.f, 0.f);
    __syncthreads();   // all have read row_left
    sweep();
    __syncthreads();
  }
  const int parity = (round - 1) & 1;
  if (rank == 0) {
    for (int i = tid; i < n; i += kThreads) a.path[q0 + i] = i < state_len ? path[i] : -1;
    if (tid == 0) a.path_len[b] = state_len;
    if (tid == 0 && !row_left) a.next[b] = -1;
  }
  if (!row_left) return;
  // The warp in whose run t is passed; rounding aside there is one, else the last
  // that holds anything.
  Sum2 t;
  auto chosen = [&](const Sum2& up_to, bool any) -> int {   // the lane, or -1 if none holds anything
    const unsigned held = __ballot_sync(0xffffffffu, any);
    const unsigned hit = __ballot_sync(0xffffffffu, any && up_to.above(t));
    return hit ? __ffs(hit) - 1 : held ? 31 - __clz(held) : -1;
  };
  if (warp == 0) {
    const float chance = __ldg(a.sample + b);
    t.hi = chance * row.hi;
    t.lo = fmaf(chance, row.hi, -t.hi) + chance * row.lo;
    Sum2 sum, at;
    int who = -1;
    for (int k0 = 0; k0 < ranks * kWarps; k0 += 32) {
      Sum2 mine;
      if (k0 + lane < ranks * kWarps) {
        mine.hi = sums_of[parity][k0 + lane].x;
        mine.lo = sums_of[parity][k0 + lane].y;
      }
      const Sum2 up_to = prefix(sum, mine, lane);
      const int k = chosen(up_to, mine.positive());
      if (k >= 0) {
        who = k0 + k;
        at = k > 0 ? of_lane(up_to, k - 1) : sum;
      }
      if (__any_sync(0xffffffffu, mine.positive() && up_to.above(t))) break;
      sum = of_lane(up_to, 31);
    }
    if (lane == 0) {
      owner_warp = who - rank * kWarps;   // another CTA's: none of this one's
      owner_before = make_float2(at.hi, at.lo);
      threshold = make_float2(t.hi, t.lo);
    }
  }
  __syncthreads();
  if (warp != owner_warp) return;
  t.hi = threshold.x;
  t.lo = threshold.y;
  Sum2 sum;
  sum.hi = owner_before.x;
  sum.lo = owner_before.y;
  // Each lane sums its share of the run, in order; then the warp goes through the
  // share in which t is passed.
  const int share = per_warp / 32;   // a multiple of N
  const int begin = run0 + lane * share, end = min(begin + share, run1);
  Sums2 sums;
  for (int e = begin; e < end; e += kDepth * N) {
    uint4 p[kDepth], q[kDepth];
#pragma unroll
    for (int k = 0; k < kDepth; ++k) load(e + k * N < end ? e + k * N : run1, p[k], q[k]);
#pragma unroll
    for (int k = 0; k < kDepth; ++k) add_left(e + k * N < end ? e + k * N : run1, p[k], q[k], sums);
  }
  const Sum2 own = sums.both();
  Sum2 up_to = prefix(sum, own, lane);
  const int lucky = max(0, chosen(up_to, own.positive()));
  if (lucky > 0) sum = of_lane(up_to, lucky - 1);
  const int from = run0 + lucky * share, to = min(from + share, run1);
  int answer = -1;
  for (int e0 = from; e0 < to; e0 += 32) {
    const int e = e0 + lane;
    Sum2 x;
    if (e < to) {
      float p = as_prob(Elem<T>::to_f32(prow[e])), q = 0.f;
      if (less.x != 0.f) q = as_prob(Elem<T>::to_f32(qrow[e]));
      const uint32_t at = (uint32_t)(e - cta_begin);
      if (marked && (out[at >> 5] >> (at & 31)) & 1u) p = 0.f;
      Pair r, l;
      left_of(make_float2(p, 0.f), make_float2(q, 0.f), less.x, less.y, r, l);
      x.hi = parts(r).x;
      x.lo = parts(l).x;
    }
    up_to = prefix(sum, x, lane);
    const int k = chosen(up_to, x.positive());
    if (k >= 0) answer = e0 + k;   // or the last one that holds anything, so far
    if (__any_sync(0xffffffffu, x.positive() && up_to.above(t))) break;
    sum = of_lane(up_to, 31);
  }
  if (lane == 0) a.next[b] = answer;
}

template <typename T, bool kVec, int kThreads>
cudaError_t launch_t(const VerifyArgs& a, cudaStream_t stream) {
  constexpr int kWarps = kThreads / 32;
  auto kern = verify_tree_kernel<T, kVec, kThreads>;
  // CTAs a sequence: as many as are all on the device at once (a little less than its
  // places, as a cluster's lie close together), or, where that is one or two, in two turns;
  // none with less than a tile a warp, and so many at least that the tokens' bits fit
  // shared memory.  One turn and two, 128256 chosen and 50000 drawn tokens: 80 sequences
  // 16.3, 14.7 and 18.2, 18.7 us; 128: 21.1, 20.0 and 21.6, 23.0; 160: 28.4, 25.2 and 28.5,
  // 28.1; 200: 48.7, 37.8 and 34.0, 29.3; 256: 54.2, 41.6 and 42.9, 39.1.
  constexpr int kTile = 512 / (int)sizeof(T);
  const int places = kVerifyResident / kThreads * a.num_sms * 97 / 100;
  const int least = (a.vocab + kVerifyRun - 1) / kVerifyRun;
  int ranks = places / a.B;
  if (ranks < 3) ranks = 2 * places / a.B;
  ranks = std::min(std::max(ranks, 1), kVerifyCluster);
  while (ranks > 1 && a.vocab <= ranks * kWarps * kTile) --ranks;
  ranks = std::max(ranks, least);
  const int run = kWarps * (((a.vocab + ranks * kWarps - 1) / (ranks * kWarps) + kTile - 1) / kTile * kTile);
  const size_t smem = a.draft ? 0 : (size_t)(run + 31) / 32 * 4;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, ranks);
}

template <typename T>
cudaError_t launch_rows(const VerifyArgs& a, cudaStream_t stream) {
  constexpr int N = 16 / (int)sizeof(T);
  const bool vec = (reinterpret_cast<uintptr_t>(a.target) & 15u) == 0 && a.target_stride % N == 0 &&
                   (!a.draft || ((reinterpret_cast<uintptr_t>(a.draft) & 15u) == 0 &&
                                 a.draft_stride % N == 0));
  // Larger CTAs while all of a full cluster's are on the device at once, else smaller
  // ones, of which they are (64 x 1 node over 128256 tokens: 16.5, 12.6 us; 38: 14.3, 12.5;
  // 32 x 1..48 chosen nodes over 99991: 11.7, 13.6).
  if ((int64_t)a.B * kVerifyCluster * 512 * 9 <= (int64_t)kVerifyResident * a.num_sms * 8)
    return vec ? launch_t<T, true, 512>(a, stream) : launch_t<T, false, 512>(a, stream);
  return vec ? launch_t<T, true, 256>(a, stream) : launch_t<T, false, 256>(a, stream);
}

}  // namespace

cudaError_t launch_verify_tree(const VerifyArgs& a, cudaStream_t stream) {
  switch (a.dtype) {
    case 0: return launch_rows<float>(a, stream);
    case 1: return launch_rows<__half>(a, stream);
    default: return launch_rows<__nv_bfloat16>(a, stream);
  }
}

}  // namespace photon
