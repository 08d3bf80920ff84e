// verify_tree.cu -- rejection sampling of drafted trees against the target's
// probabilities, from given random numbers.
//
// PhotonInfer README, "Key features / GPU-optimized kernels" (zero-copy GPU
// sampling); "Roadmap" (speculative decoding).
//
// At node c with the target's p and the draft's q, r = p and Z = 1; a child x is
// accepted if r(x) > u Z q(x), else r <- max(0, r / Z - q), Z <- sum r.  With
// r / Z = (A p - B q)+ this is A <- A / Z, B <- B / Z + 1: one pair of numbers
// stands for the whole row, and a rejection costs one pass over two rows for Z,
// none if no sibling follows (the sampling pass finds the sum by itself).  Without
// q a child is a point mass: Z loses r(x), and the row needs no pass at all.
//
// What it answers are whole numbers, so what they hang on is held to about 48 bits:
// tests in double (one product and one comparison a child), row sums as pairs of
// floats whose rounding errors are carried along (two-sum), joined in double; the
// rate of doubles is too low for the rows themselves.
//
// A cluster of CTAs takes a sequence.  All of them walk the tree, each for itself,
// from the nodes' probabilities in shared memory; a pass over a row is cut into one
// run per CTA and warp, the sums meet through distributed shared memory, and the
// warp in whose run the sampled sum is passed goes through it once more (L2).  So
// a step is one launch, and even one sequence has several SMs to read with.
#include <math.h>

#include <algorithm>

#include "speculate.cuh"

namespace photon {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCluster = 8;   // most CTAs of a cluster
constexpr int kVerifyRun = kVerifyVocab / kVerifyCluster;   // most tokens of a CTA's run

// A sum held in two floats.
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x, float rest) {
    const float s = hi + x, b = s - hi;
    lo += ((hi - (s - b)) + (x - b)) + rest;
    hi = s;
  }
  __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
  // the sum over `lanes` neighbouring lanes, in all of them
  __device__ __forceinline__ void over(int lanes) {
    for (int o = 1; o < lanes; o <<= 1) {
      const float x = __shfl_xor_sync(0xffffffffu, hi, o), y = __shfl_xor_sync(0xffffffffu, lo, o);
      add(x, y);
    }
  }
};
// Inclusive prefix sums over a warp.
__device__ __forceinline__ double prefix(double x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// An entry as a probability: NaN and negative ones are 0, ones above 1 are 1.
__device__ __forceinline__ float as_prob(float x) { return fminf(fmaxf(x, 0.f), 1.f); }

// r = (A p - B q)+ of a row: mode 0 is p, 1 is p - q, 2 has A and B in two floats
// each; `out` marks the tokens of the CTA's run that count as 0 (mode 0 alone).
struct Rest {
  int mode;
  float ah, al, bh, bl;
  __device__ __forceinline__ void of(float p, float q, float& r, float& rest) const {
    rest = 0.f;
    if (mode == 0) {
      r = p;
    } else if (mode == 1) {
      r = p - q;
      rest = (p - r) - q;   // exact where p >= q
      if (!(r > 0.f)) r = rest = 0.f;
    } else {
      const float x = ah * p, y = bh * q;
      const float xl = fmaf(ah, p, -x) + al * p, yl = fmaf(bh, q, -y) + bl * q;
      r = x - y;
      const float b = r - x;
      rest = ((x - (r - b)) + (-y - b)) + (xl - yl);
      if (!(r + rest > 0.f)) r = rest = 0.f;
    }
  }
};

template <typename T, bool kVec>
__device__ __forceinline__ void load_probs(const T* row, int e, int vocab, float* f) {
  constexpr int N = 16 / sizeof(T);
  if (kVec && e + N <= vocab) {
    const uint4 c = __ldg(reinterpret_cast<const uint4*>(row + e));
    Elem<T>::widen(c, f);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = as_prob(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      f[i] = e + i < vocab ? as_prob(Elem<T>::to_f32(row[e + i])) : 0.f;
  }
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Stores a double into the same place of another CTA's shared memory.
__device__ __forceinline__ void store_peer(double* p, int rank, double v) {
  asm volatile(
      "{\n.reg .b32 at;\nmapa.shared::cluster.u32 at, %0, %1;\nst.shared::cluster.f64 [at], %2;\n}" ::
          "r"(smem_addr(p)),
      "r"(rank), "d"(v)
      : "memory");
}

// kVec: rows begin on 16-byte boundaries.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kVerifyThreads)
    verify_tree_kernel(const VerifyArgs a, int ranks) {
  constexpr int N = 16 / sizeof(T), kTile = 32 * N, kDepth = 2;   // elements of a lane, of a warp; loads ahead
  __shared__ int parent[kTreeNodes], token[kTreeNodes], path[kTreeNodes];
  __shared__ float prob[kTreeNodes], draft[kTreeNodes], number[kTreeNodes];
  __shared__ float2 warp_sum[kVerifyWarps];
  __shared__ double cta_sum[2][kVerifyCluster], row_sum;
  __shared__ double state_a, state_b, state_z, owner_before;
  __shared__ int owner_warp;
  __shared__ int state_node, state_last, state_len, state_sweep;
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
  const T* target = static_cast<const T*>(a.target) + (int64_t)q0 * a.target_stride;
  const T* drafts = a.draft ? static_cast<const T*>(a.draft) + (int64_t)q0 * a.draft_stride : nullptr;
  const int V = a.vocab;
  // each warp's run, in whole tiles
  const int per_warp = ((V + ranks * kVerifyWarps - 1) / (ranks * kVerifyWarps) + kTile - 1) / kTile * kTile;
  const int64_t cta_begin = (int64_t)rank * kVerifyWarps * per_warp;
  const int run0 = (int)min((int64_t)V, cta_begin + (int64_t)warp * per_warp);
  const int run1 = (int)min((int64_t)V, cta_begin + (int64_t)(warp + 1) * per_warp);

  for (int i = tid; i < n; i += kVerifyThreads) {
    int up = __ldg(a.parents + q0 + i);
    int x = __ldg(a.tokens + q0 + i);
    if (up < -1 || up >= i || x >= V) {
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
  if (tid == 0) {
    state_node = state_last = 0;
    state_len = 1;
    path[0] = 0;
    state_a = state_z = 1.0;
    state_b = 0.0;
  }
  __syncthreads();

  Rest rest{};
  const T* prow = target;
  const T* qrow = drafts;
  bool marked = false;   // some tokens of the run are out

  // r of the N elements from e on, whose sum is wanted
  auto left = [&](int e, const float* p, const float* q, float* r, float* l) {
    uint32_t gone = 0;
    if (marked && e < run1) {
      const uint32_t at = (uint32_t)(e - cta_begin);
      gone = out[at >> 5] >> (at & 31);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      rest.of((gone >> i) & 1u ? 0.f : p[i], q[i], r[i], l[i]);
    }
  };
  auto load = [&](int e, float* p, float* q) {
    if (e < run1) {
      load_probs<T, kVec>(prow, e, V, p);
      if (rest.mode > 0) load_probs<T, kVec>(qrow, e, V, q);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] = q[i] = 0.f;
    }
    if (rest.mode == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) q[i] = 0.f;
    }
  };
  int round = 0;
  // The sum of r over the row; the CTAs' sums are in cta_sum[parity], the warps' in
  // warp_sum.
  auto sweep = [&]() -> double {
    Sum2 sum;
    for (int e0 = run0 + lane * N; e0 < run1; e0 += kDepth * kTile) {
      float p[kDepth][N], q[kDepth][N];
#pragma unroll
      for (int k = 0; k < kDepth; ++k) load(e0 + k * kTile, p[k], q[k]);
#pragma unroll
      for (int k = 0; k < kDepth; ++k) {
        float r[N], l[N];
        left(e0 + k * kTile, p[k], q[k], r, l);
#pragma unroll
        for (int i = 0; i < N; ++i) sum.add(r[i], l[i]);
      }
    }
    sum.over(32);
    const int parity = round++ & 1;
    if (lane == 0) warp_sum[warp] = make_float2(sum.hi, sum.lo);
    __syncthreads();
    if (warp == 0) {
      Sum2 all;
      if (lane < kVerifyWarps) {
        all.hi = warp_sum[lane].x;
        all.lo = warp_sum[lane].y;
      }
      all.over(kVerifyWarps);
      if (lane < ranks) store_peer(&cta_sum[parity][rank], lane, all.value());
    }
    cluster_sync();
    if (warp == 0) {
      double total = lane < ranks ? cta_sum[parity][lane] : 0.0;
#pragma unroll
      for (int o = 1; o < kVerifyCluster; o <<= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      if (lane == 0) row_sum = total;
    }
    __syncthreads();
    return row_sum;
  };
  auto take_rest = [&](double A, double B) {
    rest.mode = B == 0.0 ? 0 : (A == 1.0 && B == 1.0 ? 1 : 2);
    rest.ah = (float)A;
    rest.al = (float)(A - (double)rest.ah);
    rest.bh = (float)B;
    rest.bl = (float)(B - (double)rest.bh);
  };

  // ---- the walk: warp 0, up to the next pass that it needs
  while (true) {
    if (warp == 0) {
      int node = state_node, last = state_last, len = state_len;
      double A = state_a, B = state_b, Z = state_z;
      int want = 0;
      while (true) {
        // the node's next child
        int j = n;
        for (int i0 = (last + 1) & ~31; i0 < n && j == n; i0 += 32) {
          const int i = i0 + lane;
          const unsigned hit = __ballot_sync(0xffffffffu, i > last && i < n && parent[i] == node);
          if (hit) j = i0 + __ffs(hit) - 1;
        }
        if (j == n) break;
        if (token[j] < 0) {   // no token
          last = j;
          continue;
        }
        if (Z < 0.0) {   // not known yet: the sum of what a rejection left
          want = 1;
          break;
        }
        last = j;
        double r = (double)prob[j], q = 1.0;
        if (drafts) {
          q = (double)draft[j];
          r = fmax(A * r - B * q, 0.0);
        } else if (B != 0.0) {   // a sibling before it had the same token
          bool same = false;
          for (int i = lane; i < j; i += 32) same |= parent[i] == node && token[i] == token[j];
          if (__any_sync(0xffffffffu, same)) r = 0.0;
        }
        if (r > (double)number[j] * Z * q) {
          if (lane == 0) path[len] = j;
          ++len;
          node = j;
          A = Z = 1.0;
          B = 0.0;
        } else if (drafts) {
          const double safe = Z > 0.0 ? Z : 1.0;
          A = A / safe;
          B = B / safe + 1.0;
          Z = -1.0;
        } else {
          Z = fmax(Z - r, 0.0);
          B = 1.0;   // tokens are out
        }
      }
      if (lane == 0) {
        state_node = node;
        state_last = last;
        state_len = len;
        state_a = A;
        state_b = B;
        state_z = Z;
        state_sweep = want;
      }
    }
    __syncthreads();
    if (!state_sweep) break;
    prow = target + (int64_t)state_node * a.target_stride;
    qrow = drafts + (int64_t)state_node * a.draft_stride;
    take_rest(state_a, state_b);
    const double z = sweep();
    if (tid == 0) state_z = z;
    __syncthreads();
  }

  // ---- the token that follows
  const int node = state_node, len = state_len;
  prow = target + (int64_t)node * a.target_stride;
  if (drafts) {
    qrow = drafts + (int64_t)node * a.draft_stride;
    take_rest(state_a, state_b);
  } else {
    rest.mode = 0;
    if (state_b != 0.0) {
      // all of the node's children are out: mark them in the CTA's run
      const int words = (kVerifyWarps * per_warp + 31) / 32;
      for (int i = tid; i < words; i += kVerifyThreads) out[i] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += kVerifyThreads) {
        const int64_t at = (int64_t)token[i] - cta_begin;
        if (parent[i] == node && token[i] >= 0 && at >= 0 && at < (int64_t)kVerifyWarps * per_warp)
          atomicOr(&out[at >> 5], 1u << (at & 31));
      }
      __syncthreads();
      marked = true;
    }
  }
  double total = sweep();
  if (!(total > 0.0) && (marked || rest.mode != 0)) {   // nothing is left: the target's own row
    marked = false;
    rest.mode = 0;
    total = sweep();
  }
  const int parity = (round - 1) & 1;
  const float chance = __ldg(a.sample + b);
  const double t = (double)chance * total;
  if (rank == 0) {
    for (int i = tid; i < n; i += kVerifyThreads) a.path[q0 + i] = i < len ? path[i] : -1;
    if (tid == 0) a.path_len[b] = len;
    if (tid == 0 && !(total > 0.0)) a.next[b] = -1;
  }
  if (!(total > 0.0)) return;
  // The CTA in whose run t is passed, and there the warp; rounding aside there is
  // one, else the last that holds anything.
  if (warp == 0) {
    auto passed = [&](double mine, double before, double& at) -> int {
      const double up_to = before + prefix(mine, lane);
      unsigned hit = __ballot_sync(0xffffffffu, up_to > t && mine > 0.0);
      if (!hit) hit = 0x80000000u >> __clz(__ballot_sync(0xffffffffu, mine > 0.0));
      const int k = __ffs(hit) - 1;
      at = __shfl_sync(0xffffffffu, up_to - mine, k);
      return k;
    };
    double at = 0.0;
    int who = passed(lane < ranks ? cta_sum[parity][lane] : 0.0, 0.0, at);
    if (who == rank) {
      Sum2 mine;
      if (lane < kVerifyWarps) {
        mine.hi = warp_sum[lane].x;
        mine.lo = warp_sum[lane].y;
      }
      who = passed(mine.value(), at, at);
    } else {
      who = -1;
    }
    if (lane == 0) {
      owner_warp = who;
      owner_before = at;
    }
  }
  __syncthreads();
  if (warp != owner_warp) return;
  double sum = owner_before;
  int answer = -1, positive = -1;   // where t is passed; the last one that holds anything
  for (int e0 = run0; e0 < run1 && answer < 0; e0 += kTile) {
    const int e = e0 + lane * N;
    float p[N], q[N], r[N], l[N];
    load(e, p, q);
    left(e, p, q, r, l);
    Sum2 own;
#pragma unroll
    for (int i = 0; i < N; ++i) own.add(r[i], l[i]);
    const double held = own.value(), scan = prefix(held, lane);
    int highest = -1;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (r[i] + l[i] > 0.f) highest = e + i;
    const unsigned hit = __ballot_sync(0xffffffffu, sum + scan > t && highest >= 0);
    if (hit) {
      const int from = __ffs(hit) - 1;
      int found = highest;
      if (lane == from) {
        double c = sum + (scan - held);
        bool yet = false;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          c += (double)r[i] + (double)l[i];
          if (!yet && r[i] + l[i] > 0.f && c > t) {
            found = e + i;
            yet = true;
          }
        }
      }
      answer = __shfl_sync(0xffffffffu, found, from);
    }
    positive = max(positive, __reduce_max_sync(0xffffffffu, highest));
    sum += __shfl_sync(0xffffffffu, scan, 31);
  }
  if (lane == 0) a.next[b] = answer >= 0 ? answer : positive;
}

template <typename T, bool kVec>
cudaError_t launch_t(const VerifyArgs& a, cudaStream_t stream) {
  auto kern = verify_tree_kernel<T, kVec>;
  // as many CTAs a sequence as the device holds at once, but none with less than a
  // tile or two a warp
  constexpr int kTile = 512 / (int)sizeof(T);
  int ranks = 1;
  while (ranks < kVerifyCluster &&
         (a.vocab > ranks * kVerifyRun ||   // the tokens' bits fit shared memory
          (a.B * ranks < 4 * a.num_sms && a.vocab > 2 * ranks * kVerifyWarps * kTile)))
    ranks *= 2;
  const int run = kVerifyWarps * (((a.vocab + ranks * kVerifyWarps - 1) / (ranks * kVerifyWarps) + kTile - 1) / kTile * kTile);
  const size_t smem = a.draft ? 0 : (size_t)(run + 31) / 32 * 4;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * ranks));
  cfg.blockDim = dim3(kVerifyThreads);
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
  return vec ? launch_t<T, true>(a, stream) : launch_t<T, false>(a, stream);
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
