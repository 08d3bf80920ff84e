// cache_compact.cu -- the accepted nodes' cached rows moved together behind the
// context, in the pools of every layer at once.
//
// PhotonInfer README, "Technical details / Paged attention" (one kernel for the
// K/V rows of many sequences); "Roadmap" (speculative decoding).
//
// Row j of a path of m nodes goes from position first + path[j] to first + j.
// path[j] >= j and both rise, so a thread that takes the same 16 bytes of every
// row and reads a few rows ahead of writing them never overwrites what it still
// has to read; threads do not meet.  Rows that stay are neither read nor written.
// It moves 2 m rows a sequence and pool: a launch for a step, memory for many layers.
//
// Measured: 4 sequences, 2 pools 2.4 us, a launch and four dependent loads; 64 sequences,
// 32 pools of 8 heads x 128 in 16 bits (20.7 MB moved) 5.9 us = 3.5 TB/s: the same, and
// then memory, in 3.1 us at the copy rate.
#include "speculate.cuh"

namespace photon {
namespace {

constexpr int kCompactThreads = 128;
constexpr int kCompactAhead = 8;   // rows read before the first of them is written

// grid (sequences, groups of pools): a CTA takes its sequence's rows in each pool
// of its group.
__global__ void __launch_bounds__(kCompactThreads)
    cache_compact_kernel(const __grid_constant__ CompactArgs a, int pools_each) {
  __shared__ int64_t from[kTreeNodes], to[kTreeNodes];   // rows (pool row = Hkv rows apart), -1: none
  __shared__ int bad;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int b = blockIdx.x, tid = threadIdx.x;
  const bool first_group = blockIdx.y == 0;
  const int q0 = __ldg(a.query_start + b), q1 = __ldg(a.query_start + b + 1);
  const int ctx = __ldg(a.context_lens + b), m = __ldg(a.path_len + b);
  if (q0 < 0 || q1 < q0 || q1 > a.num_tokens || q1 - q0 > a.max_query_len) {
    if (first_group && tid == 0) raise_error(a.err, kErrQuery);
    return;
  }
  const int n = q1 - q0;
  const bool bad_path = m < 0 || m > n;
  // (a sequence without nodes has no use for its context)
  if (bad_path || (n > 0 && (ctx < n || ctx > a.MBS * kBlockSize))) {
    if (first_group && tid == 0) raise_error(a.err, bad_path ? kErrTree : kErrContext);
    return;
  }
  if (m == 0) return;
  if (tid == 0) bad = 0;
  __syncthreads();
  const int first = ctx - n;
  const int32_t* table = a.block_tables + (int64_t)b * a.MBS;
  for (int j = tid; j < m; j += kCompactThreads) {
    const int node = __ldg(a.path + q0 + j);
    const int before = j > 0 ? __ldg(a.path + q0 + j - 1) : -1;
    if (node <= before || node >= n || node < 0) {
      atomicOr(&bad, (int)kErrTree);
      continue;
    }
    const int of = first + node, at = first + j;
    const int x = __ldg(table + of / kBlockSize), y = __ldg(table + at / kBlockSize);
    if (x < 0 || x >= a.NB || y < 0 || y >= a.NB) {
      atomicOr(&bad, (int)kErrBlock);
      continue;
    }
    from[j] = (int64_t)x * a.Hkv * kBlockSize + of % kBlockSize;
    to[j] = (int64_t)y * a.Hkv * kBlockSize + at % kBlockSize;
  }
  __syncthreads();
  if (bad) {   // the sequence is left as it is
    if (first_group && tid == 0) raise_error(a.err, (uint32_t)bad);
    return;
  }
  const int chunks = a.row_bytes / 16, columns = a.Hkv * chunks;
  const int p1 = min(a.num_pools, (int)(blockIdx.y + 1) * pools_each);
  for (int p = blockIdx.y * pools_each; p < p1; ++p) {
    unsigned char* pool = static_cast<unsigned char*>(a.pools[p]);
    for (int c = tid; c < columns; c += kCompactThreads) {
      unsigned char* column =
          pool + (int64_t)(c / chunks) * kBlockSize * a.row_bytes + (c % chunks) * 16;
      for (int j0 = 0; j0 < m; j0 += kCompactAhead) {
        uint4 held[kCompactAhead];
#pragma unroll
        for (int i = 0; i < kCompactAhead; ++i)
          if (j0 + i < m && from[j0 + i] != to[j0 + i])
            held[i] = *reinterpret_cast<const uint4*>(column + from[j0 + i] * a.row_bytes);
#pragma unroll
        for (int i = 0; i < kCompactAhead; ++i)
          if (j0 + i < m && from[j0 + i] != to[j0 + i])
            *reinterpret_cast<uint4*>(column + to[j0 + i] * a.row_bytes) = held[i];
      }
    }
  }
}

}  // namespace

cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t stream) {
  // enough CTAs for every SM to hold several; past that a CTA's pools share what it
  // has found out about its sequence
  const int want = (8 * a.num_sms + a.B - 1) / a.B;
  const int groups = a.num_pools < want ? a.num_pools : want;
  const int each = (a.num_pools + groups - 1) / groups;
  return launch_pdl(cache_compact_kernel, dim3(a.B, (a.num_pools + each - 1) / each),
                    dim3(kCompactThreads), 0, stream, a, each);
}

}  // namespace photon
