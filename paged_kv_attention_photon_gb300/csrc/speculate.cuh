// speculate.cuh -- launch arguments of a speculative step's operators: rotation on
// the way into the cache, attention of drafted trees, their verification, and the
// accepted rows' move.
#pragma once

#include "photon_common.cuh"

namespace photon {

enum : uint32_t { kErrTree = 64u };
// Most nodes of a sequence's tree.
constexpr int kTreeNodes = 256;

struct RopeAppendArgs {
  const void* q;              // null: keys and values alone (Hq is 0 then)
  const void* k;
  const void* v;
  const int32_t* positions;   // [T]
  const float2* cs;           // [max_pos][half] (cos, sin)
  const int64_t* slots;       // [T]
  void* q_out;
  void* k_cache;
  void* v_cache;
  uint32_t* err;
  int64_t q_stride, k_stride, v_stride, q_out_stride;   // elements from token to token
  int T, Hq, Hkv, D, NB, max_pos, dtype;
  int half;                   // pairs that turn: rotary_dim / 2
  int interleaved;            // a pair is two neighbours, not two elements half a rotary_dim apart
};
cudaError_t launch_rope_append(const RopeAppendArgs& a, cudaStream_t stream);

struct TreeArgs {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;   // [B + 1]
  const int32_t* parents;       // [num_tokens]
  void* out;
  int4* ws_split;  // [CTA][2] the pair that its run begins in the midst of: first row of q,
                   // nodes, KV head, row group; first and last CTA (last -1: none)
  float2* ws_ml;   // [row] maximum (unscaled) and sum of weights of a partial ..
  float* ws_o;     // [row][D] .. and its weighted V sum
  uint32_t* err;
  float qscale;    // scale * log2(e)
  int B, Hq, Hkv, D, NB, MBS, num_tokens, max_query_len, dtype, num_sms;
  // set by launch_tree_attention: whether pairs are split over CTAs; up to how many chunks
  // one tile takes an item alone
  bool split;
  int one_tile;
};
cudaError_t launch_tree_attention(const TreeArgs& a, cudaStream_t stream);
// Query rows of a group: what one CTA holds at a time.
constexpr int kTreeRows = 256;
// Most CTAs of the attention grid: each has kTreeRows rows of partials in the
// workspace, whose size so does not depend on the device.
constexpr int kTreeMaxCtas = 160;
// Keys of a chunk, and the chunks that beginning and ending a pair counts for.  With 1,
// 2, 3, 4: a batch-256 mix 204, 193, 200, 205 us, 64 long contexts 93.9, 94.6, 95.6,
// 97.7, 32 contexts x 256 rows 59.8, 57.9, 57.9, 60.4.
constexpr int kTreeChunk = 128;
constexpr int kTreePairCost = 2;

// Largest vocabulary.
constexpr int kVerifyVocab = 1 << 20;

struct VerifyArgs {
  const void* target;      // [num_tokens] rows of `vocab` probabilities
  const void* draft;       // the same, or null
  int64_t target_stride, draft_stride;
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* query_start;
  const float* accept;     // [num_tokens]
  const float* sample;     // [B]
  int32_t* path;           // [num_tokens]
  int32_t* path_len;       // [B]
  int32_t* next;           // [B]
  uint32_t* err;
  int B, num_tokens, max_query_len, vocab, dtype, num_sms;
};
cudaError_t launch_verify_tree(const VerifyArgs& a, cudaStream_t stream);

// Pools of one call: their addresses travel with the launch.
constexpr int kCompactPools = 256;
struct CompactArgs {
  void* pools[kCompactPools];
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  const int32_t* path;
  const int32_t* path_len;
  uint32_t* err;
  int num_pools, B, Hkv, row_bytes, NB, MBS, num_tokens, max_query_len, num_sms;
};
cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t stream);

}  // namespace photon
