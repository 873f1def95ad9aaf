// Launch interface between the C-ABI layer and the sm_100a kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime_api.h>

#include <cstdint>

#include "mla_internal.h"

namespace mla {

// Kernel parameters of the attention kernel (the tensor maps travel beside them).
struct AttnParams {
  const WorkItem* work;
  const int32_t* kv_indices;
  const void* q_nope;  // bf16 [T*H, 512] (the kernel reads part of Q directly)
  const void* q_pe;    // bf16 [T*H, 64]; unused when rope_dim == 0
  const void* cache;   // bf16 [cache rows, 512 + rope_dim]
  void* out;         // bf16 [T*H, 512]
  float* lse;        // fp32 [T*H] or nullptr
  void* ws_o;        // bf16 (of a tree plan fp32) [partial rows, 512]
  float* ws_lse;     // fp32 [partial rows]
  int32_t* status;   // device status word
  int32_t* status_mirror;  // host-mapped pinned copy of the first error recorded, or null
  float scale_log2;  // sm_scale * log2(e)
  float nan_guard;   // always NaN: `x != nan_guard` is true for every x, yet the compiler
                     // cannot fold it, so a vote on it waits for x to be computed
  int32_t num_heads;
  int32_t page_size;
  int32_t box_rows;  // rows per KV box: min(page_size, 64)
  int32_t rope_dim;  // kpe width: 64, or 0 (cache rows are then 512 wide)
  uint64_t timeout_ns;
  int32_t debug_flags;
  const TreeItem* tree_items = nullptr;  // tree plans: beside work
  const uint64_t* tree_words = nullptr;
};

// Everything one attention launch needs; the launcher encodes the TMA tensor maps from
// the raw pointers, because their box shapes belong to the kernel's tiling.
struct AttnLaunch {
  AttnParams p;
  const void* q_nope;   // bf16 [rows, 512]
  const void* q_pe;     // bf16 [rows, 64] (null when rope_dim == 0)
  const void* cache;    // bf16 [cache_rows, 512 + rope_dim]
  uint64_t rows;        // T * H
  uint64_t cache_rows;  // num_pages * page_size
  int num_work;         // launch slots (CTA pairs)
  bool wait_prior_grid; // launched as a programmatic dependent of the previous kernel
                        // (an append): the key loads wait for that grid's writes
  bool few_rows = false;  // every batch row's queries leave lane quarters of a tile idle
};

struct MergeParams {
  const MergeItem* merge;
  const int32_t* refs;
  const void* ws_o;
  const float* ws_lse;
  void* out;
  float* lse;
  bool tree;  // of a tree plan
};

// Latent-cache append: token t's row of src goes to cache row rows[t] (skipped if < 0).
struct AppendParams {
  const int32_t* rows;  // [tokens]
  const void* src;      // bf16 [tokens, width]
  void* cache;          // bf16 [cache_rows, width]
  int32_t width;        // 512 + rope_dim
};

// Merge of two attention states by their log-sum-exps.
struct MergeStateParams {
  const void* out_a;
  const float* lse_a;
  const void* out_b;
  const float* lse_b;
  void* out;
  float* lse;  // may be null
  int64_t rows;
};

// Verification of drafted trees (mla_verify_tree).
struct VerifyParams {
  const TreeRow* rows;
  const TreeNode* nodes;
  const int32_t* draft_tokens;
  const void* target;
  const void* draft;  // may be null: point masses
  int64_t ld_target;
  int64_t ld_draft;
  int32_t vocab;
  const float* uniform;
  const float* uniform_next;
  int32_t* accept_index;
  int32_t* num_accepted;
  int32_t* next_token;
};

// Layers' caches named by one launch (they travel as kernel parameters).
constexpr int32_t kMaxCaches = 128;

// Move of the accepted nodes' rows (mla_compact_kv).
struct CompactParams {
  const TreeRow* rows;
  const int32_t* append_rows;  // [tokens]: every step token's cache row
  const int32_t* accept_index;
  const int32_t* num_accepted;
  int32_t width;  // 512 + rope_dim
  int32_t num_caches;
  void* caches[kMaxCaches];
};

// Page copies of one launch (mla_copy_pages).
struct CopyPair {
  int32_t src;
  int32_t dst;
  int32_t bytes;  // a multiple of the cache row's size
};
constexpr int32_t kMaxCopyPairs = 1024;
// Both lists travel as kernel parameters, and a launch pays for the parameters' size, so
// the few pairs of a fork have a smaller form.
template <int32_t kPairs, int32_t kCaches>
struct CopyParams {
  static constexpr int32_t max_pairs = kPairs, max_caches = kCaches;
  int64_t page_bytes;
  int32_t num_pairs;
  int32_t num_caches;
  void* caches[kCaches];
  CopyPair pairs[kPairs];
};
using CopyParamsSmall = CopyParams<64, 64>;  // 1.3 KB
using CopyParamsLarge = CopyParams<kMaxCopyPairs, kMaxCaches>;  // 13 KB

// cudaErrorInvalidValue when a tensor map cannot be encoded.
cudaError_t launch_attention(const AttnLaunch& a, cudaStream_t stream);
cudaError_t launch_merge(const MergeParams& p, int num_merge, cudaStream_t stream);
cudaError_t launch_append(const AppendParams& p, int num_tokens, cudaStream_t stream);
cudaError_t launch_merge_state(const MergeStateParams& p, cudaStream_t stream);
cudaError_t launch_verify(const VerifyParams& p, int rows, bool bf16, int num_sms, cudaStream_t stream);
cudaError_t launch_compact(const CompactParams& p, int rows, cudaStream_t stream);
// max_bytes: the largest pair of the launch
template <typename Params>
cudaError_t launch_copy_pages(const Params& p, int32_t max_bytes, cudaStream_t stream);

}  // namespace mla
