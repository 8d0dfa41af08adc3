// prompt_common.cuh -- the launch records of msa_prompt.h's operators.
#pragma once

#include "msa_internal.cuh"
#include "msa_prompt.h"

namespace msa {

// Largest group of query heads on one KV head (a tile of 128 rows holds a
// token's whole group) and number of KV heads.
constexpr int kMaxGroup = 128;
constexpr int kMaxKvHeads = 64;

// One tile pair whose blocks are shared by several CTAs (written by the second
// of them): partials of CTAs c - 1 .. last.
struct PromptSplit {
  int32_t nrows;  // rows x group; 0: none
  int32_t row0;   // first row in the batch
  int32_t head;   // KV head
  int32_t last;
};

struct PromptLaunch {
  msa_batch batch;
  const uint16_t* q;
  int num_heads, num_kv_heads;
  const uint8_t* k;
  const uint8_t* v;
  int kv_fp8, scale_mode;
  const float* k_scale;
  const float* v_scale;
  const float* sinks;
  float softmax_scale;
  uint16_t* out;
  float* lse;
  uint32_t* status;
  bool whole;          // a pair to a CTA, none split
  PromptSplit* split;  // [grid]
  int32_t* part_bad;   // [2 * grid]
  float2* part_ml;     // [2 * grid, 256]
  float* part_o;       // [2 * grid, 32, 256, 4]
};
cudaError_t launch_prompt_attn(const PromptLaunch& p, cudaStream_t stream);

// One vector kind of the insertion: `heads` vectors of `dim` a row
struct RopeVec {
  const uint16_t* src;
  long long stride;  // elements from row to row
  int heads, dim;
  const uint16_t* norm;  // [dim], or null
};
struct RopeLaunch {
  msa_batch batch;
  RopeVec q, k, v, idx_q, idx_k;
  float eps, shift;
  const float* cos_sin;
  int max_pos, rotary, near;
  const int32_t* positions;
  uint16_t* q_out;
  uint16_t* idx_q_out;
  uint8_t* k_cache;
  uint8_t* v_cache;
  int kv_fp8, scale_mode;
  float* k_scale;
  float* v_scale;
  uint8_t* idx_cache;
  int idx_fp8;
  float* idx_scale;
  float* mass;
  uint32_t* status;
};
cudaError_t launch_qk_rope_insert(const RopeLaunch& p, cudaStream_t stream);

struct ForkLaunch {
  msa_cache_view from;
  const int32_t* refs;
  const int32_t* parent;
  const int32_t* grow;
  msa_page_set to;
  uint32_t* status;
};
cudaError_t launch_page_fork(const ForkLaunch& p, cudaStream_t stream);

// One array of a layer as the copy sees it: rows of `row` bytes per token
struct CopyPool {
  uint8_t* base;
  int row;
};
constexpr int kCopyPools = 240;  // of one launch (kernel parameters of 4 KB)
struct CopyLaunch {
  const int32_t* src;
  const int32_t* dst;
  const int32_t* tokens;
  int num_copies, num_pages, num_pools;
  CopyPool pool[kCopyPools];
  uint32_t* status;
};
cudaError_t launch_page_copy(const CopyLaunch& p, cudaStream_t stream);

}  // namespace msa
