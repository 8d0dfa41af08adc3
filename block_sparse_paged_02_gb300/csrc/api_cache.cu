// api_cache.cu -- the entry points of msa_cache.h: argument checks, workspace
// layout and launches.  As in api.cu nothing here touches device data or
// synchronises.
#include "tree_common.cuh"

namespace msa {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
msa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA; }

int rows_bound(int num_rows, int max_q_len) {
  if (max_q_len > 0) return max_q_len;
  return num_rows < 1 ? 1 : num_rows < MSA_TREE_MAX_ROWS ? num_rows : MSA_TREE_MAX_ROWS;
}

struct TreeWs {
  int list_cap, list_words;
  size_t list_count, list_blk, list_rows, split, part_bad, part_ml, part_o, total;
};

TreeWs tree_layout(int num_reqs, int bt_stride, int num_heads, int max_rows, int topk) {
  TreeWs w;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = round_up(off + bytes, 256);
    return at;
  };
  const size_t grid = (size_t)device_sm_count(), tile = (size_t)tree_part_rows(max_rows, num_heads);
  w.list_cap = w.list_words = 0;
  w.list_count = w.list_blk = w.list_rows = 0;
  if (topk > 0) {
    // every row's selection, and the blocks from the context's last one on
    const long long most = (long long)max_rows * topk + (max_rows + kBlock - 1) / kBlock + 1;
    w.list_cap = most < bt_stride ? (int)most : bt_stride;
    w.list_words = (max_rows + 31) / 32;
    w.list_count = take((size_t)num_reqs * 4);
    w.list_blk = take((size_t)num_reqs * w.list_cap * 4);
    w.list_rows = take((size_t)num_reqs * w.list_cap * w.list_words * 4);
  }
  w.split = take(grid * sizeof(TreeSplit));
  w.part_bad = take(2 * grid * 4);
  w.part_ml = take(2 * grid * tile * 8);
  w.part_o = take(2 * grid * tile * kHeadDim * 4);
  w.total = off;
  return w;
}

// Checks shared by the attention and the weight accumulation
msa_status check_tree(const msa_batch* b, const msa_tree* t, const msa_attn_args* a,
                      const void* status) {
  if (!b || !t || !a || !status) return MSA_ERR_NULL;
  if (b->num_reqs < 0 || b->num_rows < 0 || b->num_pages < 0 || b->bt_stride < 1 ||
      b->max_q_len < 0)
    return MSA_ERR_SHAPE;
  if (!b->cu_seqlens_q) return MSA_ERR_NULL;
  if (b->num_reqs > 0 && (!b->cu_seqlens_k || !b->context_lens || !b->block_table))
    return MSA_ERR_NULL;
  if (b->num_reqs > kMaxReqs || b->bt_stride > kMaxBlocksPerRow) return MSA_ERR_UNSUPPORTED;
  if (b->max_q_len > MSA_TREE_MAX_ROWS) return MSA_ERR_UNSUPPORTED;
  if (a->kv_dtype != MSA_KV_BF16 && a->kv_dtype != MSA_KV_FP8_E4M3) return MSA_ERR_DTYPE;
  if (a->scale_mode < MSA_SCALE_NONE || a->scale_mode > MSA_SCALE_PER_TOKEN_HEAD)
    return MSA_ERR_DTYPE;
  if (a->num_heads < 1 || a->num_kv_heads < 1 || a->num_heads % a->num_kv_heads != 0)
    return MSA_ERR_SHAPE;
  if (a->num_rows != b->num_rows || a->num_pages != b->num_pages) return MSA_ERR_SHAPE;
  if (a->num_kv_heads != 1 || a->head_dim != kHeadDim || a->num_heads > kMaxHeads)
    return MSA_ERR_UNSUPPORTED;
  if (t->mask && t->mask_words < 1) return MSA_ERR_SHAPE;
  if (t->topk_idx && t->topk < 1) return MSA_ERR_SHAPE;
  if (t->topk_idx && t->topk > kMaxTopk) return MSA_ERR_UNSUPPORTED;
  if (!aligned16(t->mask) || !aligned16(t->topk_idx)) return MSA_ERR_SHAPE;
  if (b->num_rows > 0) {
    if (!a->q || !a->k_cache || !a->lse) return MSA_ERR_NULL;
    if (a->scale_mode != MSA_SCALE_NONE && !a->k_scale) return MSA_ERR_NULL;
  }
  if (!aligned16(a->q) || !aligned16(a->k_cache) || !aligned16(a->lse)) return MSA_ERR_SHAPE;
  if (a->scale_mode == MSA_SCALE_PER_TOKEN_HEAD && !aligned16(a->k_scale)) return MSA_ERR_SHAPE;
  return MSA_OK;
}

// The launch record on a checked call's workspace
msa_status make_tree(const msa_batch* b, const msa_tree* t, const msa_attn_args* a, void* workspace,
                     size_t workspace_bytes, uint32_t* status, TreeLaunch* p) {
  const int max_rows = rows_bound(b->num_rows, b->max_q_len);
  const TreeWs w = tree_layout(b->num_reqs, b->bt_stride, a->num_heads, max_rows,
                               t->topk_idx ? t->topk : 0);
  if (!workspace || workspace_bytes < w.total || !aligned16(workspace)) return MSA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p->batch = *b;
  p->mask = t->mask;
  p->mask_words = t->mask_words;
  p->topk_idx = t->topk_idx;
  p->topk = t->topk;
  p->q = static_cast<const uint16_t*>(a->q);
  p->num_heads = a->num_heads;
  p->k = static_cast<const uint8_t*>(a->k_cache);
  p->v = static_cast<const uint8_t*>(a->v_cache);
  p->kv_fp8 = a->kv_dtype == MSA_KV_FP8_E4M3;
  p->scale_mode = a->scale_mode;
  p->k_scale = a->k_scale;
  p->v_scale = a->v_scale;
  p->sinks = a->sinks;
  p->softmax_scale = a->softmax_scale;
  p->out = static_cast<uint16_t*>(a->out);
  p->lse = a->lse;
  p->mass = nullptr;
  p->status = status;
  p->max_rows = max_rows;
  p->list_cap = w.list_cap;
  p->list_words = w.list_words;
  p->list_count = reinterpret_cast<int32_t*>(ws + w.list_count);
  p->list_blk = reinterpret_cast<int32_t*>(ws + w.list_blk);
  p->list_rows = reinterpret_cast<uint32_t*>(ws + w.list_rows);
  p->split = reinterpret_cast<TreeSplit*>(ws + w.split);
  p->part_bad = reinterpret_cast<int32_t*>(ws + w.part_bad);
  p->part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
  p->part_o = reinterpret_cast<float*>(ws + w.part_o);
  return MSA_OK;
}

msa_status check_view(const msa_cache_view* c, const void* status) {
  if (!c || !status) return MSA_ERR_NULL;
  if (c->num_reqs < 0 || c->num_pages < 0 || c->bt_stride < 1) return MSA_ERR_SHAPE;
  if (c->num_reqs > kMaxReqs || c->bt_stride > kMaxBlocksPerRow) return MSA_ERR_UNSUPPORTED;
  if (c->num_reqs > 0 && (!c->lens || !c->block_table)) return MSA_ERR_NULL;
  return MSA_OK;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

size_t msa_tree_attn_workspace_size(int32_t num_reqs, int32_t num_rows, int32_t bt_stride,
                                    int32_t num_heads, int32_t max_q_len, int32_t topk) {
  if (num_reqs < 0 || num_rows < 0 || bt_stride < 1 || num_heads < 1 || num_heads > kMaxHeads ||
      max_q_len < 0 || max_q_len > MSA_TREE_MAX_ROWS || topk < 0 || topk > kMaxTopk)
    return 0;
  return tree_layout(num_reqs, bt_stride, num_heads, rows_bound(num_rows, max_q_len), topk).total;
}

msa_status msa_tree_attn(const msa_batch* batch, const msa_tree* tree, const msa_attn_args* attn,
                         void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                         cudaStream_t stream) {
  msa_status st = check_tree(batch, tree, attn, dev_status);
  if (st != MSA_OK) return st;
  if (batch->num_rows > 0) {
    if (!attn->v_cache || !attn->out) return MSA_ERR_NULL;
    if (attn->scale_mode != MSA_SCALE_NONE && !attn->v_scale) return MSA_ERR_NULL;
  }
  if (!aligned16(attn->v_cache) || !aligned16(attn->out)) return MSA_ERR_SHAPE;
  if (attn->scale_mode == MSA_SCALE_PER_TOKEN_HEAD && !aligned16(attn->v_scale))
    return MSA_ERR_SHAPE;
  if (batch->num_rows == 0) return MSA_OK;
  if (batch->num_reqs == 0) return MSA_ERR_SHAPE;  // rows without any request
  TreeLaunch p;
  st = make_tree(batch, tree, attn, workspace, workspace_bytes, dev_status, &p);
  if (st != MSA_OK) return st;
  return cuda_status(launch_tree_attn(p, stream));
}

msa_status msa_attn_mass(const msa_batch* batch, const msa_tree* tree, const msa_attn_args* attn,
                         float* mass, void* workspace, size_t workspace_bytes,
                         uint32_t* dev_status, cudaStream_t stream) {
  msa_status st = check_tree(batch, tree, attn, dev_status);
  if (st != MSA_OK) return st;
  if (batch->num_rows > 0 && !mass) return MSA_ERR_NULL;
  if (!aligned16(mass)) return MSA_ERR_SHAPE;
  if (batch->num_rows == 0) return MSA_OK;
  if (batch->num_reqs == 0) return MSA_ERR_SHAPE;
  TreeLaunch p;
  st = make_tree(batch, tree, attn, workspace, workspace_bytes, dev_status, &p);
  if (st != MSA_OK) return st;
  p.mass = mass;
  return cuda_status(launch_attn_mass(p, stream));
}

msa_status msa_evict_select(const msa_cache_view* cache, const float* mass, int32_t budget,
                            int32_t keep_first, int32_t keep_recent, int32_t* keep,
                            int32_t* keep_len, uint32_t* dev_status, cudaStream_t stream) {
  const msa_status st = check_view(cache, dev_status);
  if (st != MSA_OK) return st;
  if (budget < 1 || keep_first < 0 || keep_recent < 0 ||
      (int64_t)keep_first + keep_recent > budget)
    return MSA_ERR_SHAPE;
  if (cache->num_reqs == 0) return MSA_OK;
  if (!mass || !keep || !keep_len) return MSA_ERR_NULL;
  if (!aligned16(mass) || !aligned16(keep) || !aligned16(keep_len)) return MSA_ERR_SHAPE;
  EvictLaunch p{*cache, mass, budget, keep_first, keep_recent, keep, keep_len, dev_status};
  return cuda_status(launch_evict_select(p, stream));
}

msa_status msa_kv_compact(const msa_cache_view* cache, const int32_t* base, const int32_t* keep,
                          int32_t keep_stride, const int32_t* keep_len, const msa_kv_pools* pools,
                          uint32_t* dev_status, cudaStream_t stream) {
  const msa_status st = check_view(cache, dev_status);
  if (st != MSA_OK) return st;
  if (!pools) return MSA_ERR_NULL;
  if (pools->kv_dtype != MSA_KV_BF16 && pools->kv_dtype != MSA_KV_FP8_E4M3) return MSA_ERR_DTYPE;
  if (pools->scale_mode < MSA_SCALE_NONE || pools->scale_mode > MSA_SCALE_PER_TOKEN_HEAD)
    return MSA_ERR_DTYPE;
  if (pools->num_kv_heads < 1 || keep_stride < 1) return MSA_ERR_SHAPE;
  if (pools->head_dim != kHeadDim || pools->num_kv_heads > 64) return MSA_ERR_UNSUPPORTED;
  const msa_index_cache* x = pools->index;
  if (x) {
    if (x->dtype != MSA_KV_BF16 && x->dtype != MSA_KV_FP8_E4M3) return MSA_ERR_DTYPE;
    if (!((x->heads == 1 && (x->dim == 64 || x->dim == 128)) || (x->heads == 2 && x->dim == 64)))
      return MSA_ERR_UNSUPPORTED;
  }
  if (cache->num_reqs == 0) return MSA_OK;
  const bool token_scales = pools->scale_mode == MSA_SCALE_PER_TOKEN_HEAD;
  if (!keep || !keep_len || !pools->k_cache || !pools->v_cache) return MSA_ERR_NULL;
  if (token_scales && (!pools->k_scale || !pools->v_scale)) return MSA_ERR_NULL;
  if (x && !x->k_cache) return MSA_ERR_NULL;
  if (!aligned16(pools->k_cache) || !aligned16(pools->v_cache) || !aligned16(keep) ||
      !aligned16(pools->mass) || (token_scales && (!aligned16(pools->k_scale) || !aligned16(pools->v_scale))) ||
      (x && (!aligned16(x->k_cache) || !aligned16(x->k_scale))))
    return MSA_ERR_SHAPE;
  CompactLaunch p = {};
  p.cache = *cache;
  p.base = base;
  p.keep = keep;
  p.keep_stride = keep_stride;
  p.keep_len = keep_len;
  p.status = dev_status;
  const int h = pools->num_kv_heads;
  const int row = h * kHeadDim * (pools->kv_dtype == MSA_KV_FP8_E4M3 ? 1 : 2);
  p.pool[0] = {static_cast<uint8_t*>(pools->k_cache), row};
  p.pool[1] = {static_cast<uint8_t*>(pools->v_cache), row};
  if (x) p.pool[2] = {static_cast<uint8_t*>(x->k_cache), x->heads * x->dim * (x->dtype == MSA_KV_FP8_E4M3 ? 1 : 2)};
  if (token_scales) {
    p.pool[3] = {reinterpret_cast<uint8_t*>(pools->k_scale), 4 * h};
    p.pool[4] = {reinterpret_cast<uint8_t*>(pools->v_scale), 4 * h};
  }
  if (x && x->dtype == MSA_KV_FP8_E4M3 && x->k_scale)
    p.pool[5] = {reinterpret_cast<uint8_t*>(x->k_scale), 4 * x->heads};
  p.pool[6] = {reinterpret_cast<uint8_t*>(pools->mass), 4};
  return cuda_status(launch_kv_compact(p, stream));
}

}  // extern "C"
