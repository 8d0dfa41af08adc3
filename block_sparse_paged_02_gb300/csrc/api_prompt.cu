// api_prompt.cu -- the entry points of msa_prompt.h: argument checks, workspace
// layout and launches.  As in api.cu nothing here touches device data or
// synchronises.
#include "prompt_common.cuh"

namespace msa {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
msa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA; }

struct PromptWs {
  size_t split, part_bad, part_ml, part_o, total;
};

// The records and the partials: two pairs of 128-row tiles a CTA
PromptWs prompt_layout() {
  PromptWs w;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = round_up(off + bytes, 256);
    return at;
  };
  const size_t grid = (size_t)device_sm_count();
  w.split = take(grid * sizeof(PromptSplit));
  w.part_bad = take(2 * grid * 4);
  w.part_ml = take(2 * grid * 256 * 8);
  w.part_o = take(2 * grid * 256 * kHeadDim * 4);
  w.total = off;
  return w;
}

bool heads_supported(int num_heads, int num_kv_heads) {
  return num_kv_heads >= 1 && num_kv_heads <= kMaxKvHeads && num_heads >= 1 &&
         num_heads % num_kv_heads == 0 && num_heads / num_kv_heads <= kMaxGroup;
}

msa_status check_batch(const msa_batch* b) {
  if (b->num_reqs < 0 || b->num_rows < 0 || b->num_pages < 0 || b->bt_stride < 1) return MSA_ERR_SHAPE;
  if (!b->cu_seqlens_q) return MSA_ERR_NULL;
  if (b->num_reqs > 0 && (!b->cu_seqlens_k || !b->context_lens || !b->block_table)) return MSA_ERR_NULL;
  if (b->num_reqs > kMaxReqs || b->bt_stride > kMaxBlocksPerRow) return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

bool index_supported(const msa_index_cache* x) {
  return (x->heads == 1 && (x->dim == 64 || x->dim == 128)) || (x->heads == 2 && x->dim == 64);
}

// The pools of one layer, whose pages an operator writes
msa_status check_pools(const msa_kv_pools* p) {
  if (p->kv_dtype != MSA_KV_BF16 && p->kv_dtype != MSA_KV_FP8_E4M3) return MSA_ERR_DTYPE;
  if (p->scale_mode < MSA_SCALE_NONE || p->scale_mode > MSA_SCALE_PER_TOKEN_HEAD) return MSA_ERR_DTYPE;
  if (p->num_kv_heads < 1) return MSA_ERR_SHAPE;
  if (p->head_dim != kHeadDim || p->num_kv_heads > kMaxKvHeads) return MSA_ERR_UNSUPPORTED;
  const msa_index_cache* x = p->index;
  if (x) {
    if (x->dtype != MSA_KV_BF16 && x->dtype != MSA_KV_FP8_E4M3) return MSA_ERR_DTYPE;
    if (!index_supported(x)) return MSA_ERR_UNSUPPORTED;
  }
  return MSA_OK;
}
msa_status check_pool_pointers(const msa_kv_pools* p) {
  const msa_index_cache* x = p->index;
  const bool token = p->scale_mode == MSA_SCALE_PER_TOKEN_HEAD;
  if (!p->k_cache || !p->v_cache || (x && !x->k_cache)) return MSA_ERR_NULL;
  if (token && (!p->k_scale || !p->v_scale)) return MSA_ERR_NULL;
  if (!aligned16(p->k_cache) || !aligned16(p->v_cache) || !aligned16(p->mass) ||
      (token && (!aligned16(p->k_scale) || !aligned16(p->v_scale))) ||
      (x && (!aligned16(x->k_cache) || !aligned16(x->k_scale))))
    return MSA_ERR_SHAPE;
  return MSA_OK;
}

// A row's vectors: the stride holds them, 16-byte loads
bool stride_ok(int64_t stride, int heads, int dim) {
  return stride >= (int64_t)heads * dim && stride % 8 == 0;
}

// Memory of a call: `rows` runs of `len` bytes, `stride` (at least len) from one to the next
struct Span {
  const void* at;
  long long rows, stride, len;
};
Span packed(const void* at, long long bytes) { return {at, at && bytes > 0 ? 1 : 0, bytes, bytes}; }
// whether a packed span touches any run of the other
bool touch(const Span& one, const Span& runs) {
  if (one.rows == 0 || runs.rows == 0 || runs.len == 0) return false;
  const long long a = (long long)reinterpret_cast<uintptr_t>(one.at) - (long long)reinterpret_cast<uintptr_t>(runs.at);
  const long long first = a < runs.len ? 0 : (a - runs.len) / runs.stride + 1;  // the first run that ends behind a
  return first < runs.rows && first * runs.stride < a + one.len;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

msa_status msa_qk_rope_insert(const msa_batch* batch, const msa_qkv* qkv, const msa_rope* rope,
                              const msa_kv_pools* pools, uint32_t* dev_status, cudaStream_t stream) {
  if (!batch || !qkv || !rope || !pools || !dev_status) return MSA_ERR_NULL;
  msa_status st = check_batch(batch);
  if (st != MSA_OK) return st;
  st = check_pools(pools);
  if (st != MSA_OK) return st;
  const msa_index_cache* x = pools->index;
  if (qkv->num_heads < 1 || qkv->num_kv_heads != pools->num_kv_heads || qkv->head_dim != pools->head_dim)
    return MSA_ERR_SHAPE;
  if (qkv->num_heads > 1024) return MSA_ERR_UNSUPPORTED;
  if (rope->rotary_dim < 0 || rope->max_pos < 0) return MSA_ERR_SHAPE;
  if (rope->rotary_dim % 16 != 0 || rope->rotary_dim > kHeadDim || (x && rope->rotary_dim > x->dim))
    return MSA_ERR_UNSUPPORTED;
  const int hk = qkv->num_kv_heads;
  if (!stride_ok(qkv->q_stride, qkv->num_heads, kHeadDim) || !stride_ok(qkv->k_stride, hk, kHeadDim) ||
      !stride_ok(qkv->v_stride, hk, kHeadDim) ||
      (x && (!stride_ok(qkv->idx_q_stride, x->heads, x->dim) || !stride_ok(qkv->idx_k_stride, x->heads, x->dim))))
    return MSA_ERR_SHAPE;
  if (batch->num_rows == 0) return MSA_OK;
  if (batch->num_reqs == 0) return MSA_ERR_SHAPE;  // rows without any request
  if (!qkv->q || !qkv->k || !qkv->v || !qkv->q_out) return MSA_ERR_NULL;
  if (x && (!qkv->idx_q || !qkv->idx_k || !qkv->idx_q_out)) return MSA_ERR_NULL;
  if (rope->rotary_dim > 0 && !rope->cos_sin) return MSA_ERR_NULL;
  st = check_pool_pointers(pools);
  if (st != MSA_OK) return st;
  const bool fp8 = pools->kv_dtype == MSA_KV_FP8_E4M3;
  if (fp8 && pools->scale_mode != MSA_SCALE_NONE && (!pools->k_scale || !pools->v_scale)) return MSA_ERR_NULL;
  const void* every[] = {qkv->q, qkv->k, qkv->v, qkv->q_out, qkv->q_norm, qkv->k_norm, rope->cos_sin, rope->positions};
  for (const void* ptr : every)
    if (!aligned16(ptr)) return MSA_ERR_SHAPE;
  if (x && (!aligned16(qkv->idx_q) || !aligned16(qkv->idx_k) || !aligned16(qkv->idx_q_out) ||
            !aligned16(qkv->idx_q_norm) || !aligned16(qkv->idx_k_norm)))
    return MSA_ERR_SHAPE;
  // in place only where the rows are packed
  if ((qkv->q_out == qkv->q && qkv->q_stride != (int64_t)qkv->num_heads * kHeadDim) ||
      (x && qkv->idx_q_out == qkv->idx_q && qkv->idx_q_stride != (int64_t)x->heads * x->dim))
    return MSA_ERR_SHAPE;
  // otherwise the outputs lie apart from each other and from every vector
  {
    const long long n = batch->num_rows;
    const auto rows = [&](const void* src, int64_t stride, int heads, int dim) {
      return Span{src, n, 2 * (long long)stride, 2ll * heads * dim};
    };
    const Span q_out = packed(qkv->q_out, n * qkv->num_heads * kHeadDim * 2);
    const Span idx_q_out = packed(x ? qkv->idx_q_out : nullptr, x ? n * x->heads * x->dim * 2 : 0);
    Span in[5] = {rows(qkv->q, qkv->q_stride, qkv->num_heads, kHeadDim), rows(qkv->k, qkv->k_stride, hk, kHeadDim),
                  rows(qkv->v, qkv->v_stride, hk, kHeadDim), {}, {}};
    if (x) {
      in[3] = rows(qkv->idx_q, qkv->idx_q_stride, x->heads, x->dim);
      in[4] = rows(qkv->idx_k, qkv->idx_k_stride, x->heads, x->dim);
    }
    bool shared = touch(q_out, idx_q_out);
    for (int i = 0; i < 5; ++i) {
      shared |= (i != 0 || qkv->q_out != qkv->q) && touch(q_out, in[i]);
      shared |= (i != 3 || qkv->idx_q_out != qkv->idx_q) && touch(idx_q_out, in[i]);
    }
    if (shared) return MSA_ERR_SHAPE;
  }
  RopeLaunch p = {};
  p.batch = *batch;
  const auto vec = [](const void* src, int64_t stride, int heads, int dim, const void* norm) {
    return RopeVec{static_cast<const uint16_t*>(src), (long long)stride, heads, dim,
                   static_cast<const uint16_t*>(norm)};
  };
  p.q = vec(qkv->q, qkv->q_stride, qkv->num_heads, kHeadDim, qkv->q_norm);
  p.k = vec(qkv->k, qkv->k_stride, hk, kHeadDim, qkv->k_norm);
  p.v = vec(qkv->v, qkv->v_stride, hk, kHeadDim, nullptr);
  if (x) {
    p.idx_q = vec(qkv->idx_q, qkv->idx_q_stride, x->heads, x->dim, qkv->idx_q_norm);
    p.idx_k = vec(qkv->idx_k, qkv->idx_k_stride, x->heads, x->dim, qkv->idx_k_norm);
    p.idx_q_out = static_cast<uint16_t*>(qkv->idx_q_out);
    p.idx_cache = static_cast<uint8_t*>(x->k_cache);
    p.idx_fp8 = x->dtype == MSA_KV_FP8_E4M3;
    p.idx_scale = p.idx_fp8 ? x->k_scale : nullptr;
  }
  p.eps = qkv->eps;
  p.shift = qkv->norm_shift;
  p.cos_sin = rope->cos_sin;
  p.max_pos = rope->max_pos;
  p.rotary = rope->rotary_dim;
  p.near = rope->interleaved != 0;
  p.positions = rope->positions;
  p.q_out = static_cast<uint16_t*>(qkv->q_out);
  p.k_cache = static_cast<uint8_t*>(pools->k_cache);
  p.v_cache = static_cast<uint8_t*>(pools->v_cache);
  p.kv_fp8 = fp8;
  p.scale_mode = pools->scale_mode;
  p.k_scale = pools->k_scale;
  p.v_scale = pools->v_scale;
  p.mass = pools->mass;
  p.status = dev_status;
  return cuda_status(launch_qk_rope_insert(p, stream));
}

size_t msa_prompt_attn_workspace_size(int32_t num_heads, int32_t num_kv_heads) {
  return heads_supported(num_heads, num_kv_heads) ? prompt_layout().total : 0;
}

msa_status msa_prompt_attn(const msa_batch* batch, const msa_attn_args* a, void* workspace,
                           size_t workspace_bytes, uint32_t* dev_status, cudaStream_t stream) {
  if (!batch || !a || !dev_status) return MSA_ERR_NULL;
  const msa_status st = check_batch(batch);
  if (st != MSA_OK) return st;
  if (a->kv_dtype != MSA_KV_BF16 && a->kv_dtype != MSA_KV_FP8_E4M3) return MSA_ERR_DTYPE;
  if (a->scale_mode < MSA_SCALE_NONE || a->scale_mode > MSA_SCALE_PER_TOKEN_HEAD) return MSA_ERR_DTYPE;
  if (a->num_heads < 1 || a->num_kv_heads < 1 || a->num_heads % a->num_kv_heads != 0) return MSA_ERR_SHAPE;
  if (a->num_rows != batch->num_rows || a->num_pages != batch->num_pages) return MSA_ERR_SHAPE;
  if (a->head_dim != kHeadDim || !heads_supported(a->num_heads, a->num_kv_heads) ||
      a->num_pages >= (1 << 24))
    return MSA_ERR_UNSUPPORTED;
  if (batch->num_rows == 0) return MSA_OK;
  if (batch->num_reqs == 0) return MSA_ERR_SHAPE;  // rows without any request
  if (!a->q || !a->k_cache || !a->v_cache || !a->out || !a->lse) return MSA_ERR_NULL;
  if (a->scale_mode != MSA_SCALE_NONE && (!a->k_scale || !a->v_scale)) return MSA_ERR_NULL;
  if (!aligned16(a->q) || !aligned16(a->k_cache) || !aligned16(a->v_cache) || !aligned16(a->out) ||
      !aligned16(a->lse))
    return MSA_ERR_SHAPE;
  if (a->scale_mode == MSA_SCALE_PER_TOKEN_HEAD && (!aligned16(a->k_scale) || !aligned16(a->v_scale)))
    return MSA_ERR_SHAPE;
  const PromptWs w = prompt_layout();
  if (!workspace || workspace_bytes < w.total || !aligned16(workspace)) return MSA_ERR_WORKSPACE;
  // out may take q's place; nothing else of what is written shares memory with q or out
  const long long vectors = (long long)a->num_rows * a->num_heads;
  const Span q = packed(a->q, vectors * kHeadDim * 2), out = packed(a->out, vectors * kHeadDim * 2);
  const Span lse = packed(a->lse, vectors * 4);
  if ((a->out != a->q && touch(out, q)) || touch(lse, q) || touch(lse, out)) return MSA_ERR_SHAPE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PromptLaunch p = {};
  p.batch = *batch;
  p.q = static_cast<const uint16_t*>(a->q);
  p.num_heads = a->num_heads;
  p.num_kv_heads = a->num_kv_heads;
  p.k = static_cast<const uint8_t*>(a->k_cache);
  p.v = static_cast<const uint8_t*>(a->v_cache);
  p.kv_fp8 = a->kv_dtype == MSA_KV_FP8_E4M3;
  p.scale_mode = a->scale_mode;
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.sinks = a->sinks;
  p.softmax_scale = a->softmax_scale;
  p.out = static_cast<uint16_t*>(a->out);
  p.lse = a->lse;
  p.status = dev_status;
  p.split = reinterpret_cast<PromptSplit*>(ws + w.split);
  p.part_bad = reinterpret_cast<int32_t*>(ws + w.part_bad);
  p.part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
  p.part_o = reinterpret_cast<float*>(ws + w.part_o);
  return cuda_status(launch_prompt_attn(p, stream));
}

msa_status msa_page_fork(const msa_cache_view* from, const int32_t* refs, const int32_t* parent,
                         const int32_t* grow, const msa_page_set* to, uint32_t* dev_status,
                         cudaStream_t stream) {
  if (!from || !to || !dev_status) return MSA_ERR_NULL;
  if (from->num_reqs < 0 || from->num_pages < 0 || from->bt_stride < 1 || to->num_reqs < 0 || to->bt_stride < 1)
    return MSA_ERR_SHAPE;
  if (from->num_reqs > kMaxReqs || from->bt_stride > kMaxBlocksPerRow || to->num_reqs > kMaxReqs ||
      to->bt_stride > kMaxBlocksPerRow || from->num_pages >= (1 << 30))
    return MSA_ERR_UNSUPPORTED;
  if (from->num_reqs > 0 && (!from->lens || !from->block_table)) return MSA_ERR_NULL;
  if (from->num_pages > 0 && (!refs || !to->refs)) return MSA_ERR_NULL;
  if (to->num_reqs > 0 && (!parent || !to->lens || !to->block_table || !to->copy_src || !to->copy_dst ||
                           !to->copy_tokens))
    return MSA_ERR_NULL;
  const void* every[] = {from->lens, from->block_table, refs, parent, grow, to->lens, to->block_table, to->refs,
                         to->copy_src, to->copy_dst, to->copy_tokens, from->blocks, to->blocks};
  for (const void* ptr : every)
    if (!aligned16(ptr)) return MSA_ERR_SHAPE;
  const long long n = to->num_reqs, row = 4ll * to->bt_stride;
  const Span in[] = {packed(from->lens, 4ll * from->num_reqs),
                     packed(from->block_table, 4ll * from->num_reqs * from->bt_stride),
                     packed(refs, 4ll * from->num_pages), packed(parent, 4 * n), packed(grow, 4 * n),
                     packed(from->blocks, 4ll * from->num_reqs)};
  const Span out[] = {packed(to->lens, 4 * n),     packed(to->block_table, n * row), packed(to->refs, 4ll * from->num_pages),
                      packed(to->copy_src, 4 * n), packed(to->copy_dst, 4 * n),      packed(to->copy_tokens, 4 * n),
                      packed(to->blocks, 4 * n)};
  constexpr int kOut = sizeof(out) / sizeof(out[0]);
  for (int i = 0; i < kOut; ++i) {
    for (const Span& x : in)
      if (touch(out[i], x)) return MSA_ERR_SHAPE;
    for (int j = 0; j < i; ++j)
      if (touch(out[i], out[j])) return MSA_ERR_SHAPE;
  }
  return cuda_status(launch_page_fork({*from, refs, parent, grow, *to, dev_status}, stream));
}

msa_status msa_page_copy(const msa_kv_pools* layers, int32_t num_layers, int32_t num_pages,
                         const int32_t* src, const int32_t* dst, const int32_t* tokens,
                         int32_t num_copies, uint32_t* dev_status, cudaStream_t stream) {
  if (!dev_status) return MSA_ERR_NULL;
  if (num_layers < 0 || num_copies < 0 || num_pages < 0) return MSA_ERR_SHAPE;
  if (num_layers > 0 && !layers) return MSA_ERR_NULL;
  if (num_copies > (1 << 22)) return MSA_ERR_UNSUPPORTED;
  for (int i = 0; i < num_layers; ++i) {
    const msa_status st = check_pools(layers + i);
    if (st != MSA_OK) return st;
  }
  if (num_copies == 0 || num_layers == 0) return MSA_OK;
  if (!src || !dst || !tokens) return MSA_ERR_NULL;
  if (!aligned16(src) || !aligned16(dst) || !aligned16(tokens)) return MSA_ERR_SHAPE;
  for (int i = 0; i < num_layers; ++i) {
    const msa_status st = check_pool_pointers(layers + i);
    if (st != MSA_OK) return st;
  }
  CopyLaunch p = {};
  p.src = src;
  p.dst = dst;
  p.tokens = tokens;
  p.num_copies = num_copies;
  p.num_pages = num_pages;
  p.status = dev_status;
  cudaError_t error = cudaSuccess;
  const auto flush = [&]() {
    if (error == cudaSuccess && p.num_pools > 0) error = launch_page_copy(p, stream);
    p.num_pools = 0;
  };
  const auto add = [&](void* base, int row) {
    if (!base) return;
    if (p.num_pools == kCopyPools) flush();
    p.pool[p.num_pools++] = {static_cast<uint8_t*>(base), row};
  };
  for (int i = 0; i < num_layers; ++i) {
    const msa_kv_pools& l = layers[i];
    const int h = l.num_kv_heads, row = h * kHeadDim * (l.kv_dtype == MSA_KV_FP8_E4M3 ? 1 : 2);
    add(l.k_cache, row);
    add(l.v_cache, row);
    if (l.scale_mode == MSA_SCALE_PER_TOKEN_HEAD) {
      add(l.k_scale, 4 * h);
      add(l.v_scale, 4 * h);
    }
    if (l.index) {
      const msa_index_cache& x = *l.index;
      add(x.k_cache, x.heads * x.dim * (x.dtype == MSA_KV_FP8_E4M3 ? 1 : 2));
      if (x.dtype == MSA_KV_FP8_E4M3) add(x.k_scale, 4 * x.heads);
    }
    add(l.mass, 4);
  }
  flush();
  return cuda_status(error);
}

}  // extern "C"
