/*
 * msa_cache.h -- C ABI of libmsa, second part: attention for a tree of
 * drafted tokens over the paged cache, and eviction from the cache by
 * accumulated attention weight.
 *
 * One serving step with drafts uses them in this order: msa_kv_insert writes
 * the drafted tokens behind the context, msa_tree_attn attends for all of
 * them at once (msa_attn_mass then adds up the weight each cached token
 * received), and msa_kv_compact moves the accepted path together.  When a
 * request outgrows its budget, msa_evict_select names the tokens to keep and
 * msa_kv_compact moves them to the front, so that the pages behind them are
 * free.
 *
 * The conventions of msa.h hold for every entry point: device pointers owned
 * by the caller and 16-byte aligned, work enqueued on `stream` without any
 * host synchronisation or allocation, argument errors returned before
 * anything is launched, errors in device data reported in *dev_status with
 * defined outputs for the affected requests.  The calls are made with the
 * device current that owns the pointers and the stream.
 */
#ifndef MSA_CACHE_H
#define MSA_CACHE_H

#include "msa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of drafted rows per request. */
#define MSA_TREE_MAX_ROWS 256

/* What the drafted rows of a batch see.  Row j of request q (its position in
 * the cache is context_lens[q] + j, as everywhere) sees
 *   - of the cached tokens t < context_lens[q]: all of them when topk_idx is
 *     NULL; otherwise those of the blocks that topk_idx names for the row,
 *     and those of the block that holds position context_lens[q] (the
 *     context's partial last block);
 *   - of the drafted tokens i < q_len: those whose bit i of the row's mask is
 *     set (bit i % 32 of word i / 32; bits at and above q_len are ignored),
 *     or, when mask is NULL, i <= j (a causal chain).  A row sees itself
 *     only when its own bit is set.
 *   mask      [num_rows, mask_words] uint32, or NULL; a request with more
 *             than 32 * mask_words rows is poisoned (MSA_DEV_MALFORMED)
 *   topk_idx  [num_rows, topk] int32 block numbers as msa_topk_build_table
 *             writes them, or NULL (then topk is ignored); numbers outside
 *             the request's blocks are ignored, repeated ones count once */
typedef struct msa_tree {
  const uint32_t* mask;
  int32_t mask_words;
  const int32_t* topk_idx;
  int32_t topk;
} msa_tree;

/* Bytes of workspace that msa_tree_attn and msa_attn_mass need for these
 * sizes (topk: the width of topk_idx, 0 without one).  It needs no
 * initialisation and holds nothing between calls; calls that share one must
 * not overlap on the GPU. */
size_t msa_tree_attn_workspace_size(int32_t num_reqs, int32_t num_rows, int32_t bt_stride,
                                    int32_t num_heads, int32_t max_q_len, int32_t topk);

/* Attention of every drafted row over the tokens it sees, each request's
 * cached tokens read once for all its rows.  For row r and head h:
 *   s_t = softmax_scale * k_scale_t * (q_h . k_t),  m = max(max_t s_t, sink_h)
 *   den = sum_t exp(s_t - m) + exp(sink_h - m)
 *   out = sum_t exp(s_t - m) * v_scale_t * v_t / den,  lse = m + ln(den)
 * over the visible t (no sink: the sink terms are absent).  A row that sees
 * nothing gives out = 0 and lse = sink_h (or -inf).  Tokens that a row does
 * not see do not reach its result, whatever their bytes hold.  With one row
 * per request this is single-token decode over the whole cache.
 *   batch->max_q_len  upper bound of any request's q_len (at most
 *             MSA_TREE_MAX_ROWS; 0: not known, taken as min(num_rows,
 *             MSA_TREE_MAX_ROWS)); a request with more rows is poisoned.  The
 *             kernel for the whole batch is chosen by it: give the exact
 *             bound, and batches of single rows apart from wide trees, for
 *             speed (the workspace size takes the same value)
 *   batch->min_q_len  as elsewhere: requests with fewer rows are poisoned
 *   attn      as for msa_sparse_paged_attn (num_rows, num_pages as in batch).
 *             exp(s_t - m) times a v_scale per token is rounded to 16 bits
 *             relative to the row's largest such product, whatever the scale
 *             of a token of less weight; magnitudes from 2^-40 to 2^80, and 0,
 *             keep that precision.  With e4m3 pools q is converted to fp16,
 *             so |q| must stay below 65504 (msa_attn_mass likewise)
 * A poisoned request (MSA_DEV_BAD_PAGE, _BAD_LEN, _MALFORMED) gets the
 * outputs of empty rows.  Supported: as msa_sparse_paged_attn (one KV head,
 * head_dim 128, 1..16 heads); topk <= 2048. */
msa_status msa_tree_attn(const msa_batch* batch, const msa_tree* tree, const msa_attn_args* attn,
                         void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                         cudaStream_t stream);

/* The attention weight that the step's rows gave each token, added up over
 * rows and heads into a paged array (the accumulated weight that eviction
 * goes by).  For token t of request q at pool slot i = (block_table[q,
 * t/128], t % 128):
 *   w_t = sum over rows j and heads h that see t of exp(s_t - lse[j, h])
 *   mass[i] = mass[i] + w_t  for t < context_lens[q]
 *   mass[i] = w_t            for the step's own tokens, whose slots are new
 * with s_t and the visibility of msa_tree_attn, and lse as that call wrote it
 * (a row whose lse is -inf gives nothing).  Slots of no visited token are
 * left as they are, and so are those of tokens that a step writes without
 * calling this: they hold what an evicted token left there, and the caller
 * clears them before the next call counts them as cached.  The sum over rows and heads is taken in fp32 in a fixed
 * order: the same inputs give the same bits.
 *   attn      q, k_cache, k_scale and lse are read; v_cache, v_scale, sinks
 *             and out are not used and may be NULL
 *   mass      fp32 [num_pages, 128]
 * Requests of one call must not share pages, nor may one name a page twice (a
 * shared slot would be updated by several blocks at once).  Poisoned requests
 * leave mass as it is. */
msa_status msa_attn_mass(const msa_batch* batch, const msa_tree* tree, const msa_attn_args* attn,
                         float* mass, void* workspace, size_t workspace_bytes,
                         uint32_t* dev_status, cudaStream_t stream);

/* The cached tokens of a set of requests.
 *   lens         [num_reqs] tokens in the cache
 *   block_table  [num_reqs, bt_stride] page of each 128-token block; the
 *                first ceil(lens/128) entries of a row are read
 *   num_pages    P, pages in the pools (bounds check) */
typedef struct msa_cache_view {
  const int32_t* lens;
  const int32_t* block_table;
  int32_t bt_stride;
  int32_t num_reqs;
  int32_t num_pages;
} msa_cache_view;

/* The tokens that each request keeps under a budget.  For a request of L =
 * lens[r] tokens: if L <= budget all of them; otherwise positions
 * [0, keep_first), [L - keep_recent, L), and of the others the budget -
 * keep_first - keep_recent with the largest mass (equal masses go to the
 * lower position; -0 equals 0; NaN ranks below every number).
 *   mass      fp32 [num_pages, 128], paged like K
 *   keep      [num_reqs, budget] int32: the kept positions ascending, then -1
 *   keep_len  [num_reqs] int32
 * A request with a length below 0 or above 128 * bt_stride
 * (MSA_DEV_MALFORMED) or a page id out of range (MSA_DEV_BAD_PAGE) keeps
 * nothing: keep_len = -1 and its row of keep is -1 (msa_kv_compact leaves
 * such a request as it is).  budget >= 1, keep_first, keep_recent >= 0 and
 * keep_first + keep_recent <= budget, else MSA_ERR_SHAPE.  Supported:
 * bt_stride <= 16384, num_reqs <= 4096. */
msa_status msa_evict_select(const msa_cache_view* cache, const float* mass, int32_t budget,
                            int32_t keep_first, int32_t keep_recent, int32_t* keep,
                            int32_t* keep_len, uint32_t* dev_status, cudaStream_t stream);

/* The pools that hold a token's data, all paged alike.
 *   k_cache, v_cache  [P, 128, num_kv_heads, head_dim] of kv_dtype
 *   k_scale, v_scale  fp32 [P, 128, num_kv_heads] with scale_mode
 *                     MSA_SCALE_PER_TOKEN_HEAD; otherwise not touched
 *   index             the index-K cache (with its k_scale when given), or NULL
 *   mass              fp32 [P, 128], or NULL */
typedef struct msa_kv_pools {
  void* k_cache;
  void* v_cache;
  int32_t kv_dtype;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t scale_mode;
  float* k_scale;
  float* v_scale;
  const msa_index_cache* index;
  float* mass;
} msa_kv_pools;

/* Moves kept tokens together, in place: for every request r and i <
 * keep_len[r], the token at position base[r] + keep[r, i] moves to position
 * base[r] + i in every pool given.  Kept positions ascend strictly, so a
 * token only ever moves down; the positions behind the moved ones keep what
 * they held.  The caller takes base[r] + keep_len[r] as the new length.
 * After an eviction base is NULL (0) and keep is msa_evict_select's; to
 * commit a draft tree base is the context length, lens the context plus the
 * drafted rows, and keep the accepted rows of the request.
 *   cache     lens: the tokens that exist (base + keep must lie below them)
 *   base      [num_reqs] int32, or NULL
 *   keep      [num_reqs, keep_stride] int32
 *   keep_len  [num_reqs] int32; 0 or below moves nothing
 * A request whose list is not strictly ascending from 0 or does not fit
 * (keep_len > keep_stride, base + keep >= lens, base < 0) is left as it is
 * and sets MSA_DEV_BAD_TABLE; a length out of range sets MSA_DEV_MALFORMED,
 * a bad page id among the request's blocks MSA_DEV_BAD_PAGE, likewise.
 * Pages of a request must not be shared with another request of the call, nor
 * named twice.
 * Supported: head_dim 128, 1 <= num_kv_heads <= 64, keep_stride >= 1, the
 * index shapes of msa_index_cache, num_reqs <= 4096, bt_stride <= 16384. */
msa_status msa_kv_compact(const msa_cache_view* cache, const int32_t* base, const int32_t* keep,
                          int32_t keep_stride, const int32_t* keep_len, const msa_kv_pools* pools,
                          uint32_t* dev_status, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MSA_CACHE_H */
