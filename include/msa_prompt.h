/*
 * msa_prompt.h -- C ABI of libmsa, third part: a prompt's way into the paged
 * cache, and the sharing of its pages by the requests that go on from it.
 *
 * A serving step uses them in this order: msa_page_fork gives every request
 * of the step the pages it writes (new ones, its own copy of a shared partial
 * page) and msa_page_copy fills the copies; in each layer msa_qk_rope_insert
 * norms and rotates the new tokens' queries and keys and writes K, V and the
 * index keys into the pools, and msa_prompt_attn attends for whole prompts or
 * their chunks (or msa_decode, msa_tree_attn for few rows).
 *
 * The conventions of msa.h hold for every entry point: device pointers owned
 * by the caller and 16-byte aligned, work enqueued on `stream` without any
 * host synchronisation or allocation, argument errors returned before
 * anything is launched, errors in device data reported in *dev_status with
 * defined outputs for what they affect.  The calls are made with the device
 * current that owns the pointers and the stream.
 */
#ifndef MSA_PROMPT_H
#define MSA_PROMPT_H

#include "msa_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further device status bits */
#define MSA_DEV_BAD_POS 32u  /* a row's rotary position lies outside the table: the row is not
                                written, its q_out and idx_q_out are 0 */
#define MSA_DEV_NO_PAGES 64u /* fewer free pages than msa_page_fork needs: nothing is forked */

/* Rotation of queries and keys by position.  With c_i, s_i the cosine and
 * sine of the row's position and i < rotary_dim / 2, a pair (a, b) of a
 * vector becomes (a c_i - b s_i, b c_i + a s_i); the dims behind rotary_dim
 * stay.
 *   cos_sin     fp32 [max_pos, rotary_dim]: the rotary_dim / 2 cosines of a
 *               position, then the sines (not read when rotary_dim is 0)
 *   rotary_dim  0 (no rotation), or a multiple of 16 up to the vectors' dim
 *   interleaved 0: pair i is dims (i, i + rotary_dim / 2); 1: (2i, 2i + 1)
 *   positions   int32 [num_rows], or NULL: row j of request q is at
 *               context_lens[q] + j.  Only the rotation goes by it (drafted
 *               tokens of a tree rotate by their depth); the slot written is
 *               always that of context_lens[q] + j. */
typedef struct msa_rope {
  const float* cos_sin;
  int32_t max_pos;
  int32_t rotary_dim;
  int32_t interleaved;
  const int32_t* positions;
} msa_rope;

/* The new tokens' vectors, bf16, as projections give them.  Vector h of row r
 * of x begins at x + r * x_stride + h * dim: slices of one projection's output
 * need no copy.  Strides are in elements, multiples of 8, at least heads * dim.
 *   q  num_heads vectors of head_dim;  k, v  num_kv_heads vectors of head_dim
 *   idx_q, idx_k  index->heads vectors of index->dim (of the pools' index
 *             cache; without one they are not read and may be NULL)
 *   *_norm    bf16 [dim] weights of the RMS norm of every head of that kind,
 *             or NULL: that kind is not normed
 *   eps, norm_shift  y = x * (mean(x^2) + eps)^-1/2 * (weight + norm_shift)
 *   q_out     [num_rows, num_heads, head_dim] bf16, may be q itself when
 *             q_stride is num_heads * head_dim
 *   idx_q_out [num_rows, index->heads, index->dim] bf16, likewise
 * Otherwise the outputs share no memory with each other or with any of the
 * vectors (MSA_ERR_SHAPE). */
typedef struct msa_qkv {
  const void* q;
  const void* k;
  const void* v;
  const void* idx_q;
  const void* idx_k;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  int64_t idx_q_stride;
  int64_t idx_k_stride;
  int32_t num_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  const void* q_norm;
  const void* k_norm;
  const void* idx_q_norm;
  const void* idx_k_norm;
  float eps;
  float norm_shift;
  void* q_out;
  void* idx_q_out;
} msa_qkv;

/* Norm, rotation and insertion in one pass: every row of the batch is a new
 * token (as for msa_kv_insert).  q, k, idx_q and idx_k are normed (where a
 * weight is given) and rotated in fp32 and rounded once: q and idx_q to bf16
 * into q_out and idx_q_out, k and idx_k, with v as it came, to the pools' type
 * at page block_table[q, pos/128], slot pos%128, by the rules of msa_kv_insert
 * (e4m3: saturating round to nearest of x / s; pools->scale_mode SCALAR takes
 * s = k_scale[0], v_scale[0]; PER_TOKEN_HEAD sets and writes s = max|x| / 448;
 * an FP8 index cache by its k_scale).
 *   pools     k_cache, v_cache, kv_dtype, scale_mode, k_scale, v_scale as
 *             above; index NULL: no index vectors are read or written (index
 *             reuse layers); mass, when given, is set to 0 at the new tokens'
 *             slots, as msa_attn_mass and msa_evict_select want it
 * Rows of requests that fail the device checks (MSA_DEV_BAD_PAGE, _BAD_LEN,
 * _MALFORMED) are not written; their q_out and idx_q_out are 0.  Supported:
 * head_dim 128, 1 <= num_heads <= 1024, 1 <= num_kv_heads <= 64, the index
 * shapes of msa_index_cache, num_reqs <= 4096, bt_stride <= 16384, rotary_dim
 * up to the index dim when there is an index. */
msa_status msa_qk_rope_insert(const msa_batch* batch, const msa_qkv* qkv, const msa_rope* rope,
                              const msa_kv_pools* pools, uint32_t* dev_status,
                              cudaStream_t stream);

/* Bytes of workspace that msa_prompt_attn needs (0: unsupported heads).  It
 * needs no initialisation and holds nothing between calls; calls that share
 * one must not overlap on the GPU. */
size_t msa_prompt_attn_workspace_size(int32_t num_heads, int32_t num_kv_heads);

/* Causal attention of whole prompts, or of their chunks behind cached tokens:
 * row j of request q, at position context_lens[q] + j, sees tokens 0 ..
 * context_lens[q] + j of the request's pages.  For head h and KV head
 * h / (num_heads / num_kv_heads):
 *   s_t = softmax_scale * k_scale_t * (q_h . k_t),  m = max(max_t s_t, sink_h)
 *   den = sum_t exp(s_t - m) + exp(sink_h - m)
 *   out = sum_t exp(s_t - m) * v_scale_t * v_t / den,  lse = m + ln(den)
 * (no sink: the sink terms are absent).  Tokens that a row does not see do
 * not reach its result, whatever their bytes hold.  Any number of rows per
 * request, none among them.
 *   attn      as for msa_tree_attn, with any num_heads that num_kv_heads
 *             divides.  out may be q itself; otherwise out and lse share no
 *             memory with q or each other (MSA_ERR_SHAPE).  The weights
 *             exp(s_t - m) (times a v_scale per token) are rounded to 16 bits
 *             for the product with V; with e4m3 pools q is converted to fp16,
 *             so |q| must stay below 65504, and below 2^-14 it is held to
 *             2^-25, not to its own size
 *   batch->max_q_len  not used
 *   batch->min_q_len  as elsewhere: requests with fewer rows are poisoned
 * A poisoned request (MSA_DEV_BAD_PAGE, _BAD_LEN, _MALFORMED) gets the
 * outputs of empty rows: 0, and sink_h or -inf.  The same call gives the same
 * bits; how a row's sums are cut, and so their last bits, goes by the whole
 * batch, bt_stride (which decides whether pairs of tiles are shared by CTAs)
 * and the GPU's number of SMs.  Supported: head_dim 128,
 * num_heads / num_kv_heads <= 128, num_kv_heads <= 64, num_reqs <= 4096,
 * bt_stride <= 16384, num_pages < 2^24. */
msa_status msa_prompt_attn(const msa_batch* batch, const msa_attn_args* attn, void* workspace,
                           size_t workspace_bytes, uint32_t* dev_status, cudaStream_t stream);

/* What msa_page_fork writes for the requests that go on (num_reqs of them).
 *   lens        [num_reqs] tokens held
 *   block_table [num_reqs, bt_stride]
 *   refs        [num_pages] how many tables (and other holders) name a page
 *   copy_src, copy_dst, copy_tokens  [num_reqs] the pages to copy: the first
 *               copy_tokens[i] slots of page copy_src[i] to copy_dst[i]
 *               (-1, -1, 0 where request i needs none)
 *   blocks      [num_reqs] pages held, ceil((lens + grow) / 128); may be NULL */
typedef struct msa_page_set {
  int32_t* lens;
  int32_t* block_table;
  int32_t* refs;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* copy_tokens;
  int32_t bt_stride;
  int32_t num_reqs;
  int32_t* blocks;
} msa_page_set;

/* The requests of the next step and their pages.  Request i of `to` goes on
 * from request parent[i] of `from` (-1: it begins, with no tokens) and is
 * about to write grow[i] tokens: so one call drops requests (that nobody goes
 * on from), reorders, forks and grows them.  With n = lens[parent[i]]:
 *   - to->lens[i] = n; the first ceil(n / 128) blocks are the parent's pages,
 *     shared, except a partial last page of a request that grows: when no
 *     other holder of that page is left, the lowest such i keeps it, and any
 *     other gets a new page and its copy entry;
 *   - new pages follow, so that n + grow[i] tokens fit;
 *   - pages that an old request holds behind its tokens (from->blocks) are
 *     given back, not handed on: the new ones stand for them;
 *   - new pages are the free ones (refs 0) of lowest number, in the order of i
 *     and block; pages that lose their last holder in this call are free;
 *   - to->refs counts the holders after it: refs, less the tables of `from`,
 *     plus those of `to`.  Holders outside the tables (a prefix cache) count
 *     in refs and stay.
 * grow is what a request may write: where fewer tokens came to be (rejected
 * drafts, an early stop, an eviction), its table names more pages than lens
 * tells of, and from->blocks has to say so at the next call (to->blocks of the
 * call before does): without it, pages behind ceil(lens / 128) keep their
 * count, which nobody takes off any more.
 * Shared pages are read by any operator, but none may write them: requests
 * that share are not compacted after an eviction (msa_kv_compact), and
 * msa_attn_mass takes them one to a call.
 * Entries of to->block_table behind a request's last block are left as they
 * are.  Nothing of `from` or refs is written, and `to` shares no memory with
 * them (MSA_ERR_SHAPE): the caller keeps two sets and swaps them.
 *   refs      [from->num_pages] int32;  parent, grow  [to->num_reqs] int32
 *             (grow may be NULL: 0, nothing is copied or added)
 * A length outside 0 .. 128 * bt_stride, blocks outside ceil(lens / 128) ..
 * bt_stride, a parent outside -1 .. from->num_reqs - 1, a negative grow or
 * one that does not fit to->bt_stride (MSA_DEV_MALFORMED), a page id out of
 * range among a request's blocks (MSA_DEV_BAD_PAGE), one whose refs is below 1
 * (MSA_DEV_BAD_TABLE), or too few free pages (MSA_DEV_NO_PAGES) stop the whole
 * call: to->lens (and to->blocks) is -1 everywhere, the copy entries are
 * empty, to->refs equals refs and to->block_table is left as it is.  A request
 * may not name a page twice.
 * Supported: num_reqs of both <= 4096, bt_stride of both <= 16384. */
msa_status msa_page_fork(const msa_cache_view* from, const int32_t* refs, const int32_t* parent,
                         const int32_t* grow, const msa_page_set* to, uint32_t* dev_status,
                         cudaStream_t stream);

/* Copies pages in the pools of num_layers layers, all of num_pages pages: for
 * i < num_copies the first tokens[i] (at most 128; 0 or below: none) slots of
 * page src[i] to page dst[i] in K, V, the per-token scales, the index cache
 * and mass of every layer (those that its msa_kv_pools has).  Pages that one
 * entry writes must not be read or written by another.  An entry with a page
 * out of range (MSA_DEV_BAD_PAGE) or tokens above 128 (MSA_DEV_MALFORMED) is
 * skipped.  The layers' structs are read on the host before the call returns.
 * Supported: as msa_kv_compact, layer by layer. */
msa_status msa_page_copy(const msa_kv_pools* layers, int32_t num_layers, int32_t num_pages,
                         const int32_t* src, const int32_t* dst, const int32_t* tokens,
                         int32_t num_copies, uint32_t* dev_status, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MSA_PROMPT_H */
