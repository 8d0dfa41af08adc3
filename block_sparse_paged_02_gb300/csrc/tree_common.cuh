// tree_common.cuh -- what the draft-tree attention and the weight
// accumulation share: the launch record, the requests' geometry, the split of
// a flat item list over the CTAs, and the visibility bits of 16 tokens.
#pragma once

#include "msa_cache.h"
#include "msa_internal.cuh"

namespace msa {

constexpr float kTreeLog2e = 1.4426950408889634f;
constexpr float kTreeLn2 = 0.6931471805599453f;

// One tile whose blocks are shared by several CTAs (written by the second of
// them): rows [row0 * H, row0 * H + nrows), partials of CTAs c - 1 .. last.
struct TreeSplit {
  int32_t nrows;  // 0: none
  int32_t row0;
  int32_t last;
  int32_t pad;
};

struct TreeLaunch {
  msa_batch batch;
  const uint32_t* mask;
  int mask_words;
  const int32_t* topk_idx;
  int topk;
  const uint16_t* q;
  int num_heads;
  const uint8_t* k;
  const uint8_t* v;
  int kv_fp8, scale_mode;
  const float* k_scale;
  const float* v_scale;
  const float* sinks;
  float softmax_scale;
  uint16_t* out;
  float* lse;
  float* mass;
  uint32_t* status;
  int max_rows;  // bound on a request's rows
  // selected blocks (topk_idx): per request the visited blocks ascending, how
  // many (-1: a bad page), and per block one bit per row that selects it
  int list_cap, list_words;
  int32_t* list_count;   // [R]
  int32_t* list_blk;     // [R, list_cap]
  uint32_t* list_rows;   // [R, list_cap, list_words]
  // split tiles: records [grid], partials [2 * grid] of tile_rows rows
  TreeSplit* split;
  int32_t* part_bad;     // [2 * grid]
  float2* part_ml;       // [2 * grid, tile_rows]
  float* part_o;         // [2 * grid, tile_rows, 128]
};

cudaError_t launch_tree_plan(const TreeLaunch& p, cudaStream_t stream);
cudaError_t launch_tree_attn(const TreeLaunch& p, cudaStream_t stream);
cudaError_t launch_attn_mass(const TreeLaunch& p, cudaStream_t stream);
int tree_tile_rows(int max_rows, int num_heads);

struct EvictLaunch {
  msa_cache_view cache;
  const float* mass;
  int budget, first, recent;
  int32_t* keep;
  int32_t* keep_len;
  uint32_t* status;
};
cudaError_t launch_evict_select(const EvictLaunch& p, cudaStream_t stream);

// One pool as the move sees it: rows of `row` bytes per token
struct CompactPool {
  uint8_t* base;
  int row;
};
constexpr int kCompactPools = 7;
struct CompactLaunch {
  msa_cache_view cache;
  const int32_t* base;
  const int32_t* keep;
  int keep_stride;
  const int32_t* keep_len;
  CompactPool pool[kCompactPools];  // base NULL: absent
  uint32_t* status;
};
cudaError_t launch_kv_compact(const CompactLaunch& p, cudaStream_t stream);

#ifdef __CUDACC__

struct TreeReq {
  int q0, qlen, ctx, nb;
  uint32_t bad;
};

__device__ __forceinline__ TreeReq tree_request(const TreeLaunch& p, int q) {
  TreeReq r;
  r.bad = request_lengths(p.batch, q, &r.q0, &r.qlen, &r.ctx, &r.nb);
  if (r.bad == 0 && (r.qlen > p.max_rows || (p.mask && r.qlen > 32 * p.mask_words)))
    r.bad = MSA_DEV_MALFORMED;
  return r;
}

// Blocks a request's rows visit; a poisoned request counts as one, so that
// some CTA writes its rows.
__device__ __forceinline__ int tree_visits(const TreeLaunch& p, int q, TreeReq& r) {
  if (r.bad) return 1;
  if (!p.topk_idx) return r.nb;
  const int n = p.list_count[q];
  if (n < 0) {
    r.bad = MSA_DEV_BAD_PAGE;
    return 1;
  }
  return n;
}

// Visibility of tokens [t0, t0 + 16) (positions) for row j of the request:
// bit i for token t0 + i.  `cached`: the row reads this block's cached
// tokens (always without a selection).
__device__ __forceinline__ uint32_t tree_vis16(const TreeLaunch& p, int row, int j, int ctx,
                                               int qlen, int t0, bool cached) {
  uint32_t bits = 0;
  const int n = min(max(ctx - t0, 0), 16);
  if (cached) bits = (1u << n) - 1u;
  if (n == 16) return bits;
  const int off = t0 - ctx;  // drafted index of token t0 (> -16)
  uint32_t d = 0;
  if (p.mask) {
    const uint32_t* m = p.mask + (long long)row * p.mask_words;
    if (off < 0) {
      d = __ldg(m) << -off;
    } else if (off < 32 * p.mask_words) {
      const int w = off >> 5;
      const uint32_t hi = w + 1 < p.mask_words ? __ldg(m + w + 1) : 0u;
      d = __funnelshift_r(__ldg(m + w), hi, off & 31);
    }
  } else {
    const int cnt = j + 1 - off;  // tokens t0 .. with drafted index <= j
    d = cnt >= 16 ? 0xffffu : cnt > 0 ? (1u << cnt) - 1u : 0u;
  }
  // drafted tokens only: indexes 0 .. qlen - 1
  const int end = min(max(qlen - off, 0), 16);
  d &= ((1u << end) - 1u) & ~((1u << n) - 1u);
  return bits | d;
}

// Whether row j of the request reads the cached tokens of the visited block
// at place `at` of its list.
__device__ __forceinline__ bool tree_row_selects(const uint32_t* rows, int j) {
  return !rows || ((__ldg(rows + (j >> 5)) >> (j & 31)) & 1u);
}

// The CTA's slice of a flat item list over the requests (cost(q) items for
// request q): items [begin, end) of total, cut into `ctas` equal parts, none
// empty (later CTAs idle).  Every thread of the CTA takes part; s_ll: 40 long
// longs of shared scratch, free again after a barrier.
struct TreeSlice {
  long long total, begin, end, pre;  // pre: first item of request q
  int q, ctas;
  bool tiled;  // cu_seqlens_q tiles [0, num_rows); otherwise the rest is 0
};

template <int NT, typename Cost>
__device__ __forceinline__ TreeSlice tree_slice(const TreeLaunch& p, Cost cost, long long* s_ll) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = p.batch.num_reqs;
  TreeSlice s;
  bool ok = p.batch.cu_seqlens_q[0] == 0 && p.batch.cu_seqlens_q[R] == p.batch.num_rows;
  for (int q = tid; q < R; q += NT) ok &= p.batch.cu_seqlens_q[q + 1] >= p.batch.cu_seqlens_q[q];
  s.tiled = __syncthreads_and(ok) != 0;
  s.total = s.begin = s.end = s.pre = 0;
  s.q = 0;
  s.ctas = 1;
  if (!s.tiled) return s;
  long long mine = 0, keep = 0;
  for (int q = tid; q < R; q += NT) {
    keep = cost(q);
    mine += keep;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) s_ll[warp] = mine;
  __syncthreads();
  for (int w = 0; w < NT / 32; ++w) s.total += s_ll[w];
  s.ctas = (int)max(1ll, min((long long)gridDim.x, s.total));
  if ((int)blockIdx.x < s.ctas) {
    s.begin = s.total * blockIdx.x / s.ctas;
    s.end = s.total * (blockIdx.x + 1) / s.ctas;
  }
  __syncthreads();
  if (s.begin >= s.end) return s;
  // the request that holds item s.begin
  long long base = 0;
  for (int q0 = 0; q0 < R; q0 += NT) {
    const int q = q0 + tid;
    long long c = 0;
    if (q < R) c = R <= NT ? keep : cost(q);
    long long inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long n = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += n;
    }
    if (lane == 31) s_ll[warp] = inc;
    __syncthreads();
    long long before = base, sum = 0;
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) before += s_ll[w];
      sum += s_ll[w];
    }
    const long long pre = before + inc - c;
    if (c > 0 && pre <= s.begin && s.begin < pre + c) {
      s_ll[32] = q;
      s_ll[33] = pre;
    }
    base += sum;
    __syncthreads();
    if (base > s.begin) break;
  }
  s.q = (int)s_ll[32];
  s.pre = s_ll[33];
  return s;
}

#endif  // __CUDACC__

}  // namespace msa
