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
cudaError_t launch_tree_attn_tc(const TreeLaunch& p, int grid, cudaStream_t stream);
int tree_part_rows(int max_rows, int num_heads);

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

// 2^x, results below 2^-126 as 0
__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What P, rounded to 16 bits, is kept relative to: 2^m with m the largest exponent met
// so far (log2 units), moved only when one exceeds it by more than kSlack.  Where P is
// f16 it is kept kHalfHead above that, so that f16's full steps (from 2^-14) reach weights
// of 2^-21 of the row's largest; kHalfHead + kSlack stays below f16's 2^16.
constexpr float kSlack = 8.f;
constexpr float kHalfHead = 7.f;

// With a scale per token P carries it, so the exponent is that of the product, s +
// log2 |v_scale|: a token of little weight cannot cost the others their range, however
// large its scale.  The same 2^m divides the sum of the weights, which is fp32 and has
// room for it: scales below 2^-40 (0 among them) count as 2^-40 here, which keeps 2^(s - m)
// below 2^56.  The log2 is the exponent field with the mantissa as its fraction, low by
// 0.09 at most; infinities and NaN give a finite value.
__device__ __forceinline__ uint32_t scale_bits(float x) {
  return max(__float_as_uint(x) & 0x7fffffffu, __float_as_uint(0x1p-40f));
}
__device__ __forceinline__ float bits_log2(uint32_t b) { return (float)b * 0x1p-23f - 127.f; }
__device__ __forceinline__ float log2_scale(float x) { return bits_log2(scale_bits(x)); }

// two products a * b + c in one instruction
__device__ __forceinline__ void fma2(float& x0, float& x1, float b, float c) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\t"
      "mov.b64 z, {%3, %3};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float& x0, float& x1, float a0, float a1) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(a0), "f"(a1));
}

// the same with a factor for each
__device__ __forceinline__ void fma2p(float& x0, float& x1, float b0, float b1, float c) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "mov.b64 z, {%4, %4};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(b0), "f"(b1), "f"(c));
}
__device__ __forceinline__ void mul2v(float& x0, float& x1, float b0, float b1) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(b0), "f"(b1));
}
// the same with an addend for each
__device__ __forceinline__ void fma2v(float& x0, float& x1, float b, float c0, float c1) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\t"
      "mov.b64 z, {%3, %4};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(b), "f"(c0), "f"(c1));
}

// A row's end: (m, l) in log2 units, the sink joined in
struct TreeRowEnd {
  float f, lse;  // factor of the accumulators, natural-log lse
};
__device__ __forceinline__ TreeRowEnd tree_row_end(float m, float l, bool has_sink, float sink2, float vs) {
  TreeRowEnd e;
  if (m == -INFINITY && l == 0.f) {  // nothing seen
    e.f = 0.f;
    e.lse = has_sink ? sink2 * kTreeLn2 : -INFINITY;
    return e;
  }
  float f = 1.f;
  if (has_sink) {
    const float mn = fmaxf(m, sink2);
    f = ex2_ftz(m - mn);
    l = l * f + ex2_ftz(sink2 - mn);
    m = mn;
  }
  e.f = f * vs / l;
  e.lse = (m + log2f(l)) * kTreeLn2;
  return e;
}

// every row of an unusable batch, as empty rows
__device__ __forceinline__ void tree_write_all_empty(const TreeLaunch& p) {
  const long long n = (long long)p.batch.num_rows * p.num_heads;
  const long long step = (long long)gridDim.x * blockDim.x;
  const long long at = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  for (long long i = at; i < n; i += step)
    p.lse[i] = p.sinks ? __ldg(p.sinks + i % p.num_heads) : -INFINITY;
  uint4* o = reinterpret_cast<uint4*>(p.out);
  for (long long i = at; i < n * (kHeadDim / 8); i += step) o[i] = make_uint4(0u, 0u, 0u, 0u);
}

// The CTA's slice of a flat item list over the requests (cost(request, its
// visits) items each): items [begin, end) of total, cut into `ctas` equal parts, none
// empty (later CTAs idle).  Every thread of the CTA takes part; s_ll: 40 long
// longs of shared scratch, free again after a barrier.
struct TreeSlice {
  long long total, begin, end, pre;  // pre: first item of request q
  int q, ctas, visits;
  TreeReq first;  // request q, which visits `visits` blocks
  bool tiled;     // cu_seqlens_q tiles [0, num_rows); otherwise the rest is 0
};

template <int NT, typename Cost>
__device__ __forceinline__ TreeSlice tree_slice(const TreeLaunch& p, Cost cost, long long* s_ll) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = p.batch.num_reqs;
  TreeSlice s;
  s.total = s.begin = s.end = s.pre = 0;
  s.q = 0;
  s.ctas = 1;
  s.visits = 0;
  // costs and checks of NT requests at a time, their sum by a scan; with few
  // requests one round gives both the total and the place of the slice
  bool ok = true;
  long long inc = 0, c = 0;
  TreeReq rq;
  int nv = 0;
  auto round = [&](int q) {
    c = 0;
    if (q < R) {
      rq = tree_request(p, q);
      ok &= rq.qlen >= 0 && (q > 0 || rq.q0 == 0) && (q < R - 1 || rq.q0 + rq.qlen == p.batch.num_rows);
      if (ok && rq.qlen > 0) {
        nv = tree_visits(p, q, rq);
        c = cost(rq, nv);
      }
    }
    inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long n = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += n;
    }
    if (lane == 31) s_ll[warp] = inc;
  };
  for (int q0 = 0; q0 < R; q0 += NT) {
    round(q0 + tid);
    s.tiled = __syncthreads_and(ok) != 0;
    if (!s.tiled) return s;
    for (int w = 0; w < NT / 32; ++w) s.total += s_ll[w];
    if (q0 + NT < R) __syncthreads();
  }
  s.ctas = (int)max(1ll, min((long long)gridDim.x, s.total));
  if ((int)blockIdx.x < s.ctas) {
    s.begin = s.total * blockIdx.x / s.ctas;
    s.end = s.total * (blockIdx.x + 1) / s.ctas;
  }
  if (s.begin >= s.end) return s;
  long long base = 0;
  for (int q0 = 0; q0 < R; q0 += NT) {
    if (R > NT) {
      __syncthreads();
      round(q0 + tid);
      __syncthreads();
    }
    long long before = base;
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) before += s_ll[w];
      base += s_ll[w];
    }
    const long long pre = before + inc - c;
    if (c > 0 && pre <= s.begin && s.begin < pre + c) {
      // the request that holds the slice's first item, for all threads
      s_ll[32] = q0 + tid;
      s_ll[33] = pre;
      s_ll[34] = nv;
      int* g = reinterpret_cast<int*>(s_ll + 35);
      g[0] = rq.q0;
      g[1] = rq.qlen;
      g[2] = rq.ctx;
      g[3] = rq.nb;
      g[4] = (int)rq.bad;
    }
    __syncthreads();
    if (base > s.begin) break;
  }
  const int* g = reinterpret_cast<const int*>(s_ll + 35);
  s.q = (int)s_ll[32];
  s.pre = s_ll[33];
  s.visits = (int)s_ll[34];
  s.first.q0 = g[0];
  s.first.qlen = g[1];
  s.first.ctx = g[2];
  s.first.nb = g[3];
  s.first.bad = (uint32_t)g[4];
  return s;
}

// A tile counts its blocks and kTreeTileCost items more, for what its start and
// end cost (queries in, sums joined and written).  64 requests of one row: 56 us with
// one item, 53 with four, 54.5 with seven; wide trees (8 requests of 48..64 rows x 16
// heads) 83.6, 82.5, 83.7.
constexpr int kTreeTileCost = 4;

// The part of a tile that the slice holds from item `it` on, in request items
// [pre, pre + tiles * (nv + kTreeTileCost)).
struct TreeSeg {
  int tile, b0, nb;      // visited blocks [b0, b0 + nb) of the tile; nb may be 0
  long long first, end;  // items of the tile's first block, behind its last
  long long next;        // the item to go on with
};
__device__ __forceinline__ TreeSeg tree_segment(long long it, long long end, long long pre, int nv) {
  TreeSeg s;
  const int per = nv + kTreeTileCost;
  s.tile = (int)((it - pre) / per);
  const int in = (int)((it - pre) % per);
  s.end = pre + (long long)(s.tile + 1) * per;
  s.first = s.end - nv;
  s.next = min(s.end, end);
  s.b0 = max(0, in - kTreeTileCost);
  s.nb = max(0, (int)(s.next - it) + in - kTreeTileCost) - s.b0;
  return s;
}
__device__ __forceinline__ long long tree_items(int nv, int tiles) {
  return (long long)(nv + kTreeTileCost) * tiles;
}

#endif  // __CUDACC__

}  // namespace msa
