// prompt_attn.cu -- causal attention of whole prompts (or their chunks behind
// cached tokens) over the paged cache, on the 5th-generation tensor cores.
//
// For the rows of a request and one KV head, whose group of G query heads
// shares its keys: S = scale Q K^T, P = 2^(S - m) with m a running reference,
// O += P V, l += sum P; at the end O / l and lse = m + ln l, the sink joined in.
//
// A tile is 128 rows of the tensor cores: floor(128 / G) tokens with all their
// heads (one 3-D tensor copy of Q); two tiles share every block of 128 tokens'
// K and V, which is a page, and while one is in its softmax the tensor cores work
// on the other.  S and P V are tcgen05.mma M128 N128 of the same shape from one
// issuing thread, so they run in the order of issue: S of the next block goes
// out right behind P V of this one, over the same tensor memory, without a
// wait between them.
// Roles: warp 0 issues the copies; one thread of warp 1 all products; warp 2
// brings the scales per token of bf16 pools; warp 3 looks bf16 V over (below);
// warps 4-7 and 8-11 are the tiles' softmax, a thread per row.  With e4m3
// pools warps 12-15 turn the tiles into f16 (exact) and the products run in f16.
//
// The work is the list (request, KV head, tile pair), each pair counted as the
// tokens it sees and kPairCost more; it is cut into equal contiguous slices, one
// per CTA, at block boundaries.  A pair that several CTAs share goes through
// partial results (O, m, l in fp32) that a second kernel joins in CTA order, so
// that results do not depend on timing.
//
// A block that not every row sees whole (the diagonal) takes a masked softmax,
// and its V is looked over: a value that is not finite would reach rows that
// do not see it through 0 * V, so that block's P V is then added row by row,
// from the visible tokens alone.  V behind the request's end is zeroed.
#include <string.h>

#include "attn_tc.cuh"
#include "prompt_common.cuh"

namespace msa {
namespace {

constexpr int kInfos = 8;
constexpr int kLooks = 4;
constexpr int kConv = 4;  // converting warps (e4m3 pools)
// flags of a block
constexpr int kFirst = 1, kLast = 2, kWhole = 4, kNoData = 8, kPoison = 16, kEnd = 32, kMixed = 64,
              kTwo = 128, kHalves = 256, kWork0 = 512, kWork1 = 1024;

// What a tile pair's start and end cost, in tokens
constexpr int kPairCost = 256;
// Least tokens of a CTA's slice (two boundaries of blocks at least)
constexpr long long kMinSlice = 512;

struct BlockInfo {
  int flags;
  int row0, ntok, pos0;  // the pair's rows: first in the batch, count, position of the first
  int seq, t0;           // tokens of the request; position of the block's first
  int slot, head;        // partial slot; KV head
  uint32_t bad;
  int page;
};

constexpr int kRegsFew = 104, kRegsMore = 152;

template <bool FP8, bool PTH>
struct PaCfg {
  static constexpr int kThreads = FP8 ? 512 : 384;
  static constexpr int kBufs = FP8 ? 3 : PTH ? 4 : 5;  // ring of 16-bit K and V tiles, alternating
  static constexpr int kRaws = FP8 ? 3 : 0;            // ring of e4m3 tiles
  static constexpr int kSmQ = kBufs * kTile;
  static constexpr int kSmRaw = kSmQ + 2 * kTile;
  static constexpr int kSmScale = kSmRaw + kRaws * kRaw;
  static constexpr int kSmInfo = kSmScale + (PTH ? kScales * kScaleWords * 4 : 0);
  static constexpr int kSmBars = kSmInfo + kInfos * (int)sizeof(BlockInfo);
  // kv full / empty, raw full / empty, q full / empty, infos, scales; per tile s_full,
  // p_full of two halves, pv_half, pv_done, o_free; fill, drained, looked
  static constexpr int kNumBars = 2 * kBufs + 2 * kRaws + 2 + kInfos + kScales + 12 + 2 + kLooks;
  static constexpr int kSmMisc = kSmBars + kNumBars * 8;
  static constexpr int kBytes = kSmMisc + 64;
  static_assert(kBytes <= 227 * 1024, "shared memory");
  static_assert(sizeof(BlockInfo) % 8 == 0 && kSmBars % 8 == 0, "alignment");
};

constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t col_s(int t) { return 128u * t; }
__device__ __forceinline__ uint32_t col_o(int t) { return 256u + 128u * t; }

struct PromptReq {
  int q0, qlen, ctx, nb;
  uint32_t bad;
};

// (a request with unusable lengths counts as one without a context)
__device__ __forceinline__ PromptReq prompt_request(const msa_batch& b, int q) {
  PromptReq r;
  r.bad = request_lengths(b, q, &r.q0, &r.qlen, &r.ctx, &r.nb);
  if (r.bad) r.ctx = r.nb = 0;
  return r;
}

// The pairs of one KV head of a request: `wide` rows each
struct Pairs {
  int tiles, wide, qlen, ctx;
  // tokens before pair i (all of them for i = tiles)
  __device__ __forceinline__ long long before(int i) const {
    const long long n = (long long)i * (kPairCost + ctx) + (long long)wide * i * (i + 1) / 2;
    return i < tiles ? n : n - ((long long)tiles * wide - qlen);
  }
  __device__ __forceinline__ int seen(int i) const { return ctx + min((i + 1) * wide, qlen); }
  // the pair that holds token u of the list
  __device__ __forceinline__ int at(long long u) const {
    const float a = 0.5f * (float)wide, b = (float)(kPairCost + ctx) + a, f = (float)u;
    int i = (int)(2.f * f / (b + sqrtf(b * b + 4.f * a * f)));
    i = max(0, min(i, tiles - 1));
    while (i > 0 && before(i) > u) --i;
    while (i < tiles - 1 && before(i + 1) <= u) ++i;
    return i;
  }
};
__device__ __forceinline__ Pairs pairs_of(const PromptReq& r, int wide) {
  return {(int)(((long long)r.qlen + wide - 1) / wide), wide, r.qlen, r.ctx};
}

// The CTA's slice [begin, end) of the list; every thread takes part; s_ll: 40
// long longs of shared scratch.
struct PromptSlice {
  long long total, begin, end, pre;  // pre: where request q begins
  int q, ctas;
  bool tiled;  // cu_seqlens_q tiles [0, num_rows); otherwise the rest is 0
};

template <int NT>
__device__ __forceinline__ PromptSlice prompt_slice(const PromptLaunch& p, int wide, long long* s_ll) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = p.batch.num_reqs;
  PromptSlice s;
  s.total = s.begin = s.end = s.pre = 0;
  s.q = 0;
  s.ctas = 1;
  bool ok = true;
  long long inc = 0, c = 0;
  auto round = [&](int q) {
    c = 0;
    if (q < R) {
      const PromptReq r = prompt_request(p.batch, q);
      ok &= r.qlen >= 0 && (q > 0 || r.q0 == 0) && (q < R - 1 || r.q0 + r.qlen == p.batch.num_rows);
      if (ok && r.qlen > 0) {
        const Pairs a = pairs_of(r, wide);
        c = a.before(a.tiles) * p.num_kv_heads;
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
  s.ctas = (int)max(1ll, min((long long)gridDim.x, s.total / kMinSlice));
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
      s_ll[32] = q0 + tid;
      s_ll[33] = pre;
    }
    __syncthreads();
    if (base > s.begin) break;
  }
  s.q = (int)s_ll[32];
  s.pre = s_ll[33];
  return s;
}

template <bool FP8, bool PTH>
__global__ void __launch_bounds__(PaCfg<FP8, PTH>::kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ PromptLaunch p, const __grid_constant__ CUtensorMap qmap,
                       const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
  using C = PaCfg<FP8, PTH>;
  constexpr int kBufs = C::kBufs, kRaws = C::kRaws, kThreads = C::kThreads, kSmQ = C::kSmQ;
  constexpr uint32_t kIdescS = tc::idesc_16(128, 128, 0, FP8 ? 0 : 1);
  constexpr uint32_t kIdescO = tc::idesc_16(128, 128, 1, FP8 ? 0 : 1);
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + C::kSmBars);
  uint64_t* kv_empty = kv_full + kBufs;
  uint64_t* raw_full = kv_empty + kBufs;
  uint64_t* raw_empty = raw_full + kRaws;
  uint64_t* q_full = raw_empty + kRaws;
  uint64_t* q_empty = q_full + 1;
  uint64_t* info_full = q_empty + 1;
  uint64_t* sc_full = info_full + kInfos;
  uint64_t* s_full = sc_full + kScales;  // [tile]
  uint64_t* p_full = s_full + 2;         // [tile][half]
  uint64_t* pv_half = p_full + 4;        // [tile]: P V of the first half
  uint64_t* pv_done = pv_half + 2;       // [tile]
  uint64_t* o_free = pv_done + 2;        // [tile]
  uint64_t* fill = o_free + 2;
  uint64_t* drained = fill + 1;
  uint64_t* looked = drained + 1;        // [kLooks]
  BlockInfo* info = reinterpret_cast<BlockInfo*>(smem + C::kSmInfo);
  // [0] timeout, [4 + n % kLooks] n + 1: odd values in block n's V
  int* misc = reinterpret_cast<int*>(smem + C::kSmMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 8);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = p.num_heads, Hk = p.num_kv_heads, G = H / Hk;
  const int tpt = 128 / G;  // tokens per tile

  if (tid == 0) {
    for (int i = 0; i < 8; ++i) misc[i] = 0;
    for (int s = 0; s < kBufs; ++s) {
      mbar_init(&kv_full[s], FP8 ? kConv : 1);
      mbar_init(&kv_empty[s], FP8 ? 1 : 2);  // the issuer, the warp that looks V over
    }
    for (int s = 0; s < kRaws; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], kConv);
    }
    for (int s = 0; s < kScales; ++s) mbar_init(&sc_full[s], FP8 ? kConv : 1);
    mbar_init(q_full, FP8 ? kConv : 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < kInfos; ++i) mbar_init(&info_full[i], 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[2 * t], 4);
      mbar_init(&p_full[2 * t + 1], 4);
      mbar_init(&pv_half[t], 1);
      mbar_init(&pv_done[t], 1);
      mbar_init(&o_free[t], 4);
    }
    mbar_init(fill, 1);
    mbar_init(drained, 1);
    for (int i = 0; i < kLooks; ++i) mbar_init(&looked[i], 1);
    fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, kTmemCols);
  const PromptSlice sl = prompt_slice<kThreads>(p, 2 * tpt, reinterpret_cast<long long*>(smem));
  fence_proxy_async_smem();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0 && sl.begin >= sl.end) p.split[blockIdx.x].nrows = 0;
  if (!sl.tiled) {  // every row of an unusable batch, as empty rows
    const long long n = (long long)p.batch.num_rows * H, step = (long long)gridDim.x * kThreads;
    const long long at = (long long)blockIdx.x * kThreads + tid;
    for (long long i = at; i < n; i += step)
      p.lse[i] = p.sinks ? __ldg(p.sinks + i % H) : -INFINITY;
    uint4* o = reinterpret_cast<uint4*>(p.out);
    for (long long i = at; i < n * (kHeadDim / 8); i += step) o[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0 && blockIdx.x == 0) atomicOr(p.status, MSA_DEV_MALFORMED);
  }

  if (sl.begin < sl.end) {
    const auto copies = [&]() {
      // ---------------------------------------------- copies
      long long it = sl.begin, pre = sl.pre;
      int q = sl.q, n = 0, n_seg = 0, x = 0, fills = 0, checked = -1;
      uint32_t bad = 0;
      bool ok = true;
      PromptSplit rec;
      rec.nrows = 0;
      const uint32_t qbytes = 2u * 64u * (uint32_t)(G * tpt);  // of one box of Q
      auto acquire = [&]() -> int {
        constexpr int ring = FP8 ? kRaws : kBufs;
        uint64_t* freed = FP8 ? raw_empty : kv_empty;
        const int b = x % ring;
        if (x >= ring) ok = ok && warp_wait(&freed[b], ((x / ring) - 1) & 1);
        ++x;
        return b;
      };
      BlockInfo bi;
      bi.page = 0;
      auto announce = [&]() {
        if (lane == 0) {
          info[n % kInfos] = bi;
          mbar_arrive(&info_full[n % kInfos]);
        }
        ++n;
      };
      // A block's K and V (without data they still take their places, so that no block
      // is announced far ahead of the other roles), announced with its first copy.
      auto push = [&](int pg) {
        bi.page = pg;
        const CUtensorMap* maps[2] = {&kmap, &vmap};
        if constexpr (FP8) {
          for (int kv = 0; kv < 2; ++kv) {
            const int rb = acquire();
            if (!ok) return;
            if (lane == 0) {
              if (pg < 0) {
                mbar_arrive(&raw_full[rb]);
              } else {
                mbar_arrive_expect_tx(&raw_full[rb], kRaw);
                tma_load_2d(smem + C::kSmRaw + rb * kRaw, maps[kv], bi.head * kHeadDim, pg * kBlock, &raw_full[rb]);
              }
            }
            if (kv == 0) announce();
          }
          return;
        }
        const int there = min(kBlock, bi.seq - bi.t0);
        for (int kv = 0; kv < 2; ++kv) {
          const int b = acquire();
          if (!ok) return;
          uint8_t* dst = smem + b * kTile;
          // V behind the request's end is not data: zeroed before a product reads it
          const bool part = kv == 1 && pg >= 0 && there < kBlock;
          uint64_t* land = part ? fill : &kv_full[b];
          if (lane == 0) {
            if (pg < 0) {
              mbar_arrive(land);
            } else {
              mbar_arrive_expect_tx(land, kTile);
              for (int h = 0; h < 2; ++h)
                tma_load_2d(dst + h * kHalf, maps[kv], bi.head * kHeadDim + 64 * h, pg * kBlock, land);
            }
          }
          if (kv == 0) announce();
          if (part) {
            ok = warp_wait(fill, fills & 1);
            ++fills;
            if (!ok) return;
            uint4* v4 = reinterpret_cast<uint4*>(dst);
            for (int k = there * 8 + lane; k < kBlock * 8; k += 32)
              v4[k] = v4[kHalf / 16 + k] = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&kv_full[b]);
          }
        }
      };
      while (ok && it < sl.end) {
        const PromptReq rq = prompt_request(p.batch, q);
        const Pairs pr = pairs_of(rq, 2 * tpt);
        const long long one = pr.before(pr.tiles), cost = rq.qlen > 0 ? one * Hk : 0;
        if (it >= pre + cost) {
          pre += cost;
          ++q;
          continue;
        }
        const int32_t* table = p.batch.block_table + (long long)q * p.batch.bt_stride;
        if (checked != q) {  // every page of the request, once
          checked = q;
          bad = rq.bad;
          bool odd = false;
#pragma unroll 4
          for (int b = lane; b < rq.nb; b += 32) {
            const int page = __ldg(table + b);
            odd |= page < 0 || page >= p.batch.num_pages;
          }
          if (!bad && __any_sync(0xffffffffu, odd)) bad = MSA_DEV_BAD_PAGE;
        }
        const long long rel = it - pre;
        bi.head = (int)(rel / one);
        const int tile = pr.at(rel % one);
        const long long start = pre + bi.head * one + pr.before(tile);
        const int seen = pr.seen(tile), nv = (seen + kBlock - 1) / kBlock;
        // blocks of the pair in the slice: block b is the CTA's whose slice holds
        // token kPairCost + 128 b of the pair
        const auto block_at = [&](long long u) {
          const long long in = u - start;
          return in <= kPairCost ? 0 : min((long long)nv, (in - kPairCost + kBlock - 1) / kBlock);
        };
        const long long stop = start + kPairCost + seen;
        const int b0 = (int)block_at(it), nb = (int)(stop <= sl.end ? nv : block_at(sl.end)) - b0;
        const long long first = start + kPairCost;
        it = min(stop, sl.end);
        if (nb <= 0) continue;
        const int j0 = tile * 2 * tpt;
        bi.ntok = min(2 * tpt, rq.qlen - j0);
        bi.row0 = rq.q0 + j0;
        bi.pos0 = rq.ctx + j0;
        bi.seq = rq.ctx + rq.qlen;
        bi.slot = 2 * blockIdx.x + (b0 > 0 ? 0 : 1);
        bi.bad = bad;
        const int both = (nb == nv ? kWhole : 0) | (bi.ntok > tpt ? kTwo : 0);
        const auto owner = [&](long long u) { return ((u + 1) * sl.ctas - 1) / sl.total; };
        if (b0 > 0 && owner(first) == (long long)blockIdx.x - 1) {
          rec.nrows = bi.ntok * G;
          rec.row0 = bi.row0;
          rec.head = bi.head;
          rec.last = (int)owner(first + (long long)(nv - 1) * kBlock);
        }
        // (e4m3: the converting warps bring the queries)
        if (!FP8 && n_seg > 0) ok = warp_wait(q_empty, (n_seg - 1) & 1);
        if (!ok) break;
        ++n_seg;
        if (bad) {
          bi.flags = kFirst | kLast | kPoison | kNoData | both;
          bi.t0 = 0;
          if (!FP8 && lane == 0) mbar_arrive(q_full);
          push(-1);
          continue;
        }
        if (!FP8 && lane == 0) {
          const int tiles = both & kTwo ? 2 : 1;
          mbar_arrive_expect_tx(q_full, 2u * tiles * qbytes);
          for (int t = 0; t < tiles; ++t)
            for (int h = 0; h < 2; ++h)
              tma_load_3d(smem + kSmQ + t * kTile + h * kHalf, &qmap, 64 * h, bi.head * G, bi.row0 + t * tpt, q_full);
        }
        const int last0 = bi.pos0 + min(tpt, bi.ntok) - 1, last1 = bi.pos0 + bi.ntok - 1;
        for (int c0 = 0; ok && c0 < nb; c0 += 32) {
          int page = 0;
          if (c0 + lane < nb) page = __ldg(table + b0 + c0 + lane);
          for (int i = 0; ok && i < min(32, nb - c0); ++i) {
            const int pg = __shfl_sync(0xffffffffu, page, i);
            bi.t0 = kBlock * (b0 + c0 + i);
            bi.flags = both | (c0 + i == 0 ? kFirst : 0) | (c0 + i == nb - 1 ? kLast : 0) |
                       (bi.t0 + kBlock - 1 > bi.pos0 ? kMixed : 0) | (last1 >= bi.t0 + 64 ? kHalves : 0) |
                       (c0 + i == 0 || last0 >= bi.t0 ? kWork0 : 0) | (both & kTwo ? kWork1 : 0);
            push(pg);
          }
        }
      }
      if (ok) {
        bi.flags = kEnd;
        announce();
      } else {
        misc[0] = 1;
        // copies still in flight land before the CTA leaves
        const int ring = FP8 ? kRaws : kBufs;
        uint64_t* bars = FP8 ? raw_full : kv_full;
        for (int i = max(0, x - ring); i < x; ++i) mbar_wait(&bars[i % ring], (i / ring) & 1);
        if (!FP8 && n_seg > 0) mbar_wait(q_full, (n_seg - 1) & 1);
      }
      if (lane == 0) p.split[blockIdx.x] = rec;
    };
    const auto products = [&]() {
      // ---------------------------------------------- products
      // Block by block, tile by tile: P V of the two halves as their softmax is done,
      // then S of the next block over the same columns.
      if (lane != 0) return;
      bool ok = mbar_wait(&info_full[0], 0);
      int seg = -1, n = 0, fl = ok ? info[0].flags : kEnd;
      const auto s_of = [&](int t, int blk, int f) {
        if (f & (t ? kWork1 : kWork0)) {
          const uint64_t qd = tc::desc_kmajor_sw128(smem_u32(smem + kSmQ + t * kTile));
          const uint64_t kd = tc::desc_kmajor_sw128(smem_u32(smem + ((2 * blk) % kBufs) * kTile));
          tc::fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
            tc::mma_ss(tmem + col_s(t), tc::desc_advance(qd, off), tc::desc_advance(kd, off), kIdescS,
                       kk > 0 ? 1u : 0u);
          }
        }
        tc::commit(&s_full[t]);
      };
      const auto open = [&](int blk, int f) {  // K (and Q) of a block are there
        bool there = true;
        if (f & kFirst) {
          ++seg;
          there = mbar_wait(q_full, seg & 1);
        }
        return there && mbar_wait(&kv_full[(2 * blk) % kBufs], ((2 * blk) / kBufs) & 1);
      };
      const auto close = [&](int blk, int f) {  // S of both tiles is issued
        tc::commit(&kv_empty[(2 * blk) % kBufs]);
        if (f & kLast) tc::commit(q_empty);
      };
      if (ok && !(fl & kEnd)) {
        ok = open(0, fl);
        if (ok) {
          s_of(0, 0, fl);
          s_of(1, 0, fl);
          close(0, fl);
        }
      }
      while (ok && !(fl & kEnd)) {
        const int vb = (2 * n + 1) % kBufs, seg_now = seg;
        const uint64_t vd = tc::desc_mnmajor_sw128(smem_u32(smem + vb * kTile), kHalf);
        int next = kEnd;
        ok = mbar_wait(&kv_full[vb], ((2 * n + 1) / kBufs) & 1);
        for (int t = 0; ok && t < 2; ++t) {
          const bool work = (fl & (t ? kWork1 : kWork0)) != 0;
          // O of the previous segment has been read
          if ((fl & kFirst) && seg_now > 0) ok = mbar_wait(&o_free[t], (seg_now - 1) & 1);
          ok = ok && mbar_wait(&p_full[2 * t], n & 1);
          if (!ok) break;
          // (the softmax adds the block's P V itself)
          const bool hand = (fl & kMixed) && *reinterpret_cast<volatile int*>(&misc[4 + n % kLooks]) == n + 1;
          const auto pv = [&](int half) {
            if (!work || hand || (half && !(fl & kHalves))) return;
            tc::fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc::mma_ts(tmem + col_o(t), tmem + col_s(t) + half * 32 + kk * 8,
                         tc::desc_advance(vd, (half * 4 + kk) * 2048), kIdescO,
                         (kk > 0 || half > 0 || !(fl & kFirst)) ? 1u : 0u);
          };
          pv(0);
          tc::commit(&pv_half[t]);
          ok = mbar_wait(&p_full[2 * t + 1], n & 1);
          if (!ok) break;
          pv(1);
          tc::commit(&pv_done[t]);
          if (t == 1) tc::commit(&kv_empty[vb]);
          if (t == 0) {
            ok = mbar_wait(&info_full[(n + 1) % kInfos], ((n + 1) / kInfos) & 1);
            if (!ok) break;
            next = info[(n + 1) % kInfos].flags;
            if (!(next & kEnd)) ok = open(n + 1, next);
            if (!ok) break;
          }
          if (!(next & kEnd)) s_of(t, n + 1, next);
        }
        if (!ok) break;
        if (!(next & kEnd)) close(n + 1, next);
        ++n;
        fl = next;
      }
      if (!ok) misc[0] = 1;
      // every product has completed before the tensor memory is freed
      tc::commit(drained);
      if (!mbar_wait(drained, 0)) misc[0] = 1;
    };
    const auto look = [&]() {
      // ---------------------------------------------- values that are not finite
      // in the V of blocks that not every row sees (e4m3: the converting warps look)
      bool ok = true;
      for (int n = 0;; ++n) {
        ok = warp_wait(&info_full[n % kInfos], (n / kInfos) & 1);
        if (!ok) break;
        const int fl = info[n % kInfos].flags;
        if (fl & kEnd) break;
        // (every use of a place is followed, so that the ring never laps this warp)
        const int kb = (2 * n) % kBufs, vb = (2 * n + 1) % kBufs;
        ok = warp_wait(&kv_full[kb], ((2 * n) / kBufs) & 1);
        if (!ok) break;
        if (lane == 0) mbar_arrive(&kv_empty[kb]);
        ok = warp_wait(&kv_full[vb], ((2 * n + 1) / kBufs) & 1);
        if (!ok) break;
        if ((fl & kMixed) && !(fl & kNoData)) {
          const uint8_t* src = smem + vb * kTile + lane * 16;
          uint32_t odd = 0;
#pragma unroll 8
          for (int i = 0; i < kTile; i += 512) {
            const uint4 v = lds128(src + i);
            constexpr uint32_t one = 0x00800080u;  // an exponent's last bit
            odd |= (v.x & 0x7fff7fffu) + one;
            odd |= (v.y & 0x7fff7fffu) + one;
            odd |= (v.z & 0x7fff7fffu) + one;
            odd |= (v.w & 0x7fff7fffu) + one;
          }
          const bool any = __any_sync(0xffffffffu, (odd & 0x80008000u) != 0);
          if (lane == 0 && any) *reinterpret_cast<volatile int*>(&misc[4 + n % kLooks]) = n + 1;
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&looked[n % kLooks]);
          mbar_arrive(&kv_empty[vb]);
        }
      }
      if (!ok) misc[0] = 1;
    };
    // the scales of token ct of block n (a warp's 32 at a time), k's with the softmax's own
    const auto scales_of = [&](const BlockInfo& bi, int fl, int n, int ct) {
      float ks = 0.f, vs = 0.f;
      const bool data = !(fl & kNoData) && bi.t0 + ct < bi.seq;
      if (data) {
        const long long at = ((long long)bi.page * kBlock + ct) * Hk + bi.head;
        ks = __ldg(p.k_scale + at) * (p.softmax_scale * kTreeLog2e);
        vs = __ldg(p.v_scale + at);
      }
      float* sc = reinterpret_cast<float*>(smem + C::kSmScale) + (n % kScales) * kScaleWords;
      sc[ct] = ks;
      sc[kSoV + ct] = vs;
      sc[kSoLog + ct] = log2_scale(vs);
      const uint32_t mag = scale_bits(vs);
      const uint32_t hi = __reduce_max_sync(0xffffffffu, data ? mag : 0u);
      const uint32_t lo = __reduce_min_sync(0xffffffffu, data ? mag : ~0u);
      if (lane == 0)
        reinterpret_cast<float2*>(sc + kSoRange)[ct >> 5] = make_float2(bits_log2(hi), bits_log2(lo));
    };
    const auto scales = [&]() {
      // ---------------------------------------------- scales per token of bf16 pools
      bool ok = true;
      for (int n = 0;; ++n) {
        ok = warp_wait(&info_full[n % kInfos], (n / kInfos) & 1);
        if (!ok) break;
        const BlockInfo& bi = info[n % kInfos];
        const int fl = bi.flags;
        if (fl & kEnd) break;
        // (a block is announced when its K has a place, which S of block n - 2 freed: the
        // softmax is through with this place's block n - 4)
        for (int i = 0; i < 4; ++i) scales_of(bi, fl, n, 32 * i + lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_full[n % kScales]);
      }
      if (!ok) misc[0] = 1;
    };
    const auto convert = [&]() {
      // ---------------------------------------------- e4m3 tiles to f16, queries
      const int ct = tid - 12 * 32;
      int x = 0, seg = -1;  // tiles, segments
      bool ok = true;
      for (int n = 0;; ++n) {
        ok = warp_wait(&info_full[n % kInfos], (n / kInfos) & 1);
        if (!ok) break;
        const BlockInfo& bi = info[n % kInfos];
        const int fl = bi.flags;
        if (fl & kEnd) break;
        if (fl & kFirst) {
          ++seg;
          if (seg > 0) ok = warp_wait(q_empty, (seg - 1) & 1);
          if (!ok) break;
          if (!(fl & kPoison)) {
#pragma unroll 8
            for (int i = ct; i < 2 * 128 * 16; i += kConv * 32) {
              const int t = i >> 11, m = (i >> 4) & 127, ch = i & 15;
              const int mt = m / G, tok = t * tpt + mt;
              uint4 v = make_uint4(0u, 0u, 0u, 0u);
              if (mt < tpt && tok < bi.ntok)
                v = __ldg(reinterpret_cast<const uint4*>(
                              p.q + (((long long)bi.row0 + tok) * H + bi.head * G + (m - mt * G)) * kHeadDim) + ch);
              v.x = pack_f16x2(bf16lo(v.x), bf16hi(v.x));
              v.y = pack_f16x2(bf16lo(v.y), bf16hi(v.y));
              v.z = pack_f16x2(bf16lo(v.z), bf16hi(v.z));
              v.w = pack_f16x2(bf16lo(v.w), bf16hi(v.w));
              *reinterpret_cast<uint4*>(smem + kSmQ + t * kTile + (ch >> 3) * kHalf + m * 128 +
                                        (((ch & 7) ^ (m & 7)) << 4)) = v;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_full);
        }
        if constexpr (PTH) {
          // (the block's K has an e4m3 place, so V of block n - 2 is converted, over K of block
          // n - 3 that its S has read: the softmax is through with block n - 4's scales)
          scales_of(bi, fl, n, ct);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[n % kScales]);
        }
        for (int kv = 0; ok && kv < 2; ++kv, ++x) {
          const int b = x % kBufs, rb = x % kRaws;
          if (x >= kBufs) ok = warp_wait(&kv_empty[b], ((x / kBufs) - 1) & 1);
          ok = ok && warp_wait(&raw_full[rb], (x / kRaws) & 1);
          if (!ok) break;
          if (!(fl & kNoData)) {
            // (rows of 128 bytes, 16-byte chunks swizzled by the copy)
            const uint8_t* raw = smem + C::kSmRaw + rb * kRaw;
            uint8_t* tile = smem + b * kTile;
            const int there = min(kBlock, bi.seq - bi.t0);  // behind it: not data, zeros
            uint32_t odd = 0;
#pragma unroll 2
            for (int i = ct; i < kRaw / 16; i += kConv * 32) {
              const int row = i >> 3, c = i & 7, ch = 2 * c;  // 16 codes: f16 chunks ch, ch + 1
              uint4 v = lds128(raw + row * 128 + ((c ^ (row & 7)) << 4));
              if (row >= there) v = make_uint4(0u, 0u, 0u, 0u);
              // (a code of NaN: 0x7f without its sign)
              odd |= ((v.x & 0x7f7f7f7fu) + 0x01010101u) | ((v.y & 0x7f7f7f7fu) + 0x01010101u) |
                     ((v.z & 0x7f7f7f7fu) + 0x01010101u) | ((v.w & 0x7f7f7f7fu) + 0x01010101u);
              uint8_t* dst = tile + (ch >> 3) * kHalf + row * 128;
              *reinterpret_cast<uint4*>(dst + (((ch & 7) ^ (row & 7)) << 4)) =
                  make_uint4(e4m3x2_to_f16x2((uint16_t)v.x), e4m3x2_to_f16x2((uint16_t)(v.x >> 16)),
                             e4m3x2_to_f16x2((uint16_t)v.y), e4m3x2_to_f16x2((uint16_t)(v.y >> 16)));
              *reinterpret_cast<uint4*>(dst + ((((ch & 7) + 1) ^ (row & 7)) << 4)) =
                  make_uint4(e4m3x2_to_f16x2((uint16_t)v.z), e4m3x2_to_f16x2((uint16_t)(v.z >> 16)),
                             e4m3x2_to_f16x2((uint16_t)v.w), e4m3x2_to_f16x2((uint16_t)(v.w >> 16)));
            }
            fence_proxy_async_smem();
            if (kv == 1 && (fl & kMixed) && (odd & 0x80808080u))
              *reinterpret_cast<volatile int*>(&misc[4 + n % kLooks]) = n + 1;
            __syncwarp();
          }
          if (lane == 0) {
            mbar_arrive(&raw_empty[rb]);
            mbar_arrive(&kv_full[b]);
          }
        }
        if (!ok) break;
      }
      if (!ok) misc[0] = 1;
    };
    const auto softmax = [&]() {
      // ---------------------------------------------- softmax of tile t
      const int t = (warp - 4) >> 2, quarter = warp & 3;
      const int m = quarter * 32 + lane;  // row of the tile
      const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
      const uint32_t sa = tmem + lanes + col_s(t), oa = tmem + lanes + col_o(t);
      const int mtok = m / G, tok = t * tpt + mtok;  // token of the pair
      float scale2 = p.softmax_scale * kTreeLog2e, vs = 1.f;
      if (p.scale_mode == MSA_SCALE_SCALAR) {
        scale2 *= __ldg(p.k_scale);
        vs = __ldg(p.v_scale);
      }
      float m_run = -INFINITY, l_run = 0.f;
      constexpr float kHead = FP8 ? kHalfHead : 0.f;
      bool ok = true;
      for (int n = 0;; ++n) {
        ok = warp_wait(&info_full[n % kInfos], (n / kInfos) & 1);
        if (!ok) break;
        const BlockInfo& bi = info[n % kInfos];
        const int fl = bi.flags;
        if (fl & kEnd) break;
        const int vb = (2 * n + 1) % kBufs;
        if (fl & kFirst) {
          m_run = -INFINITY;
          l_run = 0.f;
        }
        const bool there = mtok < tpt && tok < bi.ntok;
        const bool work = (fl & (t ? kWork1 : kWork0)) != 0;
        bool masked = (fl & kMixed) != 0;
        uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
        if (masked) {
          const int seen = there ? bi.pos0 + tok + 1 - bi.t0 : 0;  // tokens of the block that the row sees
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int c = seen - 32 * w;
            vis[w] = c >= 32 ? ~0u : c > 0 ? (1u << c) - 1u : 0u;
          }
          masked = !__all_sync(0xffffffffu, seen >= kBlock || !there);
        }
        bool hand = false;
        float moved = 1.f;  // what the second half scaled the first one's P by
        const float* ks = nullptr;
        // (PTH, by half) log2 of the largest v scale; whether the scales lie too far apart for it
        float near0 = 0.f, near1 = 0.f;
        bool exact0 = false, exact1 = false;
        if (PTH) {
          ok = warp_wait(&sc_full[n % kScales], (n / kScales) & 1);
          if (!ok) break;
          ks = reinterpret_cast<const float*>(smem + C::kSmScale) + (n % kScales) * kScaleWords;
          const float4 r0 = *reinterpret_cast<const float4*>(ks + kSoRange);
          const float4 r1 = *reinterpret_cast<const float4*>(ks + kSoRange + 4);
          near0 = fmaxf(r0.x, r0.z);
          near1 = fmaxf(r1.x, r1.z);
          exact0 = near0 - fminf(r0.y, r0.w) > kNear;
          exact1 = near1 - fminf(r1.y, r1.w) > kNear;
        }
        ok = warp_wait(&s_full[t], n & 1);
        if (!ok) break;
        tc::fence_after();
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (work && (half == 0 || (fl & kHalves))) {
            const uint32_t v0 = half ? vis[2] : vis[0], v1 = half ? vis[3] : vis[1];
            const float* kh = PTH ? ks + 64 * half : nullptr;
            uint32_t r[64];
            tc::tmem_ld64(sa + 64 * half, r);
            // (with PTH the tokens' factors carry the softmax scale and its sign)
            const float sg = PTH ? 1.f : scale2;
            const bool exact = PTH && (half ? exact1 : exact0);
            const float near = half ? near1 : near0;
            float mx;
            if (exact)
              mx = max64<false, true, PTH, true>(r, -INFINITY, v0, v1, kh, kh + kSoLog);
            else if (masked)
              mx = sg >= 0.f ? max64<false, true, PTH>(r, -INFINITY, v0, v1, kh) * sg
                             : max64<true, true, PTH>(r, -INFINITY, v0, v1, kh) * -sg;
            else
              mx = sg >= 0.f ? max64<false, false, PTH>(r, -INFINITY, v0, v1, kh) * sg
                             : max64<true, false, PTH>(r, -INFINITY, v0, v1, kh) * -sg;
            mx += exact ? -kHead : near - kHead;
            const bool move = there && (mx > m_run + kSlack || (m_run == -INFINITY && mx > -INFINITY));
            if (__any_sync(0xffffffffu, move)) {
              float al = 1.f;
              if (there && mx > m_run) {
                al = m_run == -INFINITY ? 1.f : ex2_ftz(m_run - mx);
                m_run = mx;
              }
              l_run *= al;
              if (half) moved = al;
              // (a row without a reference has an all-zero O: nothing to rescale.  P V of
              // the block before is complete: this block's S came behind it)
              if (!((fl & kFirst) && half == 0) && __any_sync(0xffffffffu, al != 1.f)) {
                if (half) {
                  ok = warp_wait(&pv_half[t], n & 1);
                  if (!ok) break;
                }
                tc::fence_after();
#pragma unroll 1
                for (int c = 0; c < 128; c += 16) {
                  uint32_t x[16];
                  tc::tmem_ld16(oa + c, x);
#pragma unroll
                  for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * al);
                  tc::tmem_st16(oa + c, x);
                }
              }
            }
            const float base = m_run == -INFINITY ? 0.f : m_run;
            const float* vh = PTH ? kh + kSoV : nullptr;
            // P of the halves side by side, over logits that have been read
            const uint32_t pa = sa + 32 * half;
            l_run += masked ? exp64<true, FP8, PTH>(r, pa, scale2, base, v0, v1, kh, vh)
                            : exp64<false, FP8, PTH>(r, pa, scale2, base, v0, v1, kh, vh);
            tc::tmem_wait_st();
            tc::fence_before();
          }
          if (half == 0 && (fl & kMixed) && !(fl & kNoData)) {
            ok = FP8 ? warp_wait(&kv_full[vb], ((2 * n + 1) / kBufs) & 1)
                     : warp_wait(&looked[n % kLooks], (n / kLooks) & 1);
            if (!ok) break;
            hand = *reinterpret_cast<volatile int*>(&misc[4 + n % kLooks]) == n + 1;
          }
          __syncwarp();
          if (lane == 0 && !(hand && half)) mbar_arrive(&p_full[2 * t + half]);
          __syncwarp();
        }
        if (!ok) break;
        if (hand) {
          if (work) {
            tc::fence_after();
            pv_by_hand<FP8>(oa, sa, smem + vb * kTile, make_uint4(vis[0], vis[1], vis[2], vis[3]),
                            fl & kHalves ? 4 : 2, moved, (fl & kFirst) != 0);
            tc::tmem_wait_st();
            tc::fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * t + 1]);
        }
        if (fl & kLast) {
          ok = warp_wait(&pv_done[t], n & 1);
          if (!ok) break;
          tc::fence_after();
          const int hh = bi.head * G + (m - mtok * G);
          const float sink = p.sinks && there ? __ldg(p.sinks + hh) : 0.f;
          const bool none = (fl & kPoison) || (m_run == -INFINITY && l_run == 0.f);
          const TreeRowEnd e = tree_row_end(none ? -INFINITY : m_run, none ? 0.f : l_run,
                                            p.sinks != nullptr, sink * kTreeLog2e, vs);
          const bool have = (t == 0 || (fl & kTwo)) && !(fl & kPoison);
          const long long r = ((long long)bi.row0 + tok) * H + hh;  // row x head in the batch
          const int pm = t * tpt * G + m;  // row of the pair
          const long long pr = (long long)bi.slot * 256 + pm;
          __syncwarp();
          if (have) {
#pragma unroll 1
            for (int c = 0; c < 128; c += 16) {
              uint32_t v[16];
              tc::tmem_ld16(oa + c, v);
              if (there && (fl & kWhole)) {
                uint4* dst = reinterpret_cast<uint4*>(p.out + r * kHeadDim + c);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  uint32_t w[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    w[k] = none ? 0u
                                : pack_bf16x2(__uint_as_float(v[8 * i + 2 * k]) * e.f,
                                              __uint_as_float(v[8 * i + 2 * k + 1]) * e.f);
                  dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
              } else if (there) {
                // [4-dim group][row][4 dims]: the warp's rows are contiguous
                uint4* dst = reinterpret_cast<uint4*>(p.part_o) + ((long long)bi.slot * 32 + c / 4) * 256 + pm;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  dst[256 * i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
              }
              __syncwarp();
            }
          } else if (there) {  // a poisoned request's rows
            uint4* dst = reinterpret_cast<uint4*>(p.out + r * kHeadDim);
            for (int i = 0; i < kHeadDim / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
          }
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_free[t]);
          if (there) {
            if (fl & (kWhole | kPoison)) p.lse[r] = none ? (p.sinks ? sink : -INFINITY) : e.lse;
            else p.part_ml[pr] = make_float2(m_run, l_run);
          }
          if (t == 0 && m == 0) {
            if (!(fl & kWhole)) p.part_bad[bi.slot] = fl & kPoison ? 1 : 0;
            if (bi.bad) atomicOr(p.status, bi.bad);
          }
        }
      }
      if (!ok) misc[0] = 1;
    };
    if constexpr (FP8) {
      // (a warpgroup's warps give and take registers together)
      if (warp < 4) {
        regs_fewer<kRegsFew>();
        if (warp == 0) copies();
        else if (warp == 1) products();
      } else if (warp >= 12) {
        regs_fewer<kRegsFew>();
        convert();
      } else {
        regs_more<kRegsMore>();
        softmax();
      }
    } else if (warp == 0) {
      copies();
    } else if (warp == 1) {
      products();
    } else if (warp == 2) {
      if (PTH) scales();
    } else if (warp == 3) {
      look();
    } else {
      softmax();
    }
  }
  tc::fence_before();
  __syncthreads();
  if (misc[0] && tid == 0) atomicOr(p.status, MSA_DEV_TIMEOUT);
  if (warp == 1) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------ join

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kMaxMainCtas = 512;  // (the main kernel runs one CTA per SM)

// Threads x 4 dims that share a row's partials: a unit is 8 / parts rows
__device__ __forceinline__ int join_parts(int n) {
  return n <= 8 ? 1 : n <= 16 ? 2 : n <= 64 ? 4 : 8;
}

// Joins the partials of the pairs that several CTAs share.
__global__ void __launch_bounds__(kJoinThreads, 3)
    prompt_join_kernel(const __grid_constant__ PromptLaunch p, int grid_main) {
  __shared__ float4 s_o[kJoinThreads];
  __shared__ float s_m[8], s_l[8];
  __shared__ int s_bad[8], s_sum[kJoinWarps], s_base[kMaxMainCtas];
  __shared__ PromptSplit s_rec[kMaxMainCtas];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = p.num_heads, G = H / p.num_kv_heads;
  const float vs = p.scale_mode == MSA_SCALE_SCALAR ? __ldg(p.v_scale) : 1.f;
  // the split pairs' work units, by a prefix sum over the records
  int total = 0;
  for (int c0 = 0; c0 < grid_main; c0 += kJoinThreads) {
    const int c = c0 + threadIdx.x;
    PromptSplit rec;
    rec.nrows = 0;
    rec.last = c;
    if (c > 0 && c < grid_main) rec = p.split[c];
    const int per = 8 / join_parts(rec.last - c + 2);
    const int units = (rec.nrows + per - 1) / per;
    int x = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    if (c < grid_main) {
      int before = x - units;
      for (int w = 0; w < warp; ++w) before += s_sum[w];
      s_base[c] = total + before;
      s_rec[c] = rec;
    }
    for (int w = 0; w < kJoinWarps; ++w) total += s_sum[w];
    __syncthreads();
  }
  for (int unit = blockIdx.x; unit < total; unit += gridDim.x) {
    int lo = 0, hi = grid_main - 1;  // last record whose first unit is <= unit
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_base[mid] <= unit) lo = mid; else hi = mid - 1;
    }
    const int c = lo;
    const PromptSplit rec = s_rec[c];
    const int n = rec.last - c + 2;  // partials: CTAs c - 1 .. last
    const int parts = join_parts(n), per = 8 / parts;
    // neighbouring threads take the unit's rows, then the 4-dim groups, then the parts
    const int row = threadIdx.x & (per - 1), x = threadIdx.x / per;
    const int g = x & 31, part = x >> 5;
    const int m = (unit - s_base[c]) * per + row;
    const bool live = m < rec.nrows;
    float M = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    int bad = 0;
    constexpr int kLoads = 4;  // partials that a thread has in flight
    if (live) {
      for (int i0 = part; i0 < n; i0 += kLoads * parts) {
        float2 ml[kLoads];
        float4 v[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const int i = i0 + u * parts;
          ml[u] = make_float2(-INFINITY, 0.f);
          v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < n) {
            const long long slot = 2ll * (c - 1 + i) + (i == 0 ? 1 : 0);
            bad |= p.part_bad[slot];
            ml[u] = p.part_ml[slot * 256 + m];
            v[u] = reinterpret_cast<const float4*>(p.part_o)[(slot * 32 + g) * 256 + m];
          }
        }
        float mn = M;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) mn = fmaxf(mn, ml[u].x);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float f0 = M == -INFINITY ? 1.f : ex2_ftz(M - ref);
        L *= f0;
        a.x *= f0; a.y *= f0; a.z *= f0; a.w *= f0;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const float f = ml[u].x == -INFINITY ? 1.f : ex2_ftz(ml[u].x - ref);
          L += ml[u].y * f;
          a.x += v[u].x * f; a.y += v[u].y * f; a.z += v[u].z * f; a.w += v[u].w * f;
        }
        M = mn;
      }
    }
    if (parts > 1) {
      __syncthreads();  // the previous unit's sums have been read
      s_o[threadIdx.x] = a;
      if (g == 0) {
        s_m[part * per + row] = M;
        s_l[part * per + row] = L;
        s_bad[part * per + row] = bad;
      }
      __syncthreads();
      if (part == 0) {
        for (int k = 1; k < parts; ++k) {
          bad |= s_bad[k * per + row];
          M = fmaxf(M, s_m[k * per + row]);
        }
        const float ref = M == -INFINITY ? 0.f : M;
        L = 0.f;
        a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < parts; ++k) {
          const float mk = s_m[k * per + row], f = mk == -INFINITY ? 1.f : ex2_ftz(mk - ref);
          const float4 o = s_o[k * 32 * per + threadIdx.x];
          L += s_l[k * per + row] * f;
          a.x += o.x * f; a.y += o.y * f; a.z += o.z * f; a.w += o.w * f;
        }
      }
      __syncthreads();  // read before the next unit overwrites them
    }
    if (live && part == 0) {
      const bool none = bad || (M == -INFINITY && L == 0.f);
      const int h = rec.head * G + m % G;
      const float sink = p.sinks ? __ldg(p.sinks + h) : 0.f;
      const TreeRowEnd e = tree_row_end(M, L, p.sinks != nullptr, sink * kTreeLog2e, vs);
      const long long r = ((long long)rec.row0 + m / G) * H + h;
      uint2 w = make_uint2(pack_bf16x2(a.x * e.f, a.y * e.f), pack_bf16x2(a.z * e.f, a.w * e.f));
      if (none) w = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(p.out + r * kHeadDim + 4 * g) = w;
      if (g == 0) p.lse[r] = none ? (p.sinks ? sink : -INFINITY) : e.lse;
    }
  }
}

template <bool FP8, bool PTH>
cudaError_t launch(const PromptLaunch& p, cudaStream_t stream) {
  using C = PaCfg<FP8, PTH>;
  const int G = p.num_heads / p.num_kv_heads, tpt = 128 / G;
  CUtensorMap qmap, kmap, vmap;
  memset(&qmap, 0, sizeof(qmap));
  const long long toks = max(1ll, (long long)p.batch.num_pages) * kBlock;
  const long long inner = (long long)p.num_kv_heads * kHeadDim;
  const auto type = FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int size = FP8 ? 1 : 2, box = 128 / size;  // 128 bytes
  if (!encode_map_2d(&kmap, type, p.k, inner, toks, inner * size, box, kBlock) ||
      !encode_map_2d(&vmap, type, p.v, inner, toks, inner * size, box, kBlock) ||
      (!FP8 && !encode_map_3d(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.q, kHeadDim, p.num_heads,
                              p.batch.num_rows, kHeadDim * 2, (long long)p.num_heads * kHeadDim * 2, 64, G, tpt)))
    return cudaErrorInvalidValue;
  const int grid = device_sm_count();
  auto kern = prompt_attn_kernel<FP8, PTH>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e != cudaSuccess) return e;
  kern<<<grid, C::kThreads, C::kBytes, stream>>>(p, qmap, kmap, vmap);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(3 * grid);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prompt_join_kernel, p, grid);
}

}  // namespace

cudaError_t launch_prompt_attn(const PromptLaunch& p, cudaStream_t stream) {
  const bool pth = p.scale_mode == MSA_SCALE_PER_TOKEN_HEAD;
  if (p.kv_fp8) return pth ? launch<true, true>(p, stream) : launch<true, false>(p, stream);
  return pth ? launch<false, true>(p, stream) : launch<false, false>(p, stream);
}

}  // namespace msa
