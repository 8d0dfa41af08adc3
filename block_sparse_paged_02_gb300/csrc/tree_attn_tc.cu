// tree_attn_tc.cu -- the draft-tree attention for wide trees (more than 32
// rows x heads per request) on the 5th-generation tensor cores.
//
// Same mathematics, split and partials as tree_attn.cu.  A request's rows are
// cut into pairs of 128-row tiles; a CTA loads each visited block's K and V
// once for both tiles, and while one tile is in its softmax the tensor cores
// work on the other:
//   S = Q K^T   tcgen05.mma M128 N64 or N128 K128, both operands in shared memory
//   P = 2^(S' - m)  one thread per row (TMEM lane), 64 logits at a time in
//               registers; the running reference m moves only when a step's
//               maximum exceeds it by more than 2^8 (then that warp rescales
//               its rows of O); P written back over S in 16 bits
//   O += P V    tcgen05.mma with A = P from tensor memory, B = V (MN-major)
// Roles: warp 0 issues the tensor copies, one thread of warps 1 and 2 issues the
// products of tile 0 and tile 1, warp 3 looks bf16 V over (below), warps 4-7 and
// 8-11 are the tiles' softmax.  Tensor memory (512 columns): S / P and O of both
// tiles.  With e4m3 pools warps 12-15 turn the tiles into f16 (exact) and the
// products run in f16; a scale per token joins the logits and P in the softmax.
// (bf16 pools with a scale per token stay on tree_attn.cu.)
//
// Measured: 8 requests of 48..64 rows x 16 heads over 8192..32768 bf16 tokens 83 us,
// 65 GFLOP (780 TFLOP/s; 34 us at cuBLAS's rate, 13 for its 126 M exponentials at 32 a
// clock and SM); 2 of 33 rows x 12 heads over 131K e4m3 tokens with scales 102 us; 16 of
// 16..32 rows that select 16 blocks each 42 us.
// Bound by the chain of a block through S, softmax and P V at two tiles a CTA: the
// wide trees take 79 us without the 2^x, 81 with a quarter of the products, 64
// without both, of which 5 go by before the first product and 11 in the merge.
//
// A block that not every row sees whole (the drafted tokens, the context's
// end, selected blocks) takes a masked softmax, and its V is looked over: a
// value that is not finite would reach rows that do not see it through 0 * V,
// so that block's P V is then added to O row by row, from the visible tokens
// alone (pv_by_hand).
#include <string.h>

#include "attn_tc.cuh"

namespace msa {
namespace {

constexpr int kInfos = 8;
// flags of a block
constexpr int kFirst = 1, kLast = 2, kWhole = 4, kNoData = 8, kBadPage = 16, kPoison = 32,
              kEnd = 64, kMixed = 128, kTwo = 256, kHalves = 512;

struct BlockInfo {
  int flags;
  int row0, ntok, j0;  // the tile pair's drafted tokens: first row in the batch, count, index
  int ctx, qlen, seq;
  int t0;              // position of the block's first token
  int slot;
  uint32_t bad;
  int page;
  const uint32_t* rows;
};

// blocks that the warp looking V over may be ahead of the softmax, and one more (both
// rings of tiles hold it to two)
constexpr int kLooks = 4;
constexpr int kConv = 4;    // converting warps (e4m3 pools)

// e4m3: 512 threads are launched with 128 registers each; the softmax warpgroups take
// 24 more from the two others (104 + 152 + 152 + 104 = 4 * 128), which ends their
// spills: 117 us without, 102.5 with it for 2 requests of 33 rows x 12 heads over 131K
// tokens with scales, 103 with 160 and 96
constexpr int kRegsFew = 104, kRegsMore = 152;
template <bool FP8, bool PTH>
struct TcCfg {
  // (e4m3: 512 threads, 128 registers each; else 384, 168)
  static constexpr int kThreads = FP8 ? 512 : 384;
  static constexpr bool kAhead = !FP8;       // S of the next block before P V of this
  static constexpr int kBufs = FP8 ? 3 : 5;  // ring of 16-bit K and V tiles, alternating
  static constexpr int kRaws = FP8 ? 3 : 0;  // ring of e4m3 tiles
  static constexpr int kSmKv = 0;
  static constexpr int kSmQ = kBufs * kTile;
  static constexpr int kSmRaw = kSmQ + 2 * kTile;
  static constexpr int kSmScale = kSmRaw + kRaws * kRaw;
  static constexpr int kSmInfo = kSmScale + (PTH ? kScales * kScaleWords * 4 : 0);
  static constexpr int kSmBars = kSmInfo + kInfos * (int)sizeof(BlockInfo);
  // kv full / empty, raw full / empty, q full / empty, info full, scales full;
  // per tile: s_full, p_full and pv_done of the two halves, s_read, o_free, drained;
  // fill, looked
  static constexpr int kNumBars = 2 * kBufs + 2 * kRaws + 2 + kInfos + kScales + 18 + 1 + kLooks;
  static constexpr int kSmMisc = kSmBars + kNumBars * 8;
  static constexpr int kBytes = kSmMisc + 64;
  static_assert(kBytes <= 227 * 1024, "shared memory");
  static_assert(sizeof(BlockInfo) % 8 == 0 && kSmBars % 8 == 0, "alignment");
};

constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t col_s(int t) { return 128u * t; }
__device__ __forceinline__ uint32_t col_o(int t) { return 256u + 128u * t; }

template <bool FP8, bool PTH>
__global__ void __launch_bounds__(TcCfg<FP8, PTH>::kThreads, 1)
    tree_attn_tc_kernel(const __grid_constant__ TreeLaunch p, const __grid_constant__ CUtensorMap qmap,
                        const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
  using C = TcCfg<FP8, PTH>;
  constexpr int kBufs = C::kBufs, kRaws = C::kRaws, kThreads = C::kThreads;
  constexpr int kSmKv = C::kSmKv, kSmQ = C::kSmQ;
  constexpr bool kAhead = C::kAhead;
  constexpr int kSTok = kAhead ? 64 : 128;  // tokens of a product S
  constexpr uint32_t kIdescS = tc::idesc_16(128, kSTok, 0, FP8 ? 0 : 1);
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
  uint64_t* s_full = sc_full + kScales;  // [tile][half]
  uint64_t* p_full = s_full + 4;         // [tile][half]
  uint64_t* pv_done = p_full + 4;        // [tile][half]
  uint64_t* s_read = pv_done + 4;        // [tile]: the second half's logits are in registers
  uint64_t* o_free = s_read + 2;         // [tile]
  uint64_t* fill = o_free + 2;
  uint64_t* drained = fill + 1;          // [tile]
  uint64_t* looked = drained + 2;        // [kLooks]
  BlockInfo* info = reinterpret_cast<BlockInfo*>(smem + C::kSmInfo);
  int* misc = reinterpret_cast<int*>(smem + C::kSmMisc);  // [0] timeout, [4 + n % kLooks] n + 1: odd values in block n's V
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 8);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = p.num_heads;
  const int tpt = 128 / H;  // drafted tokens per tile

  if (tid == 0) {
    for (int i = 0; i < 8; ++i) misc[i] = 0;
    for (int s = 0; s < kBufs; ++s) {
      mbar_init(&kv_full[s], FP8 ? kConv : 1);
      mbar_init(&kv_empty[s], FP8 ? 2 : 3);  // the two issuers, the warp that looks V over
    }
    for (int s = 0; s < kRaws; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], kConv);
    }
    for (int s = 0; s < kScales; ++s) mbar_init(&sc_full[s], kConv);
    mbar_init(q_full, FP8 ? kConv : 1);
    mbar_init(q_empty, 2);
    for (int i = 0; i < kInfos; ++i) mbar_init(&info_full[i], 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_read[t], 4);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&s_full[2 * t + b], 1);
        mbar_init(&p_full[2 * t + b], 4);
        mbar_init(&pv_done[2 * t + b], 1);
      }
      mbar_init(&o_free[t], 4);
      mbar_init(&drained[t], 1);
    }
    mbar_init(fill, 1);
    for (int i = 0; i < kLooks; ++i) mbar_init(&looked[i], 1);
    fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, kTmemCols);
  const TreeSlice sl = tree_slice<kThreads>(
      p, [&](const TreeReq& r, int nv) { return tree_items(nv, (r.qlen + 2 * tpt - 1) / (2 * tpt)); },
      reinterpret_cast<long long*>(smem));
  fence_proxy_async_smem();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0 && sl.begin >= sl.end) p.split[blockIdx.x].nrows = 0;
  if (!sl.tiled) {
    tree_write_all_empty(p);
    if (tid == 0 && blockIdx.x == 0) atomicOr(p.status, MSA_DEV_MALFORMED);
  }

  if (sl.begin < sl.end) {
    const auto copies = [&]() {
      // ---------------------------------------------- copies
      long long it = sl.begin, pre = sl.pre;
      int q = sl.q, n = 0, n_seg = 0, x = 0, fills = 0;  // blocks, segments, ring uses
      bool ok = true;
      TreeSplit rec;
      rec.nrows = 0;
      auto acquire = [&]() -> int {
        constexpr int ring = FP8 ? kRaws : kBufs;
        uint64_t* freed = FP8 ? raw_empty : kv_empty;
        const int b = x % ring;
        if (x >= ring) ok = ok && warp_wait(&freed[b], ((x / ring) - 1) & 1);
        ++x;
        return b;
      };
      auto announce = [&](const BlockInfo& bi) {
        if (lane == 0) {
          info[n % kInfos] = bi;
          mbar_arrive(&info_full[n % kInfos]);
        }
        ++n;
      };
      BlockInfo bi;
      bi.page = 0;
      // e4m3: a block's two tiles (none for pg < 0, which still takes its places in
      // the ring, so that no block is announced far ahead of the other roles);
      // announced with the first, as the second may have to wait for a place that
      // the announced block's conversion frees
      auto push = [&](BlockInfo& b, int pg) {
        const uint8_t* src[2] = {p.k, p.v};
        b.page = pg;
        for (int kv = 0; kv < 2; ++kv) {
          const int rb = acquire();
          if (!ok) return;
          if (lane == 0) {
            if (pg < 0) {
              mbar_arrive(&raw_full[rb]);
            } else {
              mbar_arrive_expect_tx(&raw_full[rb], kRaw);
              bulk_g2s(smem + C::kSmRaw + rb * kRaw, src[kv] + (long long)pg * kRaw, kRaw, &raw_full[rb]);
            }
          }
          if (kv == 0) announce(b);
        }
      };
      while (ok && it < sl.end) {
        TreeReq rq = sl.first;
        int nv = sl.visits;
        if (q != sl.q) {
          rq = tree_request(p, q);
          nv = rq.qlen > 0 ? tree_visits(p, q, rq) : 0;
        }
        const int tiles = (rq.qlen + 2 * tpt - 1) / (2 * tpt);
        const long long cost = nv > 0 ? tree_items(nv, tiles) : 0;
        if (it >= pre + cost) {
          pre += cost;
          ++q;
          continue;
        }
        const TreeSeg sg = tree_segment(it, sl.end, pre, nv);
        const int tile = sg.tile, b0 = sg.b0, nb = sg.nb;
        it = sg.next;
        if (nb == 0) continue;
        bi.j0 = tile * 2 * tpt;
        bi.ntok = min(2 * tpt, rq.qlen - bi.j0);
        bi.row0 = rq.q0 + bi.j0;
        bi.ctx = rq.ctx;
        bi.qlen = rq.qlen;
        bi.seq = rq.ctx + rq.qlen;
        bi.slot = 2 * blockIdx.x + (b0 > 0 ? 0 : 1);
        bi.bad = rq.bad;
        bi.rows = nullptr;
        const int both = (nb == nv ? kWhole : 0) | (bi.ntok > tpt ? kTwo : 0);
        if (b0 > 0 && sl.total * (blockIdx.x - 1) / sl.ctas <= sg.first) {
          rec.nrows = bi.ntok * H;
          rec.row0 = bi.row0;
          rec.last = (int)((sg.end * sl.ctas - 1) / sl.total);
        }
        // (e4m3: the converting warps bring the queries, and pass over empty blocks)
        if (!FP8 && n_seg > 0) ok = warp_wait(q_empty, (n_seg - 1) & 1);
        if (!ok) break;
        ++n_seg;
        if (rq.bad && FP8) {
          bi.flags = kFirst | kLast | kPoison | kNoData | kWhole | both;
          bi.t0 = 0;
          push(bi, -1);
          if (!ok) break;
        } else if (rq.bad) {
          bi.flags = kFirst | kLast | kPoison | kNoData | kWhole | both;
          bi.t0 = 0;
          const int kb = acquire(), vb = acquire();
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive(q_full);
            mbar_arrive(&kv_full[kb]);
            mbar_arrive(&kv_full[vb]);
          }
          announce(bi);
        } else if (!FP8 && lane == 0) {
          mbar_arrive_expect_tx(q_full, (both & kTwo ? 2 : 1) * kTile);
          for (int t = 0; t < (both & kTwo ? 2 : 1); ++t)
            for (int h = 0; h < 2; ++h)
              tma_load_2d(smem + kSmQ + t * kTile + h * kHalf, &qmap, 64 * h,
                          (bi.row0 + t * tpt) * H, q_full);
        }
        for (int c0 = 0; !rq.bad && ok && c0 < nb; c0 += 32) {
          int blk = 0, page = 0;
          if (c0 + lane < nb) {
            blk = b0 + c0 + lane;
            if (p.topk_idx) blk = p.list_blk[(long long)q * p.list_cap + blk];
            page = p.batch.block_table[(long long)q * p.batch.bt_stride + blk];
          }
          for (int i = 0; ok && i < min(32, nb - c0); ++i) {
            const int b = __shfl_sync(0xffffffffu, blk, i), pg = __shfl_sync(0xffffffffu, page, i);
            const bool bad_page = pg < 0 || pg >= p.batch.num_pages;
            const int ntok = min(kBlock, bi.seq - kBlock * b);
            const bool cached_all = !p.topk_idx || b >= rq.ctx / kBlock;
            bi.rows = cached_all ? nullptr
                                 : p.list_rows + ((long long)q * p.list_cap + b0 + c0 + i) * p.list_words;
            bi.t0 = kBlock * b;
            bi.flags = both | (c0 + i == 0 ? kFirst : 0) | (c0 + i == nb - 1 ? kLast : 0) |
                       (bad_page ? kBadPage | kNoData : 0) |
                       (bi.t0 + kBlock > rq.ctx || !cached_all ? kMixed : 0) |
                       (!bad_page && ntok > 64 ? kHalves : 0);
            if constexpr (FP8) {
              if (bad_page && lane == 0) atomicOr(p.status, MSA_DEV_BAD_PAGE);
              push(bi, bad_page ? -1 : pg);
              continue;
            }
            const int kb = acquire(), vb = acquire();
            if (!ok) break;
            uint8_t* kd = smem + kSmKv + kb * kTile;
            uint8_t* vd = smem + kSmKv + vb * kTile;
            if (bad_page) {
              if (lane == 0) {
                mbar_arrive(&kv_full[kb]);
                mbar_arrive(&kv_full[vb]);
                atomicOr(p.status, MSA_DEV_BAD_PAGE);
              }
            } else {
              // tokens past the request's end are not data: their V rows are
              // zeroed before the product reads them
              uint64_t* land = ntok < kBlock ? fill : &kv_full[vb];
              if (lane == 0) {
                mbar_arrive_expect_tx(&kv_full[kb], kTile);
                mbar_arrive_expect_tx(land, kTile);
                for (int h = 0; h < 2; ++h) {
                  tma_load_2d(kd + h * kHalf, &kmap, 64 * h, pg * kBlock, &kv_full[kb]);
                  tma_load_2d(vd + h * kHalf, &vmap, 64 * h, pg * kBlock, land);
                }
              }
              if (ntok < kBlock) {
                // (announced first: the other roles run meanwhile)
                announce(bi);
                ok = warp_wait(fill, fills & 1);
                ++fills;
                if (!ok) break;
                uint4* v4 = reinterpret_cast<uint4*>(vd);
                for (int k = ntok * 8 + lane; k < kBlock * 8; k += 32)
                  v4[k] = v4[kHalf / 16 + k] = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&kv_full[vb]);
                continue;
              }
            }
            announce(bi);
          }
        }
      }
      if (ok) {
        bi.flags = kEnd;
        announce(bi);
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
      // ---------------------------------------------- products of tile t
      // P V of a block's two halves as their softmax is done, and S of the next.
      // kAhead (bf16): S in two products of 64 tokens.  The first goes over the
      // second half's logits as soon as they are in registers, so that the softmax
      // goes on while P V runs; the second goes over P.  In one product, behind P V,
      // 8 requests of 48..64 rows x 16 heads took a fifth longer; e4m3, whose keys are
      // converted on the way and leave a ring of three tiles, a tenth less so.
      const int t = warp - 1;
      if (lane == 0) {
        const uint64_t qd = tc::desc_kmajor_sw128(smem_u32(smem + kSmQ + t * kTile));
        uint64_t *sf = s_full + 2 * t, *pf = p_full + 2 * t, *pv = pv_done + 2 * t;
        bool ok = mbar_wait(&info_full[0], 0);
        int seg = -1, n = 0, fl = ok ? info[0].flags : kEnd;
        const auto p_at = [](int blk) { return kAhead ? 64u * (blk & 1) : 0u; };
        const auto works = [&](int f) { return (t == 0 || (f & kTwo)) && !(f & kNoData); };
        // S of a half block (with !kAhead of the whole, as the first)
        const auto s_half = [&](int blk, int half) {
          const uint64_t kd = tc::desc_advance(
              tc::desc_kmajor_sw128(smem_u32(smem + kSmKv + ((2 * blk) % kBufs) * kTile)), half * 64 * 128);
          tc::fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
            tc::mma_ss(tmem + col_s(t) + (kAhead ? 64 * ((blk ^ half) & 1) : 0), tc::desc_advance(qd, off),
                       tc::desc_advance(kd, off), kIdescS, kk > 0 ? 1u : 0u);
          }
          tc::commit(&sf[half]);
        };
        const auto open = [&](int blk, int f) {
          bool there = true;
          if (f & kFirst) {
            ++seg;
            there = mbar_wait(q_full, seg & 1);
          }
          there = there && mbar_wait(&kv_full[(2 * blk) % kBufs], ((2 * blk) / kBufs) & 1);
          if (blk > 0)
            there = there && (kAhead ? mbar_wait(&s_read[t], (blk - 1) & 1) : mbar_wait(&pv[1], (blk - 1) & 1));
          if (!there) return false;
          if (works(f)) s_half(blk, 0);
          else mbar_arrive(&sf[0]);
          return true;
        };
        if (ok && !(fl & kEnd)) ok = open(0, fl);
        while (ok && !(fl & kEnd)) {
          const bool work = works(fl);
          const int kb = (2 * n) % kBufs, vb = (2 * n + 1) % kBufs;
          if (kAhead && n > 0) ok = mbar_wait(&pv[1], (n - 1) & 1);
          if (!ok) break;
          if (work) {
            if (kAhead) {
              if (fl & kHalves) s_half(n, 1);
              else tc::commit(&sf[1]);
            }
            tc::commit(&kv_empty[kb]);
            if (fl & kLast) tc::commit(q_empty);
          } else {
            if (kAhead) mbar_arrive(&sf[1]);
            mbar_arrive(&kv_empty[kb]);
            if (fl & kLast) mbar_arrive(q_empty);
          }
          const uint64_t vd = tc::desc_mnmajor_sw128(smem_u32(smem + kSmKv + vb * kTile), kHalf);
          bool hand = false;  // the softmax adds the block's P V itself
          const auto pv_half = [&](int half) {
            if (work && !hand && (half == 0 || (fl & kHalves))) {
              tc::fence_after();
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc::mma_ts(tmem + col_o(t), tmem + col_s(t) + p_at(n) + half * 32 + kk * 8,
                           tc::desc_advance(vd, (half * 4 + kk) * 2048), kIdescO,
                           (kk > 0 || half > 0 || !(fl & kFirst)) ? 1u : 0u);
            }
            if (work) tc::commit(&pv[half]);
            else mbar_arrive(&pv[half]);
          };
          ok = mbar_wait(&kv_full[vb], ((2 * n + 1) / kBufs) & 1);
          // O of the previous segment has been read
          if ((fl & kFirst) && seg > 0) ok = ok && mbar_wait(&o_free[t], (seg - 1) & 1);
          ok = ok && mbar_wait(&pf[0], n & 1);
          if (!ok) break;
          hand = (fl & kMixed) && *reinterpret_cast<volatile int*>(&misc[4 + n % kLooks]) == n + 1;
          pv_half(0);
          int next = kFirst;
          const auto follow = [&]() {
            const bool there = mbar_wait(&info_full[(n + 1) % kInfos], ((n + 1) / kInfos) & 1);
            if (there) next = info[(n + 1) % kInfos].flags;
            return there;
          };
          if (kAhead) ok = follow();
          const bool early = ok && !(next & (kEnd | kFirst));
          if (early) ok = open(n + 1, next);
          ok = ok && mbar_wait(&pf[1], n & 1);
          if (!ok) break;
          pv_half(1);
          if (work) tc::commit(&kv_empty[vb]);
          else mbar_arrive(&kv_empty[vb]);
          if (!kAhead) ok = follow();
          if (!ok) break;
          ++n;
          fl = next;
          if (!early && !(next & kEnd)) ok = open(n, next);
        }
        if (!ok) misc[0] = 1;
        // every product has completed before the tensor memory is freed
        tc::commit(&drained[t]);
        if (!mbar_wait(&drained[t], 0)) misc[0] = 1;
      }
    };
    const auto look = [&]() {
      // ---------------------------------------------- values that are not finite
      // in the V of blocks that not every row sees (e4m3: the converting warps look)
      bool ok = true;
      for (int n = 0;; ++n) {
        ok = warp_wait(&info_full[n % kInfos], (n / kInfos) & 1);
        if (!ok) break;
        const BlockInfo& bi = info[n % kInfos];
        const int fl = bi.flags;
        if (fl & kEnd) break;
        // (every use of a place is followed, so that the ring never laps this warp)
        const int kb = (2 * n) % kBufs, vb = (2 * n + 1) % kBufs;
        ok = warp_wait(&kv_full[kb], ((2 * n) / kBufs) & 1);
        if (!ok) break;
        if (lane == 0) mbar_arrive(&kv_empty[kb]);
        ok = warp_wait(&kv_full[vb], ((2 * n + 1) / kBufs) & 1);
        if (!ok) break;
        if ((fl & kMixed) && !(fl & kNoData)) {
          // (tokens past the request's end are zeros)
          const uint8_t* src = smem + kSmKv + vb * kTile + lane * 16;
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
    const auto convert = [&]() {
      // ---------------------------------------------- e4m3 tiles to f16, queries
      const int ct = tid - 12 * 32;
      int x = 0, rx = 0, seg = -1;  // 16-bit tiles, e4m3 tiles, segments
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
            const uint16_t* src = p.q + (long long)bi.row0 * H * kHeadDim;
            const int rows = bi.ntok * H, per = tpt * H;
#pragma unroll 8
            for (int i = ct; i < 2 * 128 * 16; i += kConv * 32) {
              const int t = i >> 11, m = (i >> 4) & 127, ch = i & 15, row = t * per + m;
              uint4 v = make_uint4(0u, 0u, 0u, 0u);
              if (m < per && row < rows)
                v = __ldg(reinterpret_cast<const uint4*>(src + (long long)row * kHeadDim) + ch);
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
          // the block's scales (a thread per token), k's with the softmax's own
          float ks = 0.f, vs = 0.f;
          const bool data = !(fl & kNoData) && bi.t0 + ct < bi.seq;
          if (data) {
            const long long at = (long long)bi.page * kBlock + ct;
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
            reinterpret_cast<float2*>(sc + kSoRange)[warp - 12] = make_float2(bits_log2(hi), bits_log2(lo));
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[n % kScales]);
        }
        for (int kv = 0; ok && kv < 2; ++kv, ++x) {
          const int b = x % kBufs;
          if (x >= kBufs) ok = warp_wait(&kv_empty[b], ((x / kBufs) - 1) & 1);
          if (!ok) break;
          const int rb = rx % kRaws;
          ok = warp_wait(&raw_full[rb], (rx / kRaws) & 1);
          if (!ok) break;
          ++rx;
          if (!(fl & kNoData)) {
            const uint8_t* raw = smem + C::kSmRaw + rb * kRaw;
            uint8_t* tile = smem + kSmKv + b * kTile;
            // tokens past the request's end are not data: zeros
            const int there = min(kBlock, bi.seq - bi.t0);
            // (two at a time: eight took 106.7 us where two took 102.5, the softmax's
            // instructions wait behind them)
#pragma unroll 2
            for (int i = ct; i < kRaw / 16; i += kConv * 32) {
              const int row = i >> 3, ch = 2 * (i & 7);  // 16 codes: f16 chunks ch, ch + 1
              uint4 v = lds128(raw + 16 * i);
              if (row >= there) v = make_uint4(0u, 0u, 0u, 0u);
              uint8_t* dst = tile + (ch >> 3) * kHalf + row * 128;
              *reinterpret_cast<uint4*>(dst + (((ch & 7) ^ (row & 7)) << 4)) =
                  make_uint4(e4m3x2_to_f16x2((uint16_t)v.x), e4m3x2_to_f16x2((uint16_t)(v.x >> 16)),
                             e4m3x2_to_f16x2((uint16_t)v.y), e4m3x2_to_f16x2((uint16_t)(v.y >> 16)));
              *reinterpret_cast<uint4*>(dst + ((((ch & 7) + 1) ^ (row & 7)) << 4)) =
                  make_uint4(e4m3x2_to_f16x2((uint16_t)v.z), e4m3x2_to_f16x2((uint16_t)(v.z >> 16)),
                             e4m3x2_to_f16x2((uint16_t)v.w), e4m3x2_to_f16x2((uint16_t)(v.w >> 16)));
            }
            fence_proxy_async_smem();
            if (kv == 1 && (fl & kMixed)) {
              // a code of NaN among the thread's: 0x7f without its sign
              uint32_t odd = 0;
#pragma unroll 2
              for (int i = ct; i < kRaw / 16; i += kConv * 32) {
                const uint4 v = lds128(raw + 16 * i);
                if ((i >> 3) < there)
                  odd |= ((v.x & 0x7f7f7f7fu) + 0x01010101u) | ((v.y & 0x7f7f7f7fu) + 0x01010101u) |
                         ((v.z & 0x7f7f7f7fu) + 0x01010101u) | ((v.w & 0x7f7f7f7fu) + 0x01010101u);
              }
              if (odd & 0x80808080u) *reinterpret_cast<volatile int*>(&misc[4 + n % kLooks]) = n + 1;
            }
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
      const uint32_t oa = tmem + lanes + col_o(t);
      const int mtok = m / H, head = m % H;
      float scale2 = p.softmax_scale * kTreeLog2e, vs = 1.f;
      if (p.scale_mode == MSA_SCALE_SCALAR) {
        scale2 *= __ldg(p.k_scale);
        vs = __ldg(p.v_scale);
      }
      const float sink = p.sinks ? __ldg(p.sinks + head) : 0.f;
      float m_run = -INFINITY, l_run = 0.f;
      constexpr float kHead = FP8 ? kHalfHead : 0.f;
      bool bad = false, ok = true;
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
          bad = false;
        }
        bad |= (fl & (kBadPage | kPoison)) != 0;
        const int tok = t * tpt + mtok;  // drafted token of the pair
        const bool there = (t == 0 || (fl & kTwo)) && mtok < tpt && tok < bi.ntok;
        const bool work = (t == 0 || (fl & kTwo)) && !(fl & kNoData);
        bool masked = (fl & kMixed) != 0;
        uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
        if (masked && work) {
          const int j = bi.j0 + tok;
          const bool sel = there && tree_row_selects(bi.rows, j);
          if (bi.t0 + kBlock <= bi.ctx) {  // cached tokens alone: all or none
            vis[0] = vis[1] = vis[2] = vis[3] = sel ? ~0u : 0u;
            masked = !__all_sync(0xffffffffu, sel || !there);
          } else {
#pragma unroll
            for (int w = 0; w < 4; ++w)
              vis[w] = !there ? 0u
                              : tree_vis16(p, bi.row0 + tok, j, bi.ctx, bi.qlen, bi.t0 + 32 * w, sel) |
                                    tree_vis16(p, bi.row0 + tok, j, bi.ctx, bi.qlen, bi.t0 + 32 * w + 16, sel) << 16;
          }
        }
        bool hand = false;
        float moved = 1.f;  // what the second half scaled the first one's P by
        const float* ks = nullptr;
        // (PTH, by half) log2 of the largest v scale; whether the scales lie too far apart for it
        float near0 = 0.f, near1 = 0.f;
        bool exact0 = false, exact1 = false;
        if (PTH && work) {
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
        if (!kAhead) ok = warp_wait(&s_full[2 * t], n & 1);
        if (!ok) break;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (kAhead) ok = warp_wait(&s_full[2 * t + half], n & 1);
          if (kAhead && !ok) break;
          if (work && (half == 0 || (fl & kHalves))) {
            tc::fence_after();
            const uint32_t sa = tmem + lanes + col_s(t) + 64 * ((kAhead ? n ^ half : half) & 1);
            const uint32_t v0 = half ? vis[2] : vis[0], v1 = half ? vis[3] : vis[1];
            const float* kh = PTH ? ks + 64 * half : nullptr;
            uint32_t r[64];
            tc::tmem_ld64(sa, r);
            if (kAhead && half) {
              tc::fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&s_read[t]);
            }
            // (with PTH the tokens' factors carry the softmax scale and its sign)
            const float sg = PTH ? 1.f : scale2;
            const bool exact = PTH && (half ? exact1 : exact0);
            const float near = half ? near1 : near0;
            float mx;
            if (exact)
              mx = row_max<false, true, PTH, true>(r, -INFINITY, v0, v1, kh, kh + kSoLog);
            else if (masked)
              mx = sg >= 0.f ? row_max<false, true, PTH>(r, -INFINITY, v0, v1, kh) * sg
                             : row_max<true, true, PTH>(r, -INFINITY, v0, v1, kh) * -sg;
            else
              mx = sg >= 0.f ? row_max<false, false, PTH>(r, -INFINITY, v0, v1, kh) * sg
                             : row_max<true, false, PTH>(r, -INFINITY, v0, v1, kh) * -sg;
            mx += exact ? -kHead : near - kHead;
            const bool move = mx > m_run + kSlack || (m_run == -INFINITY && mx > -INFINITY);
            if (__any_sync(0xffffffffu, move)) {
              float al = 1.f;
              if (mx > m_run) {
                al = m_run == -INFINITY ? 1.f : ex2_ftz(m_run - mx);
                m_run = mx;
              }
              l_run *= al;
              if (half) moved = al;
              // (a row without a reference has an all-zero O: nothing to rescale)
              if (!((fl & kFirst) && half == 0) && __any_sync(0xffffffffu, al != 1.f)) {
                ok = half ? warp_wait(&pv_done[2 * t], n & 1) : warp_wait(&pv_done[2 * t + 1], (n - 1) & 1);
                if (!ok) break;
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
            const uint32_t pa = tmem + lanes + col_s(t) + (kAhead ? 64 * (n & 1) : 0) + 32 * half;
            l_run += masked ? row_exp<true, FP8, PTH>(r, pa, scale2, base, v0, v1, kh, vh)
                            : row_exp<false, FP8, PTH>(r, pa, scale2, base, v0, v1, kh, vh);
            tc::tmem_wait_st();
            tc::fence_before();
          } else if (kAhead && half && lane == 0) {
            mbar_arrive(&s_read[t]);
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
            // (P V of the blocks before is complete: this block's S waited for it)
            tc::fence_after();
            pv_by_hand<FP8>(oa, tmem + lanes + col_s(t) + (kAhead ? 64 * (n & 1) : 0),
                            smem + kSmKv + vb * kTile, make_uint4(vis[0], vis[1], vis[2], vis[3]),
                            fl & kHalves ? 4 : 2, moved, (fl & kFirst) != 0);
            tc::tmem_wait_st();
            tc::fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * t + 1]);
        }
        if (!ok) break;
        if (fl & kLast) {
          ok = warp_wait(&pv_done[2 * t + 1], n & 1);
          if (!ok) break;
          tc::fence_after();
          const bool none = bad || (m_run == -INFINITY && l_run == 0.f);
          const TreeRowEnd e = tree_row_end(none ? -INFINITY : m_run, none ? 0.f : l_run,
                                            p.sinks != nullptr, sink * kTreeLog2e, vs);
          const bool have = (t == 0 || (fl & kTwo)) && !(fl & kPoison);
          const long long r = (long long)(bi.row0 + tok) * H + head;  // row x head in the batch
          const int pm = t * tpt * H + m;  // row of the pair
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
            if (fl & kWhole) p.lse[r] = none ? (p.sinks ? sink : -INFINITY) : e.lse;
            else p.part_ml[pr] = make_float2(m_run, l_run);
          }
          if (t == 0 && m == 0) {
            if (!(fl & kWhole)) p.part_bad[bi.slot] = bad ? 1 : 0;
            if (bi.bad) atomicOr(p.status, bi.bad);
          }
        }
      }
      if (!ok) misc[0] = 1;
    };
    if constexpr (FP8) {
      // (a warpgroup's warps give and take registers together; bf16 dispatched like this
      // measured 91 us where the plain order below measures 83)
      if (warp < 4) {
        regs_fewer<kRegsFew>();
        if (warp == 0) copies();
        else if (warp < 3) products();
      } else if (warp >= 12) {
        regs_fewer<kRegsFew>();
        convert();
      } else {
        regs_more<kRegsMore>();
        softmax();
      }
    } else if (warp == 0) {
      copies();
    } else if (warp < 3) {
      products();
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

template <bool FP8, bool PTH>
cudaError_t launch_tc(const TreeLaunch& p, int grid, cudaStream_t stream) {
  using C = TcCfg<FP8, PTH>;
  CUtensorMap qmap, kmap, vmap;
  memset(&qmap, 0, sizeof(qmap));
  memset(&kmap, 0, sizeof(kmap));
  memset(&vmap, 0, sizeof(vmap));
  const long long toks = max(1ll, (long long)p.batch.num_pages) * kBlock;
  if (!FP8 &&
      (!encode_map_2d(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.q, kHeadDim,
                      (long long)p.batch.num_rows * p.num_heads, kHeadDim * 2, 64, 128) ||
       !encode_map_2d(&kmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.k, kHeadDim, toks, kHeadDim * 2, 64,
                      kBlock) ||
       !encode_map_2d(&vmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.v, kHeadDim, toks, kHeadDim * 2, 64,
                      kBlock)))
    return cudaErrorInvalidValue;
  auto kern = tree_attn_tc_kernel<FP8, PTH>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e != cudaSuccess) return e;
  kern<<<grid, C::kThreads, C::kBytes, stream>>>(p, qmap, kmap, vmap);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_attn_tc(const TreeLaunch& p, int grid, cudaStream_t stream) {
  if (!p.kv_fp8) return launch_tc<false, false>(p, grid, stream);
  return p.scale_mode == MSA_SCALE_PER_TOKEN_HEAD ? launch_tc<true, true>(p, grid, stream)
                                                  : launch_tc<true, false>(p, grid, stream);
}

}  // namespace msa
