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
// issuing thread a tile, so they run in the order of issue: S of the next block goes
// out right behind P V of this one, over the same tensor memory, without a
// wait between them.
// Roles: warp 0 issues the copies; a thread of warps 1 and 2 each the products of a
// tile; warp 3 looks bf16 V over (below) and brings the scales per token of bf16 pools;
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
//
// P is rounded to bf16 (f16 with e4m3 pools), the operand of its product; the sum l
// takes it in fp32 before that.  What bounds it: 4 * 128 * H operations a visible pair of
// tokens on the tensor cores, and beside them an exponential a pair and head (32 a clock
// and SM), about half as long; a block of a tile pair measures 2900 clocks against the
// products' 2048, the rest being the hand-over between softmax and products, which two
// tiles a CTA do not hide wholly.  Measured (16 heads, bf16): 16384 rows 671 us, 1640
// TFLOP/s of the 1842 that a library product reaches; 8 x 2048 rows 130 us; a 512-row chunk
// behind 30000 tokens 93 us.  With a scale per token the factors' way from shared memory
// (128 bits a thread and four tokens, for each row) nearly doubles the softmax: 8192 rows 311
// us against 200.
#include "attn_tc.cuh"
#include "prompt_common.cuh"

namespace msa {
namespace {

constexpr int kInfos = 8;   // segments announced
constexpr int kPages = 8;   // blocks whose page numbers are held
constexpr int kLooks = 4;   // blocks to look over
constexpr int kConv = 4;    // converting warps (e4m3 pools)
// flags of a segment
constexpr int kWhole = 1, kTwo = 2, kPoison = 4, kEnd = 8;

// What a tile pair's start and end cost, in tokens (8 x 2048 rows: 157, 130, 137 us with
// 128, 384, 768; 16 ragged prompts 192, 152, 166)
constexpr int kPairCost = 384;
// Least tokens of a CTA's slice: two boundaries of blocks at least (256 and 1024 measured
// the same)
constexpr long long kMinSlice = 512;

// A segment: blocks [b0, b0 + nb) of a tile pair that the CTA's slice holds
struct Segment {
  int flags;
  int row0, ntok, pos0;  // the pair's rows: first in the batch, count, position of the first
  int seq, b0, nb;       // tokens of the request; blocks
  int slot, head;        // partial slot; KV head
  uint32_t bad;
};

template <bool FP8, bool PTH>
struct PaCfg {
  static constexpr int kThreads = FP8 ? 512 : 384;
  // ring of 16-bit K and V tiles, alternating (4 and 5 measured the same: 16384 rows, 8 x 2048)
  static constexpr int kBufs = 3;
  static constexpr int kRaws = FP8 ? 3 : 0;            // ring of e4m3 tiles
  static constexpr int kSmQ = kBufs * kTile;
  static constexpr int kSmRaw = kSmQ + 2 * kTile;
  static constexpr int kSmScale = kSmRaw + kRaws * kRaw;
  static constexpr int kSmInfo = kSmScale + (PTH ? kScales * kScaleWords * 4 : 0);
  static constexpr int kSmBars = kSmInfo + kInfos * (int)sizeof(Segment);
  // kv full / empty, raw full / empty, q full / empty / raw, infos, scales; per tile s_full,
  // p_full of two halves, pv_done, o_free, drained, turn; fill; to look over, looked; pages
  static constexpr int kNumBars = 2 * kBufs + 2 * kRaws + 3 + kInfos + kScales + 12 + 1 + 2 * kLooks + 2 + kPages;
  static constexpr int kSmMisc = kSmBars + kNumBars * 8;
  static constexpr int kBytes = kSmMisc + 192;
  static_assert(kBytes <= 227 * 1024, "shared memory");
  static_assert(sizeof(Segment) % 8 == 0 && kSmBars % 8 == 0, "alignment");
};

constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t col_s(int t) { return 128u * t; }
__device__ __forceinline__ uint32_t col_o(int t) { return 256u + 128u * t; }

// word g of lane j of four becomes word j of lane g
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4], int lane) {
  const bool b0 = lane & 1, b1 = lane & 2;
  const uint32_t x0 = __shfl_xor_sync(0xffffffffu, b0 ? w[0] : w[1], 1);
  const uint32_t x1 = __shfl_xor_sync(0xffffffffu, b0 ? w[2] : w[3], 1);
  w[0] = b0 ? x0 : w[0];
  w[1] = b0 ? w[1] : x0;
  w[2] = b0 ? x1 : w[2];
  w[3] = b0 ? w[3] : x1;
  const uint32_t y0 = __shfl_xor_sync(0xffffffffu, b1 ? w[0] : w[2], 2);
  const uint32_t y1 = __shfl_xor_sync(0xffffffffu, b1 ? w[1] : w[3], 2);
  w[0] = b1 ? y0 : w[0];
  w[2] = b1 ? w[2] : y0;
  w[1] = b1 ? y1 : w[1];
  w[3] = b1 ? w[3] : y1;
}

// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Steps of 16 tokens from t0 on that hold one which the rows up to position `last` see; one
// at least, which starts O in a segment's first block
__device__ __forceinline__ int steps_to(int last, int t0) { return min(8, max(1, (last - t0 + 16) >> 4)); }
// The tokens of the mixed block at t0 that some product reads and some row does not see:
// first | end << 8
__device__ __forceinline__ int looks_of(const Segment& sg, int t0) {
  return max(0, sg.pos0 + 1 - t0) | 16 * steps_to(sg.pos0 + sg.ntok - 1, t0) << 8;
}

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

// The pairs of one KV head of a request: `wide` rows each.  `whole`: the list counts pairs
struct Pairs {
  int tiles, wide, qlen, ctx;
  bool whole;
  // tokens before pair i (all of them for i = tiles)
  __device__ __forceinline__ long long before(int i) const {
    if (whole) return i;
    const long long n = (long long)i * (kPairCost + ctx) + (long long)wide * i * (i + 1) / 2;
    return i < tiles ? n : n - ((long long)tiles * wide - qlen);
  }
  __device__ __forceinline__ int seen(int i) const { return ctx + min((i + 1) * wide, qlen); }
  // the pair that holds token u of the list
  __device__ __forceinline__ int at(long long u) const {
    if (whole) return (int)u;
    const float a = 0.5f * (float)wide, b = (float)(kPairCost + ctx) + a, f = (float)u;
    int i = (int)(2.f * f / (b + sqrtf(b * b + 4.f * a * f)));
    i = max(0, min(i, tiles - 1));
    while (i > 0 && before(i) > u) --i;
    while (i < tiles - 1 && before(i + 1) <= u) ++i;
    return i;
  }
};
__device__ __forceinline__ Pairs pairs_of(const PromptReq& r, int wide, bool whole) {
  return {(int)(((unsigned)r.qlen + wide - 1) / wide), wide, r.qlen, r.ctx, whole};
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
        const Pairs a = pairs_of(r, wide, p.whole);
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
  s.ctas = (int)max(1ll, min((long long)gridDim.x, p.whole ? s.total : s.total / kMinSlice));
  if (p.whole && (int)blockIdx.x < s.total) {  // (the grid holds every pair)
    s.begin = blockIdx.x;
    s.end = s.begin + 1;
  } else if (!p.whole && (int)blockIdx.x < s.ctas) {
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
  uint64_t* q_raw = q_empty + 1;         // (e4m3) Q in bf16
  uint64_t* info_full = q_raw + 1;
  uint64_t* sc_full = info_full + kInfos;
  uint64_t* s_full = sc_full + kScales;  // [tile]
  uint64_t* p_full = s_full + 2;         // [tile][half]
  uint64_t* pv_done = p_full + 4;        // [tile]
  uint64_t* o_free = pv_done + 2;        // [tile]
  uint64_t* drained = o_free + 2;        // [tile]
  uint64_t* fill = drained + 2;
  uint64_t* to_look = fill + 1;          // [kLooks]
  uint64_t* looked = to_look + kLooks;   // [kLooks]
  uint64_t* turn = looked + kLooks;      // [tile]: its products may go out
  uint64_t* page_in = turn + 2;          // [kPages] (bf16 with a scale per token) the block's page is known
  Segment* info = reinterpret_cast<Segment*>(smem + C::kSmInfo);
  // [0] timeout; [4 + j % kLooks] block to look over (-1: none any more), then whether its V
  // holds odd values; [16 + n % kPages] page of block n; [24 + j % kLooks] tokens to look over; [32 + 4 (j % kLooks)] as [8], a word
  // a converting warp
  volatile int* misc = reinterpret_cast<volatile int*>(smem + C::kSmMisc);
  volatile int *look_at = misc + 4, *look_odd = misc + 8, *pages = misc + 16, *look_from = misc + 24, *odd_fp8 = misc + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kSmMisc) + 12;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = p.num_heads, Hk = p.num_kv_heads, G = H / Hk;
  const int tpt = 128 / G;  // tokens per tile

  // (a barrier a thread)
  const auto barriers = [&](uint64_t* first, int n, int count) {
    if (warp == 3 && lane < n) mbar_init(first + lane, count);
  };
  if (tid == 0) misc[0] = 0;
  barriers(kv_full, kBufs, FP8 ? kConv : 1);
  barriers(kv_empty, kBufs, 2);  // the issuers
  barriers(raw_full, kRaws, 1);
  barriers(raw_empty, kRaws, kConv);
  barriers(q_full, 1, FP8 ? kConv : 1);
  barriers(q_empty, 1, 2);
  barriers(q_raw, 1, 1);
  barriers(info_full, kInfos, 1);
  barriers(sc_full, kScales, FP8 ? kConv : 1);
  barriers(s_full, 2, 1);
  barriers(p_full, 4, 4);
  barriers(pv_done, 2, 1);
  barriers(o_free, 2, 4);
  barriers(drained, 2, 1);
  barriers(fill, 1, 1);
  barriers(to_look, kLooks, 1);
  barriers(looked, kLooks, FP8 ? kConv : 1);
  barriers(turn, 2, 1);
  barriers(page_in, kPages, 1);
  if (warp == 3) fence_barrier_init();
  if (tid < 3) {
    const CUtensorMap* maps[3] = {&qmap, &kmap, &vmap};
    asm volatile("prefetch.tensormap [%0];" ::"l"(maps[tid]) : "memory");
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
      int n = 0, n_seg = 0, looks = 0, x = 0, fills = 0;
      bool ok = true;
      PromptSplit rec;
      rec.nrows = 0;
      const uint32_t qbytes = 2u * 64u * (uint32_t)(G * tpt);  // of one box of Q
      Segment sg;
      auto announce = [&]() {
        if (lane == 0) {
          info[n_seg % kInfos] = sg;
          mbar_arrive(&info_full[n_seg % kInfos]);
        }
        ++n_seg;
      };
      // A block's K and V (without data, pg < 0, they still take their places, so that no
      // segment is announced far ahead of the other roles)
      auto push = [&](int kv, int pg, int t0, bool mixed) {
        const CUtensorMap* map = kv ? &vmap : &kmap;
        constexpr int ring = FP8 ? kRaws : kBufs;
        const int b = x % ring;
        if (x >= ring) ok = warp_wait(&(FP8 ? raw_empty : kv_empty)[b], ((x / ring) - 1) & 1);
        if (!ok) return;
        ++x;
        if (PTH && kv == 0 && lane == 0) {
          pages[n % kPages] = pg;
          if (!FP8) mbar_arrive(&page_in[n % kPages]);
        }
        n += kv;
        if constexpr (FP8) {
          if (lane == 0) {
            if (pg < 0) {
              mbar_arrive(&raw_full[b]);
            } else {
              mbar_arrive_expect_tx(&raw_full[b], kRaw);
              tma_load_2d(smem + C::kSmRaw + b * kRaw, map, sg.head * kHeadDim, pg * kBlock, &raw_full[b]);
            }
          }
          return;
        }
        const int there = min(kBlock, sg.seq - t0);
        uint8_t* dst = smem + b * kTile;
        // V behind the request's end is not data: zeroed in the step of 16 tokens that a
        // product still reads
        const bool part = kv == 1 && pg >= 0 && (there & 15) && there < kBlock;
        uint64_t* land = part ? fill : &kv_full[b];
        if (lane == 0) {
          if (pg < 0) {
            mbar_arrive(land);
          } else {
            mbar_arrive_expect_tx(land, kTile);
            for (int h = 0; h < 2; ++h)
              tma_load_2d(dst + h * kHalf, map, sg.head * kHeadDim + 64 * h, pg * kBlock, land);
          }
        }
        if (part) {
          ok = warp_wait(fill, fills & 1);
          ++fills;
          if (!ok) return;
          uint4* v4 = reinterpret_cast<uint4*>(dst);
          for (int k = there * 8 + lane; k < ((there + 15) & ~15) * 8; k += 32)
            v4[k] = v4[kHalf / 16 + k] = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&kv_full[b]);
        }
        // (asked for when the place's earlier uses are over, so that the wait for this one
        // cannot take one of them for it)
        if (kv == 1 && mixed) {
          if (lane == 0) {
            look_at[looks % kLooks] = n - 1;
            look_from[looks % kLooks] = looks_of(sg, t0);
            mbar_arrive(&to_look[looks % kLooks]);
          }
          ++looks;
        }
      };
      // The next segment's Q, once the products have read the last one's (e4m3: the converting
      // warps turn it into f16 in its place)
      const auto queries = [&]() {
        uint64_t* land = FP8 ? q_raw : q_full;
        if (!ok) return;
        if (n_seg > 1) ok = warp_wait(q_empty, (n_seg - 2) & 1);
        if (!ok || lane != 0) return;
        if (sg.flags & kPoison) {
          mbar_arrive(land);
          return;
        }
        const int tiles = sg.flags & kTwo ? 2 : 1;
        mbar_arrive_expect_tx(land, 2u * tiles * qbytes);
        for (int t = 0; t < tiles; ++t)
          for (int h = 0; h < 2; ++h)
            tma_load_3d(smem + kSmQ + t * kTile + h * kHalf, &qmap, 64 * h, sg.head * G, sg.row0 + t * tpt, land);
      };
      int q = sl.q, tile = 0;
      PromptReq rq;
      Pairs pr;
      const int32_t* table = nullptr;
      int page0 = 0;  // the request's first 32 pages, one a lane
      uint32_t bad = 0;
      const auto request = [&]() {  // request q: lengths, every page looked at
        rq = prompt_request(p.batch, q);
        pr = pairs_of(rq, 2 * tpt, p.whole);
        table = p.batch.block_table + (long long)q * p.batch.bt_stride;
        bad = rq.bad;
        bool odd = false;
        page0 = lane < rq.nb ? __ldg(table + lane) : 0;
#pragma unroll 8
        for (int b = lane; b < rq.nb; b += 32) {
          const int page = __ldg(table + b);
          odd |= page < 0 || page >= p.batch.num_pages;
        }
        if (!bad && __any_sync(0xffffffffu, odd)) bad = MSA_DEV_BAD_PAGE;
      };
      request();
      const long long one = pr.before(pr.tiles);  // of a KV head
      sg.head = Hk == 1 ? 0 : p.whole ? (int)(sl.begin - sl.pre) / pr.tiles : (int)((sl.begin - sl.pre) / one);
      long long start = sl.pre + sg.head * one;
      tile = pr.at(sl.begin - start);
      start += pr.before(tile);
      while (ok && start < sl.end) {
        const int seen = pr.seen(tile), nv = (seen + kBlock - 1) / kBlock;
        // blocks of the pair in the slice: block b is the CTA's whose slice holds
        // token kPairCost + 128 b of the pair
        const long long first = start + kPairCost, stop = p.whole ? start + 1 : first + seen;
        const auto block_at = [&](long long u) {
          return u <= first ? 0 : (int)min((long long)nv, (u - first + kBlock - 1) / kBlock);
        };
        sg.b0 = p.whole ? 0 : block_at(sl.begin);
        sg.nb = (stop <= sl.end ? nv : block_at(sl.end)) - sg.b0;
        if (sg.nb > 0) {
          const int j0 = tile * 2 * tpt;
          sg.ntok = min(2 * tpt, rq.qlen - j0);
          sg.row0 = rq.q0 + j0;
          sg.pos0 = rq.ctx + j0;
          sg.seq = rq.ctx + rq.qlen;
          sg.slot = 2 * blockIdx.x + (sg.b0 > 0 ? 0 : 1);
          sg.bad = bad;
          sg.flags = (sg.nb == nv ? kWhole : 0) | (sg.ntok > tpt ? kTwo : 0) | (bad ? kPoison : 0);
          if (sg.b0 > 0) {
            const auto owner = [&](long long u) { return ((u + 1) * sl.ctas - 1) / sl.total; };
            if (owner(first) == (long long)blockIdx.x - 1) {
              rec.nrows = sg.ntok * G;
              rec.row0 = sg.row0;
              rec.head = sg.head;
              rec.last = (int)owner(first + (long long)(nv - 1) * kBlock);
            }
          }
          if (bad) sg.nb = 1;
          announce();
          // (its first K before its Q, whose place is free later)
          int page = sg.b0 == 0 ? page0 : 0;
          for (int i = 0; ok && i < sg.nb; ++i) {
            if ((i & 31) == 0 && sg.b0 + i > 0)
              page = !bad && i + lane < sg.nb ? __ldg(table + sg.b0 + i + lane) : 0;
            const int t0 = kBlock * (sg.b0 + i);
            const int pg = bad ? -1 : __shfl_sync(0xffffffffu, page, i & 31);
            push(0, pg, t0, false);
            if (i == 0) queries();
            if (ok) push(1, pg, t0, !bad && t0 + kBlock - 1 > sg.pos0);
          }
        }
        start = stop;
        if (++tile == pr.tiles) {
          tile = 0;
          if (++sg.head == Hk) {
            sg.head = 0;
            if (start < sl.end) {  // (so that requests with rows follow)
              do {
                ++q;
                request();
              } while (rq.qlen == 0);
            }
          }
        }
      }
      if (lane == 0) {
        look_at[looks % kLooks] = -1;
        mbar_arrive(&to_look[looks % kLooks]);
      }
      if (ok) {
        sg.flags = kEnd;
        announce();
      } else {
        misc[0] = 1;
        // copies still in flight land before the CTA leaves
        const int ring = FP8 ? kRaws : kBufs;
        uint64_t* bars = FP8 ? raw_full : kv_full;
        for (int i = max(0, x - ring); i < x; ++i) mbar_wait(&bars[i % ring], (i / ring) & 1);
        if (n_seg > 0) mbar_wait(FP8 ? q_raw : q_full, (n_seg - 1) & 1);
      }
      if (lane == 0) p.split[blockIdx.x] = rec;
    };
    const auto odd_of = [&](int j) {  // odd values in the V of mixed block j
      if (!FP8) return look_odd[j % kLooks] != 0;
      const volatile int* o = odd_fp8 + 4 * (j % kLooks);
      return (o[0] | o[1] | o[2] | o[3]) != 0;
    };
    const auto products = [&](int t) {
      // ---------------------------------------------- products of tile t
      // Block by block: P V of the two halves as their softmax is done, then S of the
      // next block over the same columns, which this thread's order keeps apart.
      if (!elect_one()) return;
      const uint64_t qd = tc::desc_kmajor_sw128(smem_u32(smem + kSmQ + t * kTile));
      const uint64_t kd0 = tc::desc_kmajor_sw128(smem_u32(smem));
      const uint64_t vd0 = tc::desc_mnmajor_sw128(smem_u32(smem), kHalf);
      const uint32_t sc = tmem + col_s(t), oc = tmem + col_o(t);
      bool ok = true, on = false, any = false;  // the tile has rows; the segment has data
      // block n of all, i of nb of segment seg, at t0; mixed blocks so far
      int n = -1, seg = -1, i = -1, nb = 0, t0 = 0, mixes = 0, pos0 = 0, last = 0, last0 = 0;
      while (true) {
        const bool next_seg = i + 1 >= nb;
        if (n >= 0) {
          // ---- P V of the block
          const int x = 2 * n + 1, b = x % kBufs;
          const bool work = on && (t == 1 || i == 0 || last0 >= t0), mixed = on && t0 + kBlock - 1 > pos0;
          const uint64_t vd = tc::desc_advance(vd0, b * kTile);
          ok = mbar_wait(&kv_full[b], (x / kBufs) & 1);
          // O of the previous segment has been read
          if (i == 0 && seg > 0) ok = ok && mbar_wait(&o_free[t], (seg - 1) & 1);
          // (the softmax writes P of the second half first)
          ok = ok && mbar_wait(&p_full[2 * t + 1], n & 1);
          // (block by block tile 0 first, so that one tile's softmax runs beside the other's products)
          if (t == 1 || n > 0) ok = ok && mbar_wait(&turn[t], (n - 1 + t) & 1);
          if (!ok) break;
          // (the softmax adds the block's P V itself)
          const bool hand = mixed && odd_of(mixes);
          const int steps = mixed ? steps_to(last, t0) : 8;
          const auto pv = [&](int half, bool on_top) {
            if (!work || hand) return;
            tc::fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (4 * half + kk < steps)
                tc::mma_ts(oc, sc + 64 * half + kk * 8, tc::desc_advance(vd, (4 * half + kk) * 2048), kIdescO,
                           (kk > 0 || on_top) ? 1u : 0u);
          };
          pv(1, i > 0);
          ok = mbar_wait(&p_full[2 * t], n & 1);
          if (!ok) break;
          pv(0, i > 0 || steps > 4);
          if (next_seg) tc::commit(&pv_done[t]);
          tc::commit(&kv_empty[b]);
          mixes += any && t0 + kBlock - 1 > pos0;
          // (the other tile does not wait for the next segment's Q)
          if (next_seg) mbar_arrive(&turn[1 - t]);
        }
        // ---- S of the next block
        ++i;
        t0 += kBlock;
        if (next_seg) {
          ++seg;
          ok = mbar_wait(&info_full[seg % kInfos], (seg / kInfos) & 1);
          if (!ok) break;
          const Segment& sg = info[seg % kInfos];
          if (sg.flags & kEnd) break;
          nb = sg.nb;
          pos0 = sg.pos0;
          i = 0;
          t0 = kBlock * sg.b0;
          any = !(sg.flags & kPoison);
          on = any && (t == 0 || (sg.flags & kTwo));
          last0 = pos0 + min(tpt, sg.ntok) - 1;
          last = t ? pos0 + sg.ntok - 1 : last0;
          ok = mbar_wait(q_full, seg & 1);
        }
        ++n;
        const int x = 2 * n, b = x % kBufs;
        ok = ok && mbar_wait(&kv_full[b], (x / kBufs) & 1);
        if (!ok) break;
        if (on && (t == 1 || i == 0 || last0 >= t0)) {
          const uint64_t kd = tc::desc_advance(kd0, b * kTile);
          tc::fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
            tc::mma_ss(sc, tc::desc_advance(qd, off), tc::desc_advance(kd, off), kIdescS, kk > 0 ? 1u : 0u);
          }
        }
        tc::commit(&s_full[t]);
        tc::commit(&kv_empty[b]);
        if (i == nb - 1) tc::commit(q_empty);
        if (!next_seg) mbar_arrive(&turn[1 - t]);
      }
      if (!ok) misc[0] = 1;
      // every product has completed before the tensor memory is freed
      tc::commit(&drained[t]);
      if (!mbar_wait(&drained[t], 0)) misc[0] = 1;
    };
    // values that are not finite in the V of mixed block j, at place vb (bf16; e4m3: the
    // converting warps look).  The block's P V waits for the softmax, and that for this.
    const auto look_over = [&](int j, int vb, int range) {
      // a row of 64 dims a lane and step
      const int from = range & 255, rows = (range >> 8) - from;
      uint32_t odd = 0;
#pragma unroll 4
      for (int i = lane; i < 16 * rows; i += 32) {
        const int row = from + (i >> 4);
        const uint8_t* src = smem + vb * kTile + ((i >> 3) & 1) * kHalf + row * 128 + (i & 7) * 16;
        const uint4 v = lds128(src);
        constexpr uint32_t one = 0x00800080u;  // an exponent's last bit
        odd |= (v.x & 0x7fff7fffu) + one;
        odd |= (v.y & 0x7fff7fffu) + one;
        odd |= (v.z & 0x7fff7fffu) + one;
        odd |= (v.w & 0x7fff7fffu) + one;
      }
      const bool any = __any_sync(0xffffffffu, (odd & 0x80008000u) != 0);
      if (lane == 0) {
        look_odd[j % kLooks] = any;
        mbar_arrive(&looked[j % kLooks]);
      }
    };
    // the j-th mixed block, once it is asked for; false without one, or when a wait ran out
    const auto look_next = [&](int j) {
      if (!warp_wait(&to_look[j % kLooks], (j / kLooks) & 1)) {
        misc[0] = 1;
        return false;
      }
      const int n = look_at[j % kLooks];
      if (n < 0) return false;
      if (!warp_wait(&kv_full[(2 * n + 1) % kBufs], ((2 * n + 1) / kBufs) & 1)) {
        misc[0] = 1;
        return false;
      }
      look_over(j, (2 * n + 1) % kBufs, look_from[j % kLooks]);
      return true;
    };
    const auto look = [&]() {
      // ---------------------------------------------- mixed blocks, as they are asked for
      for (int j = 0; look_next(j);) ++j;
    };
    // The scales of token ct of block n: asked for, then put in place (a warp's 32 at a time), k's
    // with the softmax's own
    const auto scales_of = [&](int head, bool data, int n, int ct) {
      float2 x = make_float2(0.f, 0.f);
      if (data) {
        const long long at = ((long long)pages[n % kPages] * kBlock + ct) * Hk + head;
        x = make_float2(__ldg(p.k_scale + at), __ldg(p.v_scale + at));
      }
      return x;
    };
    const auto scales_in = [&](float2 x, bool data, int n, int ct) {
      float* sc = reinterpret_cast<float*>(smem + C::kSmScale) + (n % kScales) * kScaleWords;
      sc[ct] = x.x * (p.softmax_scale * kTreeLog2e);
      sc[kSoV + ct] = x.y;
      sc[kSoLog + ct] = log2_scale(x.y);
      const uint32_t mag = scale_bits(x.y);
      const uint32_t hi = __reduce_max_sync(0xffffffffu, data ? mag : 0u);
      const uint32_t lo = __reduce_min_sync(0xffffffffu, data ? mag : ~0u);
      if (lane == 0)
        reinterpret_cast<float2*>(sc + kSoRange)[ct >> 5] = make_float2(bits_log2(hi), bits_log2(lo));
    };
    const auto scales = [&]() {
      // ---------------------------------------------- bf16 pools with a scale per token
      // The scales of every block, and mixed blocks looked over
      bool ok = true;
      int n = 0, looks = 0;
      for (int seg = 0;; ++seg) {
        ok = warp_wait(&info_full[seg % kInfos], (seg / kInfos) & 1);
        if (!ok) break;
        const Segment& sg = info[seg % kInfos];
        const int fl = sg.flags, nb = sg.nb, head = sg.head, seq = sg.seq, pos0 = sg.pos0;
        if (fl & kEnd) break;
        int t0 = sg.b0 * kBlock;
        for (int i = 0; i < nb; ++i, ++n, t0 += kBlock) {
          // (the block's K has a place, that of V of block n - 2: its page is known, and the
          // softmax is through with that block, so with block n - 4 of this place too)
          ok = warp_wait(&page_in[n % kPages], (n / kPages) & 1);
          if (!ok) break;
          float2 x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = scales_of(head, !(fl & kPoison) && t0 + 32 * k + lane < seq, n, 32 * k + lane);
#pragma unroll
          for (int k = 0; k < 4; ++k) scales_in(x[k], !(fl & kPoison) && t0 + 32 * k + lane < seq, n, 32 * k + lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[n % kScales]);
          if (!(fl & kPoison) && t0 + kBlock - 1 > pos0) {
            ok = look_next(looks++);
            if (!ok) break;
          }
        }
        if (!ok) break;
      }
      if (!ok) misc[0] = 1;
    };
    const auto convert = [&]() {
      // ---------------------------------------------- e4m3 tiles to f16, queries
      const int ct = tid - 12 * 32;
      int x = 0, looks = 0;  // tiles, mixed blocks
      bool ok = true;
      for (int seg = 0;; ++seg) {
        ok = warp_wait(&info_full[seg % kInfos], (seg / kInfos) & 1);
        if (!ok) break;
        const Segment& sg = info[seg % kInfos];
        const int fl = sg.flags, nb = sg.nb, head = sg.head, seq = sg.seq, b0 = sg.b0, pos0 = sg.pos0;
        if (fl & kEnd) break;
        ok = warp_wait(q_raw, seg & 1);
        if (!ok) break;
        if (!(fl & kPoison)) {
          // (in place, whatever lies in rows without a query)
          uint4* at = reinterpret_cast<uint4*>(smem + kSmQ) + ct;
#pragma unroll 8
          for (int i = 0; i < (fl & kTwo ? 2 : 1) * kTile / 16; i += kConv * 32) {
            uint4 v = at[i];
            v.x = pack_f16x2(bf16lo(v.x), bf16hi(v.x));
            v.y = pack_f16x2(bf16lo(v.y), bf16hi(v.y));
            v.z = pack_f16x2(bf16lo(v.z), bf16hi(v.z));
            v.w = pack_f16x2(bf16lo(v.w), bf16hi(v.w));
            at[i] = v;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        for (int i = 0; ok && i < nb; ++i) {
          const int t0 = (b0 + i) * kBlock;
          const bool mixed = !(fl & kPoison) && t0 + kBlock - 1 > pos0;
          for (int kv = 0; ok && kv < 2; ++kv, ++x) {
            constexpr int kRing = FP8 ? kRaws : 1;
            const int b = x % kBufs, rb = x % kRing;
            ok = warp_wait(&raw_full[rb], (x / kRing) & 1);
            if (!ok) break;
            // (the block's scales are asked for before its K is converted and put in place after: K
            // goes over V of block n - 2, so the softmax is through with block n - 4's)
            const bool data = !(fl & kPoison) && t0 + ct < seq;
            float2 scale = make_float2(0.f, 0.f);
            if (PTH && kv == 0) scale = scales_of(head, data, x >> 1, ct);
            if (x >= kBufs) ok = warp_wait(&kv_empty[b], ((x / kBufs) - 1) & 1);
            if (!ok) break;
            if (!(fl & kPoison)) {
              // Rows of 128 bytes, 16-byte chunks swizzled by the copy; a thread takes chunk ct % 8 of
              // every 16th row, which becomes two chunks of a half tile's row
              const int row0 = ct >> 3, c = ct & 7, sw = row0 & 7;
              const uint8_t* from = smem + C::kSmRaw + rb * kRaw + row0 * 128 + ((c ^ sw) << 4);
              uint8_t* to = smem + b * kTile + (c >> 2) * kHalf + row0 * 128;
              const int even = (((2 * c) & 7) ^ sw) << 4, odd_at = (((2 * c + 1) & 7) ^ sw) << 4;
              const int there = seq - t0;  // behind it: not data, zeros
              // rows to look over
              const int first = kv == 1 && mixed ? looks_of(sg, t0) & 255 : kBlock;
              const bool edge = there < kBlock || first < kBlock;
              uint32_t odd = 0;
#pragma unroll 4
              for (int k = 0; k < 8; ++k) {
                uint4 v = lds128(from + 2048 * k);
                if (edge) {
                  const int row = row0 + 16 * k;
                  if (row >= there) v = make_uint4(0u, 0u, 0u, 0u);
                  if (row >= first)  // (a code of NaN: 0x7f without its sign)
                    odd |= ((v.x & 0x7f7f7f7fu) + 0x01010101u) | ((v.y & 0x7f7f7f7fu) + 0x01010101u) |
                           ((v.z & 0x7f7f7f7fu) + 0x01010101u) | ((v.w & 0x7f7f7f7fu) + 0x01010101u);
                }
                *reinterpret_cast<uint4*>(to + even + 2048 * k) =
                    make_uint4(e4m3x2_to_f16x2((uint16_t)v.x), e4m3x2_to_f16x2((uint16_t)(v.x >> 16)),
                               e4m3x2_to_f16x2((uint16_t)v.y), e4m3x2_to_f16x2((uint16_t)(v.y >> 16)));
                *reinterpret_cast<uint4*>(to + odd_at + 2048 * k) =
                    make_uint4(e4m3x2_to_f16x2((uint16_t)v.z), e4m3x2_to_f16x2((uint16_t)(v.z >> 16)),
                               e4m3x2_to_f16x2((uint16_t)v.w), e4m3x2_to_f16x2((uint16_t)(v.w >> 16)));
              }
              fence_proxy_async_smem();
              if (kv == 1 && mixed) {
                // (a word a warp: the place's last readers are behind this block's K)
                const bool any = __any_sync(0xffffffffu, (odd & 0x80808080u) != 0);
                if (lane == 0) odd_fp8[4 * (looks % kLooks) + warp - 12] = any;
              }
              __syncwarp();
            }
            if (PTH && kv == 0) {
              scales_in(scale, data, x >> 1, ct);
              __syncwarp();
              if (lane == 0) mbar_arrive(&sc_full[(x >> 1) % kScales]);
            }
            if (lane == 0) {
              if (kv == 1 && mixed) mbar_arrive(&looked[looks % kLooks]);
              mbar_arrive(&raw_empty[rb]);
              mbar_arrive(&kv_full[b]);
            }
          }
          looks += mixed;
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
      constexpr float kHead = FP8 ? kHalfHead : 0.f;
      // a factor that is not positive: the logits take its sign (or 0)
      const bool turned = !PTH && !(scale2 > 0.f);
      const float flip = scale2 < 0.f ? -1.f : scale2 == 0.f ? 0.f : scale2;
      if (turned) scale2 = scale2 < 0.f ? -scale2 : 1.f;
      // one bit for each of 32 tokens of which the first c are seen
      const auto bits = [](int c) { return c >= 32 ? ~0u : c > 0 ? (1u << c) - 1u : 0u; };
      bool ok = true;
      int n = 0, looks = 0;  // blocks, mixed ones
      for (int seg = 0;; ++seg) {
        ok = warp_wait(&info_full[seg % kInfos], (seg / kInfos) & 1);
        if (!ok) break;
        const Segment& sg = info[seg % kInfos];
        const int fl = sg.flags, nb = sg.nb, pos0 = sg.pos0, ntok = sg.ntok;
        if (fl & kEnd) break;
        const bool there = mtok < tpt && tok < ntok;
        const bool on = !(fl & kPoison) && (t == 0 || (fl & kTwo));
        const int last0 = pos0 + min(tpt, ntok) - 1;
        float m_run = -INFINITY, l_run = 0.f;
        int t0 = kBlock * sg.b0;
#pragma unroll 1
        for (int i = 0; i < nb; ++i, ++n, t0 += kBlock) {
          const bool work = on && (t == 1 || i == 0 || last0 >= t0);
          const bool mixed = !(fl & kPoison) && t0 + kBlock - 1 > pos0;
          const int seen = mixed ? (there ? pos0 + tok + 1 - t0 : 0) : kBlock;  // of the block's tokens
          const float* ks = nullptr;
          if (PTH) {
            ok = warp_wait(&sc_full[n % kScales], (n / kScales) & 1);
            if (!ok) break;
            ks = reinterpret_cast<const float*>(smem + C::kSmScale) + (n % kScales) * kScaleWords;
          }
          ok = warp_wait(&s_full[t], n & 1);
          if (!ok) break;
          tc::fence_after();
          if (work) {
            // Logits that the row does not see become -inf in place, and a factor that is not
            // positive goes into them, so that what follows is the same code for every block (a
            // scale per token, which may be anything where the row does not look, is masked there).
            if (__builtin_expect((mixed && !PTH) || turned, 0)) {
              const int least = __reduce_min_sync(0xffffffffu, there ? seen : kBlock);
              const int most = __reduce_max_sync(0xffffffffu, there ? seen : 0);
#pragma unroll 1
              for (int c = turned ? 0 : max(0, least) & ~15; c < 128; c += 16) {
                uint32_t x[16];
                if (c < most) {
                  tc::tmem_ld16(sa + c, x);
#pragma unroll
                  for (int k = 0; k < 16; ++k)
                    x[k] = c + k >= seen ? 0xff800000u : turned ? __float_as_uint(__uint_as_float(x[k]) * flip) : x[k];
                } else {
#pragma unroll
                  for (int k = 0; k < 16; ++k) x[k] = 0xff800000u;
                }
                tc::tmem_st16(sa + c, x);
              }
              tc::tmem_wait_st();
            }
            uint32_t r[64];
            float mx = -INFINITY;
            if constexpr (PTH) {
              // Logits times their tokens' factors (which carry the softmax scale), -inf where the row
              // does not look, whatever the factor is; the first half's go back into their place
#pragma unroll 1
              for (int h = 0; h < 2; ++h) {
                tc::tmem_ld64(sa + 64 * h, r);
#pragma unroll
                for (int k = 0; k < 64; k += 4) {
                  const float4 f = *reinterpret_cast<const float4*>(ks + 64 * h + k);
                  float* x = reinterpret_cast<float*>(r + k);
                  mul2v(x[0], x[1], f.x, f.y);
                  mul2v(x[2], x[3], f.z, f.w);
                }
                if (__builtin_expect(mixed, 0)) {
#pragma unroll
                  for (int k = 0; k < 64; ++k)
                    if (64 * h + k >= seen) r[k] = 0xff800000u;
                }
                if (h == 0) tc::tmem_st64(sa, r);
                // log2 of the largest v scale stands for every token's where they lie near
                const float4 g = *reinterpret_cast<const float4*>(ks + kSoRange + 4 * h);
                const float near = fmaxf(g.x, g.z);
                if (__builtin_expect(near - fminf(g.y, g.w) > kNear, 0)) {
                  float m2[2] = {mx, mx};
#pragma unroll
                  for (int k = 0; k < 64; k += 4) {
                    const float4 l = *reinterpret_cast<const float4*>(ks + kSoLog + 64 * h + k);
                    m2[0] = fmax3(m2[0], __uint_as_float(r[k]) + l.x, __uint_as_float(r[k + 1]) + l.y);
                    m2[1] = fmax3(m2[1], __uint_as_float(r[k + 2]) + l.z, __uint_as_float(r[k + 3]) + l.w);
                  }
                  mx = fmaxf(m2[0], m2[1]);
                } else {
                  mx = fmaxf(mx, row_max<false, false, false>(r, -INFINITY, 0, 0, nullptr) + near);
                }
              }
              tc::tmem_wait_st();
            } else {
              tc::tmem_ld64(sa, r);
              mx = row_max<false, false, false>(r, mx, 0, 0, nullptr);
              tc::tmem_ld64(sa + 64, r);
              mx = row_max<false, false, false>(r, mx, 0, 0, nullptr);
            }
            mx = PTH ? mx - kHead : mx * scale2 - kHead;
            const bool move = there && (mx > m_run + kSlack || (m_run == -INFINITY && mx > -INFINITY));
            if (__any_sync(0xffffffffu, move)) {
              float al = 1.f;
              if (there && mx > m_run) {
                al = m_run == -INFINITY ? 1.f : ex2_ftz(m_run - mx);
                m_run = mx;
              }
              l_run *= al;
              // (a row without a reference has an all-zero O: nothing to rescale.  P V of
              // the block before is complete: this block's S came behind it)
              if (i > 0 && __any_sync(0xffffffffu, al != 1.f)) {
#pragma unroll 1
                for (int c = 0; c < 128; c += 16) {
                  uint32_t x[16];
                  tc::tmem_ld16(oa + c, x);
#pragma unroll
                  for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * al);
                  tc::tmem_st16(oa + c, x);
                }
              }
            }
            const float base = m_run == -INFINITY ? 0.f : m_run;
            bool hand = false;
            if (__builtin_expect(mixed, 0)) {
              ok = warp_wait(&looked[looks % kLooks], (looks / kLooks) & 1);
              if (!ok) break;
              hand = odd_of(looks);
            }
            // P of each half over its own logits, the second first: its logits are at hand, and
            // the first's are read again (128 at once took a fifth longer with what else lives in
            // 168 registers)
            const auto weights = [&](int h) {
              const float* vh = PTH ? ks + kSoV + 64 * h : nullptr;
              l_run += row_exp<false, FP8, PTH, PTH>(r, sa + 64 * h, scale2, base, 0, 0, nullptr, vh);
              tc::tmem_wait_st();
              if (PTH && __builtin_expect(mixed, 0)) {  // (0 times a hidden token's scale, which may be anything)
#pragma unroll 1
                for (int c = 0; c < 32; c += 16) {
                  uint32_t x[16];
                  tc::tmem_ld16(sa + 64 * h + c, x);
#pragma unroll
                  for (int k = 0; k < 16; ++k) {
                    const int left = seen - 64 * h - 2 * (c + k);
                    x[k] &= left > 1 ? ~0u : left == 1 ? 0xffffu : 0u;
                  }
                  tc::tmem_st16(sa + 64 * h + c, x);
                }
                tc::tmem_wait_st();
              }
            };
            const auto announce = [&](int h) {
              tc::fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&p_full[2 * t + h]);
            };
            weights(1);
            announce(1);
            tc::tmem_ld64(sa, r);
            weights(0);
            if (__builtin_expect(hand, 0)) {
              pv_by_hand<FP8, 64>(oa, sa, smem + ((2 * n + 1) % kBufs) * kTile,
                              make_uint4(bits(seen), bits(seen - 32), bits(seen - 64), bits(seen - 96)), 4, 1.f, i == 0);
              tc::tmem_wait_st();
            }
            announce(0);
          } else {
            if (mixed) {
              ok = warp_wait(&looked[looks % kLooks], (looks / kLooks) & 1);
              if (!ok) break;
            }
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&p_full[2 * t]);
              mbar_arrive(&p_full[2 * t + 1]);
            }
          }
          looks += mixed;
        }
        if (!ok) break;
        // ---- the segment's end: O out of tensor memory, to the rows or to a partial
        ok = warp_wait(&pv_done[t], seg & 1);
        if (!ok) break;
        tc::fence_after();
        const int hh = sg.head * G + (m - mtok * G);
        const float sink = p.sinks && there ? __ldg(p.sinks + hh) : 0.f;
        const bool none = (fl & kPoison) || (m_run == -INFINITY && l_run == 0.f);
        const TreeRowEnd e = tree_row_end(none ? -INFINITY : m_run, none ? 0.f : l_run, p.sinks != nullptr,
                                          sink * kTreeLog2e, vs);
        const long long r = ((long long)sg.row0 + tok) * H + hh;  // row x head in the batch
        const int pm = t * tpt * G + m;                           // row of the pair
        if (on && (fl & kWhole)) {
          // A lane holds two columns of a row in every eight; the four lanes of a row trade theirs
          // for eight columns each, so that a store's lines are eight rows' and not 32.
          const int rel = there ? tok * H + hh : -1;  // place behind the pair's first row
          uint16_t* const out = p.out + (long long)sg.row0 * H * kHeadDim + 8 * (lane & 3);
#pragma unroll 1
          for (int g = 0; g < 4; ++g) {
            const int upper = g >> 1, c = 64 * (g & 1);  // rows 16 * upper .. + 15, columns c .. + 63
            uint32_t v[32];
            tc::tmem_ld16x256(oa + ((uint32_t)(16 * upper) << 16) + c, v);
            if (g == 3) {
              tc::fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&o_free[t]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int row = 16 * upper + 8 * k + (lane >> 2);
              const float f = __shfl_sync(0xffffffffu, none ? 0.f : e.f, row);
              const int at = __shfl_sync(0xffffffffu, rel, row);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int y = 16 * x + 4 * i + 2 * k;
                  w[i] = f == 0.f ? 0u : pack_bf16x2(__uint_as_float(v[y]) * f, __uint_as_float(v[y + 1]) * f);
                }
                quad_transpose(w, lane);
                if (at >= 0)
                  *reinterpret_cast<uint4*>(out + (long long)at * kHeadDim + c + 32 * x) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
        } else {
          if (on) {
            // [4-dim group][row][4 dims]: the warp's rows are contiguous
            uint4* dst = reinterpret_cast<uint4*>(p.part_o) + (long long)sg.slot * 32 * 256 + pm;
#pragma unroll 1
            for (int c = 0; c < 128; c += 64) {
              uint32_t v[64];
              tc::tmem_ld64(oa + c, v);
              if (there) {
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  dst[256 * (c / 4 + k)] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
              }
            }
          } else if (there) {  // a poisoned request's rows
            uint4* dst = reinterpret_cast<uint4*>(p.out + r * kHeadDim);
            for (int k = 0; k < kHeadDim / 8; ++k) dst[k] = make_uint4(0u, 0u, 0u, 0u);
          }
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_free[t]);
        }
        if (there) {
          if (fl & (kWhole | kPoison)) p.lse[r] = none ? (p.sinks ? sink : -INFINITY) : e.lse;
          else p.part_ml[(long long)sg.slot * 256 + pm] = make_float2(m_run, l_run);
        }
        if (t == 0 && m == 0) {
          if (!(fl & kWhole)) p.part_bad[sg.slot] = fl & kPoison ? 1 : 0;
          if (sg.bad) atomicOr(p.status, sg.bad);
        }
      }
      if (!ok) misc[0] = 1;
    };
    if (warp == 0) copies();
    else if (warp < 3) products(warp - 1);
    else if (warp == 3) {
      if (!FP8) PTH ? scales() : look();
    } else if (warp < 12) {
      softmax();
    } else {
      convert();
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
  const long long toks = max(1ll, (long long)p.batch.num_pages) * kBlock;
  const long long inner = (long long)p.num_kv_heads * kHeadDim;
  const auto type = FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int size = FP8 ? 1 : 2, box = 128 / size;  // 128 bytes
  if (!encode_map_2d(&kmap, type, p.k, inner, toks, inner * size, box, kBlock) ||
      !encode_map_2d(&vmap, type, p.v, inner, toks, inner * size, box, kBlock) ||
      !encode_map_3d(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.q, kHeadDim, p.num_heads,
                              p.batch.num_rows, kHeadDim * 2, (long long)p.num_heads * kHeadDim * 2, 64, G, tpt))
    return cudaErrorInvalidValue;
  const int grid = device_sm_count();
  auto kern = prompt_attn_kernel<FP8, PTH>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e != cudaSuccess) return e;
  kern<<<grid, C::kThreads, C::kBytes, stream>>>(p, qmap, kmap, vmap);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.whole) return e;
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

// What the join takes (its launch, the partials' way through L2), in blocks of a pair
static constexpr int kJoinBlocks = 8;

cudaError_t launch_prompt_attn(const PromptLaunch& given, cudaStream_t stream) {
  PromptLaunch p = given;
  const int wide = 2 * (128 / (p.num_heads / p.num_kv_heads));
  const long long pairs = ((long long)p.batch.num_rows / wide + min(p.batch.num_rows, p.batch.num_reqs)) * p.num_kv_heads;
  // A pair to a CTA, with nothing to join, where the deepest pair takes less than a CTA's share of
  // an even split and the join behind that (one prompt, 16 heads, in a table no wider than it needs:
  // 200 rows 11.5 us, split 15.1; 1000 rows 20.2, 23.4; 2048 rows 31.3, 39.4; 2400 rows 36.0, 42.8;
  // behind cached tokens the split wins: 64 rows after 1900 tokens 19.1 against 31.6, 512 rows
  // after 1500 26.1 against 32.4).  The lengths are on the device, so the table's width stands
  // for the depth, half of it for the mean, as in a prompt from its start: 22 blocks at most, so
  // that one deep request among short ones does not hold a CTA for long.  In a table that is wider
  // than its requests (22, 256 and 8192 blocks measured the same) short prompts are split, too.
  const long long deepest = p.batch.bt_stride, sms = device_sm_count();
  p.whole = pairs <= sms && deepest <= kJoinBlocks + pairs * (deepest / 2 + kPairCost / kBlock) / sms;
  const bool pth = p.scale_mode == MSA_SCALE_PER_TOKEN_HEAD;
  if (p.kv_fp8) return pth ? launch<true, true>(p, stream) : launch<true, false>(p, stream);
  return pth ? launch<false, true>(p, stream) : launch<false, false>(p, stream);
}

}  // namespace msa
