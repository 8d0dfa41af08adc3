// attn_mass.cu -- the attention weight that a step's rows gave each cached
// token, added up over rows and heads into a paged array.
//
// Mathematics.  w_t = sum over (row, head) that see t of 2^(s - lse), both in
// log2 units, with the row's lse known from the attention: one product Q K^T
// and a sum over the rows, no second pass.  A token belongs to one CTA, which
// adds its rows in a fixed order: no atomics, the same bits every time.
//
// The product is taken as S^T = K Q^T on the 5th-generation tensor cores
// (tcgen05.mma M128, N = up to 128 rows, K128): the block's 128 tokens are the
// lanes of tensor memory, so each thread adds up its own token's columns and
// nothing crosses threads.  Per element one packed multiply-add, one 2^x, one
// packed add.  With few rows the stream of K bounds it (64 requests of one row x 16
// heads, 134 MB, in 32 us: 4.2 TB/s), with many the issue of the sums, two warps to
// a scheduler (8 windows of 32 rows x 16 heads over 8191..65000 e4m3 tokens in 43.6 us,
// 690 TFLOP/s, where 118 M exponentials alone would take 25; 16 columns at a time 47).
// A quarter of the 2^x as a polynomial cost a tenth more.
//
// Blocks go in groups of two, one per epilogue warpgroup, so that one's sums
// overlap the other's products, and each has two buffers of 128 columns, so that
// its own next product runs meanwhile.  A request of at most two chunks of rows
// keeps its queries in shared memory for all its blocks; more chunks stream
// through two buffers, each used by the group's two blocks.  e4m3 keys are
// converted to f16 (exact) by the four loader warps.
#include <string.h>

#include "tcgen05.cuh"
#include "tree_common.cuh"

namespace msa {
namespace {

constexpr int kThreads = 512;
constexpr int kHalf = 128 * 128;
constexpr int kTile = 2 * kHalf;   // 128 keys x 128 dims, 16 bits
constexpr int kRaw = 128 * 128;    // 128 keys of e4m3
constexpr int kInfos = 16;
constexpr int kLoaders = 4;        // warps 12 .. 15
// Blocks that a request's start and end count as when the work is split: its queries
// come in, its last blocks are masked by row (windows 47.6 us with 0, 45.3 with 2, 43.6
// with 4, 43.4 with 6; decode 32.7, 31.4, 32.1, 31.9)
constexpr int kStart = 4;
constexpr int kPiece = 128;        // rows x heads of a product; four of them in tensor memory

struct MassInfo {
  int flags;
  int nblk;      // blocks of the CTA's segment (on its first block)
  int q0, ctx, qlen;
  int t0;        // position of the block's first token
  int page;
  int pad;
  const uint32_t* rows;  // selection bits, or NULL
};
constexpr int kFirst = 1, kEnd = 2, kMixed = 4;

template <bool FP8, int QR>
struct MassCfg {
  static constexpr int kTiles = FP8 ? (QR == 256 ? 2 : 3) : (QR == 256 ? 3 : 6);
  static constexpr int kRaws = FP8 ? (QR == 256 ? 2 : 6) : 0;
  static constexpr int kCols = QR == 256 ? 64 : 16;  // columns summed at a time
  static constexpr int kQBuf = QR * 256;
  static constexpr int kSmK = 0;
  static constexpr int kSmQ = kTiles * kTile;
  static constexpr int kSmRaw = kSmQ + 2 * kQBuf;
  static constexpr int kSmNl = kSmRaw + kRaws * kRaw;     // [2][QR] -lse (log2 units)
  static constexpr int kSmInfo = kSmNl + 2 * QR * 4;
  static constexpr int kSmBars = kSmInfo + kInfos * (int)sizeof(MassInfo);
  // k full / empty, raw full / empty, q full / empty [2], d full / empty [2][2], drained, info full
  static constexpr int kNumBars = 2 * kTiles + 2 * kRaws + 13 + kInfos;
  static constexpr int kSmMisc = kSmBars + kNumBars * 8;
  static constexpr int kBytes = kSmMisc + 32;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
}

// Estimated cost of a block against `rows` rows x heads: the stream of its keys, or
// its products and exponentials (half and twice the 20 measure the same to 0.1 us)
__device__ __forceinline__ long long mass_weight(int rows) { return max(20, (rows + 15) / 16); }

// sum over W columns of 2^(s * f + nl) onto acc; MASKED: of those with a set bit
template <int W, bool MASKED>
__device__ __forceinline__ void add_exp(uint32_t da, float f, const float* nl, uint32_t bits0,
                                        uint32_t bits1, float (&acc)[8]) {
  uint32_t r[W];
  if constexpr (W == 64) tc::tmem_ld64(da, r);
  else tc::tmem_ld16(da, r);
#pragma unroll
  for (int t = 0; t < W; t += 4) {
    const float4 n = *reinterpret_cast<const float4*>(nl + t);
    float x[4] = {__uint_as_float(r[t]), __uint_as_float(r[t + 1]), __uint_as_float(r[t + 2]),
                  __uint_as_float(r[t + 3])};
    fma2v(x[0], x[1], f, n.x, n.y);
    fma2v(x[2], x[3], f, n.z, n.w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = ex2_ftz(x[i]);
      if (MASKED) x[i] = ((t < 32 ? bits0 : bits1) >> ((t + i) & 31)) & 1u ? x[i] : 0.f;
    }
    // (eight sums: with four, the packed adds' latency would bound the loop)
    add2(acc[t & 4], acc[(t & 4) + 1], x[0], x[1]);
    add2(acc[(t & 4) + 2], acc[(t & 4) + 3], x[2], x[3]);
  }
}

template <bool FP8, int QR>
__global__ void __launch_bounds__(kThreads, 1)
    attn_mass_kernel(const __grid_constant__ TreeLaunch p, const __grid_constant__ CUtensorMap kmap) {
  using C = MassCfg<FP8, QR>;
  constexpr int W = C::kCols;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kSmBars);
  uint64_t* k_empty = k_full + C::kTiles;
  uint64_t* raw_full = k_empty + C::kTiles;
  uint64_t* raw_empty = raw_full + C::kRaws;
  uint64_t* q_full = raw_empty + C::kRaws;  // [2]
  uint64_t* q_empty = q_full + 2;
  uint64_t* d_full = q_empty + 2;  // [warpgroup][buffer]
  uint64_t* d_empty = d_full + 4;
  uint64_t* drained = d_empty + 4;
  uint64_t* info_full = drained + 1;
  MassInfo* info = reinterpret_cast<MassInfo*>(smem + C::kSmInfo);
  int* misc = reinterpret_cast<int*>(smem + C::kSmMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 4);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = p.num_heads;

  if (tid == 0) {
    misc[0] = 0;
    for (int s = 0; s < C::kTiles; ++s) {
      mbar_init(&k_full[s], FP8 ? kLoaders : 1);
      // released by the products and, with bf16 keys, by the loaders: they then
      // follow the blocks' announcements and are never lapped
      mbar_init(&k_empty[s], FP8 ? 1 : 1 + kLoaders);
    }
    for (int s = 0; s < C::kRaws; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], kLoaders);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], kLoaders);
      mbar_init(&q_empty[s], 9);  // the issuer and the epilogue's warps
      for (int b = 0; b < 2; ++b) {
        mbar_init(&d_full[2 * s + b], 1);
        mbar_init(&d_empty[2 * s + b], 4);
      }
    }
    mbar_init(drained, 1);
    for (int s = 0; s < kInfos; ++s) mbar_init(&info_full[s], 1);
    fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, 512);
  const TreeSlice sl = tree_slice<kThreads>(
      p,
      [&](const TreeReq& r, int nv) -> long long { return r.bad ? 1 : (nv + kStart) * mass_weight(r.qlen * H); },
      reinterpret_cast<long long*>(smem));
  fence_proxy_async_smem();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  if (!sl.tiled && tid == 0 && blockIdx.x == 0) atomicOr(p.status, MSA_DEV_MALFORMED);

  if (sl.begin < sl.end) {
    if (warp == 0) {
      // ---------------------------------------------- keys
      long long pre = sl.pre;
      int n = 0;  // blocks
      bool ok = true;
      for (int q = sl.q; ok && q < p.batch.num_reqs && pre < sl.end; ++q) {
        TreeReq rq = sl.first;
        int nv = sl.visits;
        if (q != sl.q) {
          rq = tree_request(p, q);
          if (rq.qlen <= 0) continue;
          nv = tree_visits(p, q, rq);  // 1 for a poisoned request
        }
        const long long w = rq.bad ? 1 : mass_weight(rq.qlen * H);
        const long long first = pre + (rq.bad ? 0 : kStart * w);  // the first block's first item
        pre = first + nv * w;
        const int32_t* bt = p.batch.block_table + (long long)q * p.batch.bt_stride;
        if (!rq.bad) {
          // a bad page anywhere leaves the whole request as it is
          bool bad = false;
#pragma unroll 4
          for (int b = lane; b < rq.nb; b += 32) {
            const int page = __ldg(bt + b);
            bad |= page < 0 || page >= p.batch.num_pages;
          }
          if (__any_sync(0xffffffffu, bad)) rq.bad = MSA_DEV_BAD_PAGE;
        }
        if (rq.bad) {
          if (lane == 0) atomicOr(p.status, rq.bad);
          continue;
        }
        // blocks whose first item lies in the slice
        const int i0 = (int)((max(sl.begin, first) - first + w - 1) / w);
        const int i1 = (int)min((long long)nv, (max(sl.end, first) - first + w - 1) / w);
        for (int c0 = i0; ok && c0 < i1; c0 += 32) {
          int blk = 0, page = 0;
          if (c0 + lane < i1) {
            blk = c0 + lane;
            if (p.topk_idx) blk = p.list_blk[(long long)q * p.list_cap + blk];
            page = __ldg(bt + blk);
          }
          for (int i = 0; i < min(32, i1 - c0); ++i) {
            const int b = __shfl_sync(0xffffffffu, blk, i), pg = __shfl_sync(0xffffffffu, page, i);
            if constexpr (FP8) {
              const int s = n % C::kRaws;
              if (n >= C::kRaws) ok = warp_wait(&raw_empty[s], ((n / C::kRaws) - 1) & 1);
              if (!ok) break;
              if (lane == 0) {
                mbar_arrive_expect_tx(&raw_full[s], kRaw);
                bulk_g2s(smem + C::kSmRaw + s * kRaw, p.k + (long long)pg * kRaw, kRaw, &raw_full[s]);
              }
            } else {
              const int s = n % C::kTiles;
              if (n >= C::kTiles) ok = warp_wait(&k_empty[s], ((n / C::kTiles) - 1) & 1);
              if (!ok) break;
              if (lane == 0) {
                mbar_arrive_expect_tx(&k_full[s], kTile);
                for (int h = 0; h < 2; ++h)
                  tma_load_2d(smem + C::kSmK + s * kTile + h * kHalf, &kmap, 64 * h, pg * kBlock, &k_full[s]);
              }
            }
            if (lane == 0) {
              const bool all = !p.topk_idx || b >= rq.ctx / kBlock;
              MassInfo mi;
              mi.flags = (c0 + i == i0 ? kFirst : 0) | (kBlock * b + kBlock > rq.ctx || !all ? kMixed : 0);
              mi.nblk = i1 - i0;
              mi.q0 = rq.q0;
              mi.ctx = rq.ctx;
              mi.qlen = rq.qlen;
              mi.t0 = kBlock * b;
              mi.page = pg;
              mi.pad = 0;
              mi.rows = all ? nullptr : p.list_rows + ((long long)q * p.list_cap + c0 + i) * p.list_words;
              info[n % kInfos] = mi;
              mbar_arrive(&info_full[n % kInfos]);
            }
            ++n;
          }
        }
      }
      if (ok && lane == 0) {
        info[n % kInfos].flags = kEnd;
        mbar_arrive(&info_full[n % kInfos]);
      }
      if (!ok) {
        misc[0] = 1;
        // copies still in flight land before the CTA leaves
        const int ring = FP8 ? C::kRaws : C::kTiles;
        uint64_t* bars = FP8 ? raw_full : k_full;
        for (int i = max(0, n - ring); i < n; ++i) mbar_wait(&bars[i % ring], (i / ring) & 1);
      }
    } else if (warp == 1) {
      // ---------------------------------------------- products
      if (lane == 0) {
        int n0 = 0, x0 = 0;     // first block, first query load of the segment
        int steps[2] = {0, 0};  // pieces per epilogue warpgroup so far
        bool ok = true;
        for (;;) {
          ok = mbar_wait(&info_full[n0 % kInfos], (n0 / kInfos) & 1);
          if (!ok || (info[n0 % kInfos].flags & kEnd)) break;
          const int nblk = info[n0 % kInfos].nblk;
          const int rows = info[n0 % kInfos].qlen * H;
          const int chunks = (rows + QR - 1) / QR;
          const bool resident = chunks <= 2;
          for (int g = 0; ok && g < nblk; g += 2) {
            const int nb = min(2, nblk - g);
            const bool last = g + 2 >= nblk;
            for (int c = 0; ok && c < chunks; ++c) {
              const int x = x0 + (resident ? c : (g >> 1) * chunks + c), qb = x & 1;
              ok = mbar_wait(&q_full[qb], (x >> 1) & 1);
              const int n16 = (min(QR, rows - c * QR) + 15) / 16 * 16;
              const uint64_t qd = tc::desc_kmajor_sw128(smem_u32(smem + C::kSmQ + qb * C::kQBuf));
              for (int k0 = 0; ok && k0 < n16; k0 += kPiece) {
                const uint32_t idesc = tc::idesc_16(128, min(kPiece, n16 - k0), 0, FP8 ? 0 : 1);
                for (int b = 0; ok && b < nb; ++b) {
                  const int n = n0 + g + b, s = n % C::kTiles, buf = 2 * b + (steps[b] & 1);
                  if (c == 0 && k0 == 0) ok = ok && mbar_wait(&k_full[s], (n / C::kTiles) & 1);
                  if (steps[b] >= 2) ok = ok && mbar_wait(&d_empty[buf], ((steps[b] >> 1) - 1) & 1);
                  if (!ok) break;
                  tc::fence_after();
                  const uint64_t kd = tc::desc_kmajor_sw128(smem_u32(smem + C::kSmK + s * kTile));
#pragma unroll
                  for (int kk = 0; kk < 8; ++kk)
                    tc::mma_ss(tmem + kPiece * buf,
                               tc::desc_advance(kd, (kk >> 2) * kHalf + (kk & 3) * 32),
                               tc::desc_advance(qd, k0 * 128 + (kk >> 2) * (QR * 128) + (kk & 3) * 32),
                               idesc, kk > 0 ? 1u : 0u);
                  tc::commit(&d_full[buf]);
                  if (c == chunks - 1 && k0 + kPiece >= n16) tc::commit(&k_empty[s]);
                  ++steps[b];
                }
              }
              if (ok && (!resident || last)) tc::commit(&q_empty[qb]);
            }
          }
          if (!ok) break;
          x0 += resident ? chunks : (nblk + 1) / 2 * chunks;
          n0 += nblk;
        }
        if (!ok) misc[0] = 1;
        // every product has completed before the tensor memory is freed
        tc::commit(drained);
        if (!mbar_wait(drained, 0)) misc[0] = 1;
      }
    } else if (warp >= 16 - kLoaders) {
      // ---------------------------------------------- queries; e4m3 keys to f16
      const int lt = tid - (16 - kLoaders) * 32;
      int n0 = 0, x0 = 0;
      bool ok = true;
      for (;;) {
        ok = warp_wait(&info_full[n0 % kInfos], (n0 / kInfos) & 1);
        if (!ok || (info[n0 % kInfos].flags & kEnd)) break;
        const int nblk = info[n0 % kInfos].nblk, q0 = info[n0 % kInfos].q0;
        const int rows = info[n0 % kInfos].qlen * H;
        const int chunks = (rows + QR - 1) / QR;
        const bool resident = chunks <= 2;
        const uint16_t* qsrc = p.q + (long long)q0 * H * kHeadDim;
        const float* lsrc = p.lse + (long long)q0 * H;
        for (int g = 0; ok && g < nblk; g += 2) {
          if constexpr (!FP8) {
            for (int b = 0; ok && b < min(2, nblk - g); ++b) {
              const int n = n0 + g + b;
              ok = warp_wait(&info_full[n % kInfos], (n / kInfos) & 1);
              if (ok && lane == 0) mbar_arrive(&k_empty[n % C::kTiles]);
            }
          }
          if constexpr (FP8) {
            for (int b = 0; ok && b < min(2, nblk - g); ++b) {
              const int n = n0 + g + b, s = n % C::kTiles, rs = n % C::kRaws;
              ok = warp_wait(&raw_full[rs], (n / C::kRaws) & 1);
              if (n >= C::kTiles) ok = ok && warp_wait(&k_empty[s], ((n / C::kTiles) - 1) & 1);
              if (!ok) break;
              const uint8_t* raw = smem + C::kSmRaw + rs * kRaw;
              uint8_t* kt = smem + C::kSmK + s * kTile;
#pragma unroll 2
              for (int i = lt; i < kRaw / 16; i += kLoaders * 32) {
                const int row = i >> 3, ch = 2 * (i & 7);  // 16 codes: f16 chunks ch, ch + 1
                const uint4 v = lds128(raw + 16 * i);
                uint8_t* dst = kt + (ch >> 3) * kHalf + row * 128;
                *reinterpret_cast<uint4*>(dst + (((ch & 7) ^ (row & 7)) << 4)) =
                    make_uint4(e4m3x2_to_f16x2((uint16_t)v.x), e4m3x2_to_f16x2((uint16_t)(v.x >> 16)),
                               e4m3x2_to_f16x2((uint16_t)v.y), e4m3x2_to_f16x2((uint16_t)(v.y >> 16)));
                *reinterpret_cast<uint4*>(dst + ((((ch & 7) + 1) ^ (row & 7)) << 4)) =
                    make_uint4(e4m3x2_to_f16x2((uint16_t)v.z), e4m3x2_to_f16x2((uint16_t)(v.z >> 16)),
                               e4m3x2_to_f16x2((uint16_t)v.w), e4m3x2_to_f16x2((uint16_t)(v.w >> 16)));
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                mbar_arrive(&k_full[s]);
                mbar_arrive(&raw_empty[rs]);
              }
            }
          }
          for (int c = 0; ok && c < chunks && (g == 0 || !resident); ++c) {
            const int x = x0 + (resident ? c : (g >> 1) * chunks + c), qb = x & 1;
            if (x >= 2) ok = ok && warp_wait(&q_empty[qb], ((x >> 1) - 1) & 1);
            if (!ok) break;
            const int r0 = c * QR, nr = min(QR, rows - r0), n16 = (nr + 15) / 16 * 16;
            uint8_t* qd = smem + C::kSmQ + qb * C::kQBuf;
#pragma unroll 8
            for (int i = lt; i < n16 * 16; i += kLoaders * 32) {
              const int row = i >> 4, ch = i & 15;
              uint4 v = make_uint4(0u, 0u, 0u, 0u);  // rows past the end give S = 0
              if (row < nr) v = __ldg(reinterpret_cast<const uint4*>(qsrc + (long long)(r0 + row) * kHeadDim) + ch);
              if constexpr (FP8) {
                v.x = pack_f16x2(bf16lo(v.x), bf16hi(v.x));
                v.y = pack_f16x2(bf16lo(v.y), bf16hi(v.y));
                v.z = pack_f16x2(bf16lo(v.z), bf16hi(v.z));
                v.w = pack_f16x2(bf16lo(v.w), bf16hi(v.w));
              }
              *reinterpret_cast<uint4*>(qd + (ch >> 3) * (QR * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) = v;
            }
            float* nl = reinterpret_cast<float*>(smem + C::kSmNl) + qb * QR;
            for (int i = lt; i < min(QR, (nr + W - 1) / W * W); i += kLoaders * 32) {
              // a row that saw nothing (lse -inf) or lies past the end gives 2^-inf = 0
              const float l = i < nr ? __ldg(lsrc + r0 + i) : -INFINITY;
              nl[i] = l == -INFINITY ? -INFINITY : -l * kTreeLog2e;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[qb]);
          }
        }
        if (!ok) break;
        x0 += resident ? chunks : (nblk + 1) / 2 * chunks;
        n0 += nblk;
      }
      if (!ok) misc[0] = 1;
    } else if (warp >= 4) {
      // ---------------------------------------------- sums
      const int w = (warp - 4) >> 2, quarter = warp & 3;
      const int tok = quarter * 32 + lane;  // token of the block = tensor-memory lane
      const uint32_t d0 = tmem + ((uint32_t)(quarter * 32) << 16) + 2 * kPiece * w;
      float scale2 = p.softmax_scale * kTreeLog2e;
      if (p.scale_mode == MSA_SCALE_SCALAR) scale2 *= __ldg(p.k_scale);
      int n0 = 0, x0 = 0, step = 0;
      bool ok = true;
      for (;;) {
        ok = warp_wait(&info_full[n0 % kInfos], (n0 / kInfos) & 1);
        if (!ok || (info[n0 % kInfos].flags & kEnd)) break;
        const int nblk = info[n0 % kInfos].nblk, qlen = info[n0 % kInfos].qlen;
        const int q0 = info[n0 % kInfos].q0, ctx = info[n0 % kInfos].ctx;
        const int rows = qlen * H, chunks = (rows + QR - 1) / QR;
        const bool resident = chunks <= 2;
        float f_next = 0.f, old_next = 0.f;  // of the warpgroup's next block, loaded ahead
        const auto ahead = [&](int n) {
          if (!warp_wait(&info_full[n % kInfos], (n / kInfos) & 1)) return false;
          const long long at = (long long)info[n % kInfos].page * kBlock + tok;
          f_next = scale2;
          if (p.scale_mode == MSA_SCALE_PER_TOKEN_HEAD) f_next *= __ldg(p.k_scale + at);
          if (info[n % kInfos].t0 + tok < ctx) old_next = p.mass[at];
          return true;
        };
        if (w < nblk) ok = ahead(n0 + w);
        for (int g = 0; ok && g < nblk; g += 2) {
          const bool have = g + w < nblk, last = g + 2 >= nblk;
          int fl = 0, t = 0;
          const uint32_t* sel = nullptr;
          float* slot = nullptr;
          const float f = f_next, old = old_next;
          float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          if (have) {
            const MassInfo& mi = info[(n0 + g + w) % kInfos];
            fl = mi.flags;
            t = mi.t0 + tok;
            sel = mi.rows;
            slot = p.mass + (long long)mi.page * kBlock + tok;
          }
          for (int c = 0; ok && c < chunks; ++c) {
            const int x = x0 + (resident ? c : (g >> 1) * chunks + c), qb = x & 1;
            ok = warp_wait(&q_full[qb], (x >> 1) & 1);
            const int nr = min(QR, rows - c * QR);
            const float* nl = reinterpret_cast<const float*>(smem + C::kSmNl) + qb * QR;
            int j0 = -64;  // a lane holds the sight of row j0 + lane on the warp's tokens
            uint32_t win = 0;
            for (int k0 = 0; ok && have && k0 < nr; k0 += kPiece, ++step) {
              const int buf = step & 1, k1 = min(nr, k0 + kPiece);
              ok = warp_wait(&d_full[2 * w + buf], (step >> 1) & 1);
              if (!ok) break;
              tc::fence_after();
              const uint32_t da = d0 + kPiece * buf - k0;
              // W columns at a time; in a block that not every row sees whole, and
              // behind the last row, those that count are picked by a bit each
              int k = k0;
              if (!(fl & kMixed)) {
                for (; k + W <= k1; k += W) add_exp<W, false>(da + k, f, nl + k, 0u, 0u, acc);
              }
              for (; k < k1; k += W) {
                uint32_t bits[2] = {0u, 0u};
                if (fl & kMixed) {
                  // the rows that the columns belong to, in turn
                  const int first = c * QR + k, end = min(first + W, rows);
                  for (int at = first; at < end;) {
                    const int j = at / H, upto = min(end, (j + 1) * H) - first;
                    if (j >= j0 + 32) {
                      j0 = j;
                      win = 0;
                      if (j0 + lane < qlen) {
                        const int r = j0 + lane, tw = t - lane;
                        const bool rs = tree_row_selects(sel, r);
                        win = tree_vis16(p, q0 + r, r, ctx, qlen, tw, rs) |
                              tree_vis16(p, q0 + r, r, ctx, qlen, tw + 16, rs) << 16;
                      }
                    }
                    const uint32_t row = __shfl_sync(0xffffffffu, win, j - j0);
                    if ((row >> lane) & 1u) {
                      const uint64_t m = ((upto == 64 ? 0ull : 1ull << upto) - 1ull) & ~((1ull << (at - first)) - 1ull);
                      bits[0] |= (uint32_t)m;
                      bits[1] |= (uint32_t)(m >> 32);
                    }
                    at = first + upto;
                  }
                } else {
                  const uint64_t m = (1ull << (nr - k)) - 1ull;
                  bits[0] = (uint32_t)m;
                  bits[1] = (uint32_t)(m >> 32);
                }
                __syncwarp();
                add_exp<W, true>(da + k, f, nl + k, bits[0], bits[1], acc);
              }
              tc::fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&d_empty[2 * w + buf]);
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0 && (!resident || last)) mbar_arrive(&q_empty[qb]);
            // (streamed queries: the next block's place may wait for the other warpgroup,
            // which waits for this one's chunks; so behind the last of them)
            if (c == (resident ? 0 : chunks - 1) && g + 2 + w < nblk) ok = ahead(n0 + g + 2 + w);
          }
          // (a masked token of the block's rows that no row sees adds nothing)
          if (ok && have && t < ctx + qlen) {
            const float s = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
            *slot = t < ctx ? old + s : s;
          }
        }
        if (!ok) break;
        x0 += resident ? chunks : (nblk + 1) / 2 * chunks;
        n0 += nblk;
      }
      if (!ok) misc[0] = 1;
    }
  }
  tc::fence_before();
  __syncthreads();
  if (misc[0] && tid == 0) atomicOr(p.status, MSA_DEV_TIMEOUT);
  if (warp == 1) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <bool FP8, int QR>
cudaError_t launch_mass(const TreeLaunch& p, cudaStream_t stream) {
  using C = MassCfg<FP8, QR>;
  CUtensorMap kmap;
  memset(&kmap, 0, sizeof(kmap));
  if (!FP8 && !encode_map_2d(&kmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.k, kHeadDim,
                             max(1ll, (long long)p.batch.num_pages) * kBlock, kHeadDim * 2, 64, kBlock))
    return cudaErrorInvalidValue;
  auto kern = attn_mass_kernel<FP8, QR>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e != cudaSuccess) return e;
  kern<<<device_sm_count(), kThreads, C::kBytes, stream>>>(p, kmap);
  return cudaGetLastError();
}

template <bool FP8>
cudaError_t launch_rows(const TreeLaunch& p, cudaStream_t stream) {
  // rows of a chunk: one token's leave the shared memory to the stream of keys.  16
  // requests of 16384 tokens, us, chunks of 16 / 256: 16 rows x heads bf16 20.7 / 21.7,
  // e4m3 17.1 / 22.4; chunks of 256: 64 rows x heads 21.2 and 18.9, 128 25.2 and 21.6
  const int rows = p.max_rows * p.num_heads;
  return rows <= 16 ? launch_mass<FP8, 16>(p, stream) : launch_mass<FP8, 256>(p, stream);
}

}  // namespace

cudaError_t launch_attn_mass(const TreeLaunch& p, cudaStream_t stream) {
  if (p.topk_idx) {
    const cudaError_t e = launch_tree_plan(p, stream);
    if (e != cudaSuccess) return e;
  }
  return p.kv_fp8 ? launch_rows<true>(p, stream) : launch_rows<false>(p, stream);
}

}  // namespace msa
