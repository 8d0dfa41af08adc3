// tree_attn.cu -- attention of a request's drafted rows over its whole cache
// (or its selected blocks) and, by a bit mask, over each other.
//
// Mathematics.  Per row and head, out = sum_t e^(s_t - m) v_t / den over the
// visible t with den = sum_t e^(s_t - m) (+ e^(sink - m)): one pass over the
// tokens with a running maximum m and sum, and partial results (m, l, o) of
// disjoint token sets joined by o = sum_i 2^(m_i - M) o_i.  All exponents are
// in log2 units.
//
// Split.  A request's rows x heads are cut into tiles of TM rows (whole
// drafted tokens; one KV head, so a tile's rows share every key).  The flat
// list of (request, tile, visited block) is cut into equal contiguous slices,
// one per CTA of a persistent grid, from the lengths on the device: a ragged
// batch or one long request fills all SMs alike.  A CTA writes the tiles it
// covers whole; of a tile shared with its neighbours it writes a partial (at
// most two per CTA: its first and its last tile), joined by a second kernel in
// CTA order, so results do not depend on timing.
//
// This kernel works on warp MMA (m16n8k16, fp32 accumulation): with up to 32
// rows it is bound by the stream of K and V, which one producer warp keeps in
// flight (64-token stages by tensor copies, 128-byte swizzle), while 8
// consumer warps take 16 rows x 16 tokens each.  e4m3 codes become f16 in
// registers (exact).  Measured: 64 requests of one row x 16 heads over 512..32768
// bf16 tokens, 259 MB, in 53 us (4.9 TB/s); one request of 700 tokens in 11 us, the
// latencies of two launches, the list of lengths, a page number, K and V.
#include <string.h>

#include "tree_common.cuh"

namespace msa {
namespace {

constexpr int kConsWarps = 8;
constexpr int kTaThreads = (kConsWarps + 1) * 32;
constexpr int kStageTok = 64;
constexpr int kAccPad = 132;

// stage flags
constexpr int kFirst = 1, kLast = 2, kWhole = 4, kNoData = 8, kBadPage = 16, kPoison = 32,
              kEnd = 64, kMixed = 128;

struct StageInfo {
  int flags;
  int row0;   // first row (drafted token) of the tile in the batch
  int ntok;   // drafted tokens in the tile
  int j0;     // first one's index in its request
  int ctx, qlen;
  int t0;     // position of the stage's first token
  int seq;    // tokens of the request
  int cached_all;  // the block's cached tokens are visible to every row
  int slot;   // partial slot of the tile (used at kLast)
  uint32_t bad;
  int pad;
  const uint32_t* rows;  // selection bits of the block's rows, or NULL
};

template <bool FP8, int MW>
struct TaCfg {
  static constexpr int kM = 16 * MW;            // rows of a tile
  static constexpr int kNW = kConsWarps / MW;   // token groups
  static constexpr int kTile = kStageTok * kHeadDim * (FP8 ? 1 : 2);
  static constexpr int kStages = FP8 ? 8 : 5;
  static constexpr int kSmK = 0;
  static constexpr int kSmV = kSmK + kStages * kTile;
  static constexpr int kSmQ = kSmV + kStages * kTile;
  static constexpr int kSmS = kSmQ + kM * kHeadDim * 2;  // k, v scales of a stage: 2 x 64 fp32
  static constexpr int kSmAcc = kSmS + kStages * 2 * kStageTok * 4;
  static constexpr int kAccRows = kNW > 1 ? 64 : 0;
  static constexpr int kSmMl = kSmAcc + kAccRows * kAccPad * 4;
  static constexpr int kSmInfo = kSmMl + (kAccRows > 0 ? 64 * 8 : 0);
  static constexpr int kSmBar = kSmInfo + kStages * (int)sizeof(StageInfo);
  // full, empty per stage, q_empty, csync; then scan scratch
  static constexpr int kSmScan = kSmBar + (2 * kStages + 2) * 8;
  static constexpr int kBytes = kSmScan + 256 + 1024;  // + alignment slack
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <bool FP8, bool PTH, int MW>
__global__ void __launch_bounds__(kTaThreads, 1)
    tree_attn_kernel(const __grid_constant__ TreeLaunch p, const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  using C = TaCfg<FP8, MW>;
  constexpr int NW = C::kNW, M = C::kM;
  static_assert(!FP8 || NW > 1, "e4m3 pools: tiles of 32 rows at most, wider ones are tree_attn_tc.cu's");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kSmBar);
  uint64_t* empty = full + C::kStages;
  uint64_t* q_empty = empty + C::kStages;
  uint64_t* cbar = q_empty + 1;
  StageInfo* info = reinterpret_cast<StageInfo*>(smem + C::kSmInfo);
  long long* s_ll = reinterpret_cast<long long*>(smem + C::kSmAcc);  // free until the first merge
  if constexpr (C::kAccRows == 0) s_ll = reinterpret_cast<long long*>(smem + C::kSmQ);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned full_mask = 0xffffffffu;
  const int H = p.num_heads;
  const int tpt = M / H;  // drafted tokens per tile
  __shared__ float s_sink[kMaxHeads];
  if (tid < H) s_sink[tid] = p.sinks ? __ldg(p.sinks + tid) : 0.f;

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kConsWarps);
    }
    mbar_init(q_empty, kConsWarps);
    mbar_init(cbar, kConsWarps);
    fence_barrier_init();
  }
  const TreeSlice sl = tree_slice<kTaThreads>(
      p, [&](const TreeReq& r, int nv) { return tree_items(nv, (r.qlen + tpt - 1) / tpt); }, s_ll);
  fence_proxy_async_smem();
  __syncthreads();  // scratch is free, barriers are initialised
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0 && sl.begin >= sl.end) p.split[blockIdx.x].nrows = 0;
  if (!sl.tiled) {
    tree_write_all_empty(p);
    if (tid == 0 && blockIdx.x == 0) atomicOr(p.status, MSA_DEV_MALFORMED);
    return;
  }
  if (sl.begin >= sl.end) return;

  if (warp == kConsWarps) {
    // ------------------------------------------------ producer
    long long it = sl.begin, pre = sl.pre;
    int q = sl.q, n_stage = 0, n_seg = 0;
    bool ok = true;
    TreeSplit rec;
    rec.nrows = 0;
    // a stage of the ring that its last readers have released
    auto acquire = [&]() -> int {
      const int st = n_stage % C::kStages;
      if (n_stage >= C::kStages)
        ok = ok && __all_sync(full_mask, mbar_wait(&empty[st], ((n_stage / C::kStages) - 1) & 1));
      return st;
    };
    while (ok && it < sl.end) {
      TreeReq rq = sl.first;
      int nv = sl.visits;
      if (q != sl.q) {
        rq = tree_request(p, q);
        nv = rq.qlen > 0 ? tree_visits(p, q, rq) : 0;
      }
      const int tiles = (rq.qlen + tpt - 1) / tpt;
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
      const bool whole = nb == nv;
      StageInfo si;
      si.j0 = tile * tpt;
      si.ntok = min(tpt, rq.qlen - si.j0);
      si.row0 = rq.q0 + si.j0;
      si.ctx = rq.ctx;
      si.qlen = rq.qlen;
      si.seq = rq.ctx + rq.qlen;
      si.slot = 2 * blockIdx.x + (b0 > 0 ? 0 : 1);
      si.bad = rq.bad;
      si.rows = nullptr;
      if (b0 > 0 && sl.total * (blockIdx.x - 1) / sl.ctas <= sg.first) {
        // second of the CTAs that share this tile: it names them to the merge
        rec.nrows = si.ntok * H;
        rec.row0 = si.row0;
        rec.last = (int)((sg.end * sl.ctas - 1) / sl.total);
      }
      if (rq.bad) {
        const int st = acquire();
        if (!ok) break;
        si.flags = kFirst | kLast | kPoison | kNoData | kWhole;
        si.t0 = 0;
        si.cached_all = 0;
        if (lane == 0) {
          info[st] = si;
          mbar_arrive(&full[st]);
        }
        ++n_stage;
      }
      for (int c0 = 0; !rq.bad && ok && c0 < nb; c0 += 32) {
        // 32 blocks' numbers and pages at a time, one per lane
        int blk = 0, page = 0;
        if (c0 + lane < nb) {
          blk = b0 + c0 + lane;
          if (p.topk_idx) blk = p.list_blk[(long long)q * p.list_cap + blk];
          page = p.batch.block_table[(long long)q * p.batch.bt_stride + blk];
        }
        for (int i = 0; ok && i < min(32, nb - c0); ++i) {
          const int b = __shfl_sync(full_mask, blk, i), pg = __shfl_sync(full_mask, page, i);
          const bool bad_page = pg < 0 || pg >= p.batch.num_pages;
          const int ntok = min(kBlock, si.seq - kBlock * b);
          const int halves = ntok > kStageTok ? 2 : 1;
          si.cached_all = !p.topk_idx || b >= rq.ctx / kBlock;
          si.rows = si.cached_all
                        ? nullptr
                        : p.list_rows + ((long long)q * p.list_cap + b0 + c0 + i) * p.list_words;
          for (int h = 0; ok && h < halves; ++h) {
            const int st = acquire();
            const bool first = c0 + i == 0 && h == 0, last = c0 + i == nb - 1 && h == halves - 1;
            if (first && n_seg > 0)
              ok = ok && __all_sync(full_mask, mbar_wait(q_empty, (n_seg - 1) & 1));
            if (!ok) break;
            si.t0 = kBlock * b + kStageTok * h;
            si.flags = (first ? kFirst : 0) | (last ? kLast : 0) | (whole ? kWhole : 0) |
                       (bad_page ? kBadPage | kNoData : 0) |
                       (si.t0 + kStageTok > rq.ctx || !si.cached_all ? kMixed : 0);
            if (lane == 0) {
              info[st] = si;
              const uint32_t bytes = (bad_page ? 0u : 2u * C::kTile + (PTH ? 512u : 0u)) +
                                     (first ? (uint32_t)(M * kHeadDim * 2) : 0u);
              if (bytes) mbar_arrive_expect_tx(&full[st], bytes);
              else mbar_arrive(&full[st]);
              if (first) {
                tma_load_2d(smem + C::kSmQ, &qmap, 0, si.row0 * H, &full[st]);
                tma_load_2d(smem + C::kSmQ + M * 128, &qmap, 64, si.row0 * H, &full[st]);
              }
              if (!bad_page) {
                const int y = pg * kBlock + kStageTok * h;
                uint8_t* kd = smem + C::kSmK + st * C::kTile;
                uint8_t* vd = smem + C::kSmV + st * C::kTile;
                tma_load_2d(kd, &kmap, 0, y, &full[st]);
                if constexpr (!FP8) tma_load_2d(kd + C::kTile / 2, &kmap, 64, y, &full[st]);
                tma_load_2d(vd, &vmap, 0, y, &full[st]);
                if constexpr (!FP8) tma_load_2d(vd + C::kTile / 2, &vmap, 64, y, &full[st]);
                if constexpr (PTH) {
                  uint8_t* sd = smem + C::kSmS + st * 2 * kStageTok * 4;
                  bulk_g2s(sd, p.k_scale + y, 256, &full[st]);
                  bulk_g2s(sd + 256, p.v_scale + y, 256, &full[st]);
                }
              }
            }
            ++n_stage;
          }
          if (bad_page && lane == 0) atomicOr(p.status, MSA_DEV_BAD_PAGE);
        }
      }
      if (!rq.bad) ++n_seg;
    }
    if (ok) {
      const int st = acquire();
      if (ok && lane == 0) {
        info[st].flags = kEnd;
        mbar_arrive(&full[st]);
      }
    }
    if (lane == 0) p.split[blockIdx.x] = rec;
    if (!ok) {
      if (lane == 0) atomicOr(p.status, MSA_DEV_TIMEOUT);
      // copies still in flight land before the CTA leaves
      for (int i = max(0, n_stage - C::kStages); i < n_stage; ++i)
        mbar_wait(&full[i % C::kStages], (i / C::kStages) & 1);
    }
    return;
  }

  // -------------------------------------------------- consumers
  const int g = lane >> 2, c = lane & 3;
  const int mw = warp % MW, nw = warp / MW;
  float scale2 = p.softmax_scale * kTreeLog2e;
  if (p.scale_mode == MSA_SCALE_SCALAR) scale2 *= __ldg(p.k_scale);
  const float v_scalar = p.scale_mode == MSA_SCALE_SCALAR ? __ldg(p.v_scale) : 1.f;
  const uint32_t q_s = smem_u32(smem + C::kSmQ);
  constexpr float kHead = FP8 ? kHalfHead : 0.f;
  float o[16][4], m_run[2], l_run[2];
  uint32_t qa[8][4];
  bool bad = false;
  uint32_t cph = 0;
  bool dead = false;
  // all consumer warps (bounded, so that no warp waits for one that gave up)
  auto csync = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(cbar);
    dead = dead || !__all_sync(full_mask, mbar_wait(cbar, cph));
    cph ^= 1;
  };
  const int mrow[2] = {mw * 16 + g, mw * 16 + g + 8};  // this lane's rows of the tile
  const int mtok[2] = {mrow[0] / H, mrow[1] / H};
  // first column of n-tile j's pair in the accumulators: bf16 tiles hold dims
  // 8 j + 2 c, + 1; e4m3 tiles dims 32 c + j and 32 c + 16 + j
  int stage_of_tile = 0;

  for (int n = 0; !dead; ++n) {
    const int st = n % C::kStages;
    if (!__all_sync(full_mask, mbar_wait(&full[st], (n / C::kStages) & 1))) {
      dead = true;
      break;
    }
    const StageInfo& si = info[st];
    const int fl = si.flags;
    if (fl & kEnd) break;
    if (fl & kFirst) {
      m_run[0] = m_run[1] = -INFINITY;
      l_run[0] = l_run[1] = 0.f;
      bad = (fl & kPoison) != 0;
      stage_of_tile = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
      if (!(fl & kPoison)) {
        if constexpr (FP8) {
          // k-step kk, slots (2c, 2c+1) <-> dims 32c + 4kk + {0, 1}, slots (2c+8, 2c+9) <->
          // + {2, 3}: the order in which a lane's 32-byte span of a key row is read
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int row = mw * 16 + g + 8 * hh;
            const uint8_t* src = smem + C::kSmQ + (c >> 1) * (M * 128) + row * 128;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 w = lds128(src + (((4 * (c & 1) + i) ^ (row & 7)) << 4));
              qa[2 * i][hh] = pack_f16x2(bf16lo(w.x), bf16hi(w.x));
              qa[2 * i][2 + hh] = pack_f16x2(bf16lo(w.y), bf16hi(w.y));
              qa[2 * i + 1][hh] = pack_f16x2(bf16lo(w.z), bf16hi(w.z));
              qa[2 * i + 1][2 + hh] = pack_f16x2(bf16lo(w.w), bf16hi(w.w));
            }
          }
        } else {
          const int row = mw * 16 + (lane & 15);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const int ch = 2 * kk + (lane >> 4);
            ldsm4(q_s + (ch >> 3) * (M * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4), qa[kk]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty);
      }
    }
    bad |= (fl & kBadPage) != 0;
    const bool mine = NW < 8 || (nw >> 2) == (stage_of_tile & 1);
    ++stage_of_tile;
    if (mine && !(fl & kNoData)) {
      const uint8_t* ks = smem + C::kSmK + st * C::kTile;
      const uint8_t* vs = smem + C::kSmV + st * C::kTile;
      const float* scl = reinterpret_cast<const float*>(smem + C::kSmS) + st * 2 * kStageTok;
#pragma unroll 1
      for (int slab = NW >= 4 ? (nw & 3) : nw; slab < 4; slab += (NW >= 4 ? 4 : NW)) {
        const int t0 = si.t0 + 16 * slab;
        if (t0 >= si.seq) break;
        // ---- S = Q K^T, n-tile u: tokens 8u .. 8u + 7 of the slab
        float s[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.f;
        if constexpr (FP8) {
          uint32_t kw[2][8];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint8_t* kr = ks + (16 * slab + 8 * u + g) * kHeadDim;
            const uint4 a = lds128(kr + (((2 * c) ^ g) << 4)), b = lds128(kr + (((2 * c + 1) ^ g) << 4));
            kw[u][0] = a.x; kw[u][1] = a.y; kw[u][2] = a.z; kw[u][3] = a.w;
            kw[u][4] = b.x; kw[u][5] = b.y; kw[u][6] = b.z; kw[u][7] = b.w;
          }
          // (two chains per n-tile: the even and the odd k-steps)
          float s2[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
#pragma unroll
            for (int u = 0; u < 2; ++u)
              mma16816<true>(kk & 1 ? s2[u] : s[u], qa[kk], e4m3x2_to_f16x2((uint16_t)(kw[u][kk] & 0xffffu)),
                             e4m3x2_to_f16x2((uint16_t)(kw[u][kk] >> 16)));
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u][e] += s2[u][e];
        } else {
          const uint32_t kb = smem_u32(ks);
          uint32_t kf[4][2][4];
#pragma unroll
          for (int kp = 0; kp < 4; ++kp)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int row = 16 * slab + 8 * u + (lane & 7), ch = 4 * kp + (lane >> 3);
              ldsm4(kb + (ch >> 3) * (C::kTile / 2) + row * 128 + (((ch & 7) ^ (row & 7)) << 4), kf[kp][u]);
            }
          // (two chains per n-tile: the even and the odd k-steps)
          float s2[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int kp = 0; kp < 4; ++kp)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              mma16816<false>(s[u], qa[2 * kp], kf[kp][u][0], kf[kp][u][1]);
              mma16816<false>(s2[u], qa[2 * kp + 1], kf[kp][u][2], kf[kp][u][3]);
            }
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u][e] += s2[u][e];
        }
        // ---- scale and mask
        uint32_t vis[2] = {0xffffu, 0xffffu};
        if (fl & kMixed) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            vis[hh] = 0;
            if (mtok[hh] < si.ntok) {
              const int j = si.j0 + mtok[hh];
              vis[hh] = tree_vis16(p, si.row0 + mtok[hh], j, si.ctx, si.qlen, t0,
                                   tree_row_selects(si.rows, j));
            }
          }
        }
        float vsc[2][2], z[2][4];  // a token's v scale, and the exponents of P (times it)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = 8 * u + 2 * c + e;
            float f = scale2, lv = 0.f;
            if constexpr (PTH) {
              f *= scl[16 * slab + t];
              vsc[u][e] = scl[kStageTok + 16 * slab + t];
              lv = log2_scale(vsc[u][e]);
            }
            s[u][e] = (vis[0] >> t) & 1u ? s[u][e] * f : -INFINITY;
            s[u][2 + e] = (vis[1] >> t) & 1u ? s[u][2 + e] * f : -INFINITY;
            z[u][e] = PTH ? s[u][e] + lv : s[u][e];
            z[u][2 + e] = PTH ? s[u][2 + e] + lv : s[u][2 + e];
          }
        // ---- the reference of P, moved only when an exponent exceeds it by more than the slack
        float mx[2];
        bool move = false;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          mx[hh] = fmaxf(fmaxf(z[0][2 * hh], z[0][2 * hh + 1]), fmaxf(z[1][2 * hh], z[1][2 * hh + 1]));
          mx[hh] = fmaxf(mx[hh], __shfl_xor_sync(full_mask, mx[hh], 1));
          mx[hh] = fmaxf(mx[hh], __shfl_xor_sync(full_mask, mx[hh], 2)) - kHead;
          move |= mx[hh] > m_run[hh] + kSlack || (m_run[hh] == -INFINITY && mx[hh] > -INFINITY);
        }
        if (__any_sync(full_mask, move)) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float al = 1.f;
            if (mx[hh] > m_run[hh]) {
              al = m_run[hh] == -INFINITY ? 1.f : ex2_ftz(m_run[hh] - mx[hh]);
              m_run[hh] = mx[hh];
            }
            l_run[hh] *= al;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              o[j][2 * hh] *= al;
              o[j][2 * hh + 1] *= al;
            }
          }
        }
        float pr[2][4];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const float base = m_run[hh] == -INFINITY ? 0.f : m_run[hh];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              pr[u][2 * hh + e] = ex2_ftz(s[u][2 * hh + e] - base);
              l_run[hh] += pr[u][2 * hh + e];
            }
        }
        if constexpr (PTH) {
          // (the scale of a token that the row does not see may be anything)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                pr[u][2 * hh + e] = (vis[hh] >> (8 * u + 2 * c + e)) & 1u ? pr[u][2 * hh + e] * vsc[u][e] : 0.f;
        }
        uint32_t pa[4];
        if constexpr (FP8) {
          pa[0] = pack_f16x2(pr[0][0], pr[0][1]);
          pa[1] = pack_f16x2(pr[0][2], pr[0][3]);
          pa[2] = pack_f16x2(pr[1][0], pr[1][1]);
          pa[3] = pack_f16x2(pr[1][2], pr[1][3]);
        } else {
          pa[0] = pack_bf16x2(pr[0][0], pr[0][1]);
          pa[1] = pack_bf16x2(pr[0][2], pr[0][3]);
          pa[2] = pack_bf16x2(pr[1][0], pr[1][1]);
          pa[3] = pack_bf16x2(pr[1][2], pr[1][3]);
        }
        // ---- O += P V.  In a block that not every row sees whole, a value
        // that is not finite must not meet the zero weight of a row that does
        // not see it: such values are taken out of the product and added for
        // the rows that do (tokens past the end: for none).
        bool odd = false;
        if constexpr (FP8) {
          uint32_t vw[4][4];
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const int t = 2 * c + (a & 1) + 8 * (a >> 1), row = 16 * slab + t;
            const uint4 w = lds128(vs + row * kHeadDim + ((g ^ (row & 7)) << 4));
            vw[a][0] = w.x; vw[a][1] = w.y; vw[a][2] = w.z; vw[a][3] = w.w;
          }
          if (fl & kMixed) {
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                // bytes whose low seven bits are all ones (NaN)
                const uint32_t x = vw[a][w] & 0x7f7f7f7fu;
                const uint32_t nan = (x + 0x01010101u) & 0x80808080u;
                odd |= nan != 0;
                vw[a][w] &= ~((nan >> 7) * 0xffu);
              }
          }
#pragma unroll
          for (int j2 = 0; j2 < 8; ++j2) {
            const int wi = j2 >> 1, by = 2 * (j2 & 1);
            const uint32_t sel = (uint32_t)(by | ((4 + by) << 4) | ((by + 1) << 8) | ((5 + by) << 12));
            const uint32_t lo = prmt(vw[0][wi], vw[1][wi], sel);  // tokens 2c, 2c + 1
            const uint32_t hi = prmt(vw[2][wi], vw[3][wi], sel);  // tokens 2c + 8, 2c + 9
            mma16816<true>(o[2 * j2], pa, e4m3x2_to_f16x2((uint16_t)(lo & 0xffffu)),
                           e4m3x2_to_f16x2((uint16_t)(hi & 0xffffu)));
            mma16816<true>(o[2 * j2 + 1], pa, e4m3x2_to_f16x2((uint16_t)(lo >> 16)),
                           e4m3x2_to_f16x2((uint16_t)(hi >> 16)));
          }
        } else {
          const uint32_t vb = smem_u32(vs);
          uint32_t vf[8][4];
#pragma unroll
          for (int jp = 0; jp < 8; ++jp) {
            const int row = 16 * slab + (lane & 15), ch = 2 * jp + (lane >> 4);
            ldsm4t(vb + (ch >> 3) * (C::kTile / 2) + row * 128 + (((ch & 7) ^ (row & 7)) << 4), vf[jp]);
          }
          if (fl & kMixed) {
#pragma unroll
            for (int jp = 0; jp < 8; ++jp)
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                uint32_t& b = vf[jp][w];
                const bool o0 = (b & 0x7f80u) == 0x7f80u, o1 = (b & 0x7f800000u) == 0x7f800000u;
                odd |= o0 | o1;
                b &= (o0 ? 0xffff0000u : 0xffffffffu) & (o1 ? 0x0000ffffu : 0xffffffffu);
              }
          }
#pragma unroll
          for (int jp = 0; jp < 8; ++jp) {
            mma16816<false>(o[2 * jp], pa, vf[jp][0], vf[jp][1]);
            mma16816<false>(o[2 * jp + 1], pa, vf[jp][2], vf[jp][3]);
          }
        }
        if ((fl & kMixed) && __any_sync(full_mask, odd)) {
#pragma unroll 1
          for (int t = 0; t < 16; ++t) {
            const int src = (lane & ~3) | ((t & 7) >> 1);
            const float a0 = (t & 8) ? ((t & 1) ? pr[1][1] : pr[1][0]) : ((t & 1) ? pr[0][1] : pr[0][0]);
            const float a1 = (t & 8) ? ((t & 1) ? pr[1][3] : pr[1][2]) : ((t & 1) ? pr[0][3] : pr[0][2]);
            const float p0 = __shfl_sync(full_mask, a0, src), p1 = __shfl_sync(full_mask, a1, src);
            const int row = 16 * slab + t;
#pragma unroll
            for (int j = 0; j < 16; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float x;
                bool o1;
                if constexpr (FP8) {
                  const uint8_t code = vs[row * kHeadDim + (((2 * c + e) ^ (row & 7)) << 4) + j];
                  o1 = (code & 0x7f) == 0x7f;
                  x = __uint_as_float(0x7fc00000u);
                } else {
                  const int d = 8 * j + 2 * c + e;
                  const uint16_t code = *reinterpret_cast<const uint16_t*>(
                      vs + (d >> 6) * (C::kTile / 2) + row * 128 +
                      ((((d >> 3) & 7) ^ (row & 7)) << 4) + 2 * (d & 7));
                  o1 = (code & 0x7f80u) == 0x7f80u;
                  x = __uint_as_float((uint32_t)code << 16);
                }
                if (o1 && ((vis[0] >> t) & 1u)) o[j][e] += p0 * x;
                if (o1 && ((vis[1] >> t) & 1u)) o[j][2 + e] += p1 * x;
              }
          }
          __syncwarp();
        }
      }
    }
    // ---- the tile's end: join the token groups, write
    if (fl & kLast) {
      const int row0 = si.row0, ntok = si.ntok, slot = si.slot;
      const uint32_t why = si.bad;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        l_run[hh] += __shfl_xor_sync(full_mask, l_run[hh], 1);
        l_run[hh] += __shfl_xor_sync(full_mask, l_run[hh], 2);
      }
      if constexpr (NW > 1) {
        // The upper half of the token groups hands its sums to the lower half
        // (lane by lane: who reads a place writes the joined sums back to it);
        // then all threads join the 64 / M groups left and write the rows.
        float* acc = reinterpret_cast<float*>(smem + C::kSmAcc);
        float2* ml = reinterpret_cast<float2*>(smem + C::kSmMl);
        // place of accumulator (j, e) in its row: its dim (e4m3: spread over the banks)
        auto place = [&](int j, int e) {
          return FP8 ? 33 * c + 16 * e + j : 8 * j + 2 * c + e;
        };
        if (nw >= NW / 2) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int at = (nw - NW / 2) * M + mrow[hh];
            if (c == 0) ml[at] = make_float2(m_run[hh], l_run[hh]);
#pragma unroll
            for (int j = 0; j < 16; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) acc[at * kAccPad + place(j, e)] = o[j][2 * hh + e];
          }
        }
        csync();
        if (nw < NW / 2) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int at = nw * M + mrow[hh];
            const float2 x = ml[at];
            float y[16][2];
#pragma unroll
            for (int j = 0; j < 16; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) y[j][e] = acc[at * kAccPad + place(j, e)];
            const float mn = fmaxf(m_run[hh], x.x), base = mn == -INFINITY ? 0.f : mn;
            // (a side that saw nothing has m = -inf and zeros)
            const float ga = m_run[hh] == -INFINITY ? 1.f : ex2_ftz(m_run[hh] - base);
            const float gb = x.x == -INFINITY ? 1.f : ex2_ftz(x.x - base);
            __syncwarp();
            if (c == 0) ml[at] = make_float2(mn, l_run[hh] * ga + x.y * gb);
#pragma unroll
            for (int j = 0; j < 16; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                acc[at * kAccPad + place(j, e)] = o[j][2 * hh + e] * ga + y[j][e] * gb;
          }
        }
        csync();
        if (!dead) {
          constexpr int G = 64 / M, T = 256 / M;  // groups left; threads of a row
          const int m = tid / T, d0 = 4 * (tid % T);
          float mg[G], lt = 0.f, mt = -INFINITY;
#pragma unroll
          for (int i = 0; i < G; ++i) mt = fmaxf(mt, ml[i * M + m].x);
          const float base = mt == -INFINITY ? 0.f : mt;
#pragma unroll
          for (int i = 0; i < G; ++i) {
            const float2 x = ml[i * M + m];
            mg[i] = x.x == -INFINITY ? 1.f : ex2_ftz(x.x - base);
            lt += x.y * mg[i];
          }
          if (m < ntok * H) {
            const bool whole = (fl & kWhole) != 0, none = bad || (mt == -INFINITY && lt == 0.f);
            const float sink = s_sink[m % H];
            const TreeRowEnd e = tree_row_end(none ? -INFINITY : mt, none ? 0.f : lt, p.sinks != nullptr,
                                              sink * kTreeLog2e, v_scalar);
            const long long r = (long long)row0 * H + m;
            if (whole) {
              if (d0 == 0) p.lse[r] = none ? (p.sinks ? sink : -INFINITY) : e.lse;
            } else if (d0 == 0) {
              p.part_ml[(long long)slot * M + m] = make_float2(mt, lt);
              if (m == 0) p.part_bad[slot] = bad ? 1 : 0;
            }
#pragma unroll
            for (int d = d0; d < kHeadDim; d += 4 * T) {
              float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int i = 0; i < G; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  v[k] += mg[i] * acc[(i * M + m) * kAccPad + (FP8 ? d + k + (d >> 5) : d + k)];
              if (whole) {
                const uint2 w = make_uint2(pack_bf16x2(v[0] * e.f, v[1] * e.f), pack_bf16x2(v[2] * e.f, v[3] * e.f));
                *reinterpret_cast<uint2*>(p.out + r * kHeadDim + d) = none ? make_uint2(0u, 0u) : w;
              } else {
                // [4-dim group][row][4 dims]
                reinterpret_cast<float4*>(p.part_o)[((long long)slot * (kHeadDim / 4) + d / 4) * M + m] =
                    make_float4(v[0], v[1], v[2], v[3]);
              }
            }
          }
          if (bad && why && tid == 0) atomicOr(p.status, why);
        }
        csync();  // read before the next tile's sums overwrite it
      } else if (!dead) {
        if (bad && why && warp == 0 && lane == 0) atomicOr(p.status, why);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int m = mrow[hh];
          if (m >= ntok * H) continue;
          if (fl & kWhole) {
            TreeRowEnd e;
            const float sink2 = p.sinks ? __ldg(p.sinks + m % H) * kTreeLog2e : 0.f;
            if (bad) e = tree_row_end(-INFINITY, 0.f, p.sinks != nullptr, sink2, 1.f);
            else e = tree_row_end(m_run[hh], l_run[hh], p.sinks != nullptr, sink2, v_scalar);
            const long long r = (long long)row0 * H + m;
            const bool none = bad || (m_run[hh] == -INFINITY && l_run[hh] == 0.f);
            if (c == 0) p.lse[r] = p.sinks && none ? __ldg(p.sinks + m % H) : e.lse;
            uint16_t* dst = p.out + r * kHeadDim;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              *reinterpret_cast<uint32_t*>(dst + 8 * j + 2 * c) =
                  none ? 0u : pack_bf16x2(o[j][2 * hh] * e.f, o[j][2 * hh + 1] * e.f);
          } else {
            if (m == 0 && c == 0) p.part_bad[slot] = bad ? 1 : 0;
            if (c == 0) p.part_ml[(long long)slot * M + m] = make_float2(m_run[hh], l_run[hh]);
            // [4-dim group][row][4 dims]: rows of a group are contiguous
            float* dst = p.part_o + ((long long)slot * (kHeadDim / 4) * M + m) * 4;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              *reinterpret_cast<float2*>(dst + (2 * j + (c >> 1)) * M * 4 + 2 * (c & 1)) =
                  make_float2(o[j][2 * hh], o[j][2 * hh + 1]);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }
  if (dead && lane == 0) atomicOr(p.status, MSA_DEV_TIMEOUT);
}

// ------------------------------------------------------------------ merge

constexpr int kMgThreads = 256, kMgWarps = kMgThreads / 32;
constexpr int kMaxMainCtas = 512;  // (the main kernels run one CTA per SM)
constexpr int kMgSets = kMgThreads / 32;  // sets of 32 threads, 4 dims a thread
constexpr int kMgLoads = 4;               // partials that a thread has in flight

// Sets that share a row's partials.  Two rows or more to a unit fill the 32-byte
// sectors of a partial (a row to a unit from 17 partials on: 110 us against 103 for 2
// requests of 33 rows x 12 heads over 131K tokens, 39 partials to a row); a row alone
// is for tiles that most of the GPU shared.  Eight loads in flight, at two CTAs an SM,
// help small trees (24.8 us against 26.6) and cost wide ones (84.9 against 82.5, 105
// against 103).
__device__ __forceinline__ int merge_parts(int n) {
  return n <= 8 ? 1 : n <= 16 ? 2 : n <= 64 ? 4 : 8;
}

// Joins the partials of the tiles that several CTAs share.  A work unit is
// kMgSets / parts rows of a tile, each row's partials shared by `parts` sets;
// each CTA takes every gridDim-th unit.
__global__ void __launch_bounds__(kMgThreads, 3) tree_merge_kernel(const __grid_constant__ TreeLaunch p,
                                                                int grid_main, int tile_rows) {
  __shared__ float4 s_o[kMgThreads];
  __shared__ float s_m[kMgSets], s_l[kMgSets];
  __shared__ int s_bad[kMgSets], s_sum[kMgWarps], s_base[kMaxMainCtas];
  __shared__ TreeSplit s_rec[kMaxMainCtas];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = p.num_heads;
  const float vs = p.scale_mode == MSA_SCALE_SCALAR ? __ldg(p.v_scale) : 1.f;
  // the split tiles' work units, by a prefix sum over the records
  long long total = 0;
  for (int c0 = 0; c0 < grid_main; c0 += kMgThreads) {
    const int c = c0 + threadIdx.x;
    TreeSplit rec;
    rec.nrows = 0;
    if (c > 0 && c < grid_main) rec = p.split[c];
    const int n = rec.last - c + 2;  // partials: CTAs c - 1 .. last
    const int per = kMgSets / merge_parts(n);
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
      s_base[c] = (int)total + before;
      s_rec[c] = rec;
    }
    for (int w = 0; w < kMgWarps; ++w) total += s_sum[w];
    __syncthreads();
  }
  for (int unit = blockIdx.x; unit < total; unit += gridDim.x) {
    int lo = 0, hi = grid_main - 1;  // last record whose first unit is <= unit
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_base[mid] <= unit) lo = mid; else hi = mid - 1;
    }
    const int c = lo;
    const TreeSplit rec = s_rec[c];
    const int n = rec.last - c + 2;
    const int parts = merge_parts(n), per = kMgSets / parts;
    // neighbouring threads take the unit's rows, then the 4-dim groups, then the parts
    const int row = threadIdx.x & (per - 1), x = threadIdx.x / per;
    const int g = x & 31, part = x >> 5;
    const int m0 = (unit - s_base[c]) * per, m = m0 + row;
    const bool live = m < rec.nrows;
    float M = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    int bad = 0;
    if (live) {
      for (int i0 = part; i0 < n; i0 += kMgLoads * parts) {
        float2 ml[kMgLoads];
        float4 v[kMgLoads];
#pragma unroll
        for (int u = 0; u < kMgLoads; ++u) {
          const int i = i0 + u * parts;
          ml[u] = make_float2(-INFINITY, 0.f);
          v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < n) {
            const long long slot = 2ll * (c - 1 + i) + (i == 0 ? 1 : 0);
            bad |= p.part_bad[slot];
            ml[u] = p.part_ml[slot * tile_rows + m];
            v[u] = reinterpret_cast<const float4*>(p.part_o)[(slot * (kHeadDim / 4) + g) * tile_rows + m];
          }
        }
        float mn = M;
#pragma unroll
        for (int u = 0; u < kMgLoads; ++u) mn = fmaxf(mn, ml[u].x);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float f0 = M == -INFINITY ? 1.f : ex2_ftz(M - ref);
        L *= f0;
        a.x *= f0; a.y *= f0; a.z *= f0; a.w *= f0;
#pragma unroll
        for (int u = 0; u < kMgLoads; ++u) {
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
      const float sink = p.sinks ? __ldg(p.sinks + m % H) : 0.f;
      const TreeRowEnd e = tree_row_end(M, L, p.sinks != nullptr, sink * kTreeLog2e, vs);
      const long long r = (long long)rec.row0 * H + m;
      uint2 w = make_uint2(pack_bf16x2(a.x * e.f, a.y * e.f), pack_bf16x2(a.z * e.f, a.w * e.f));
      if (none) w = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(p.out + r * kHeadDim + 4 * g) = w;
      if (g == 0) p.lse[r] = none ? (p.sinks ? sink : -INFINITY) : e.lse;
    }
  }
}

// ------------------------------------------------------------------- plan

// Per request with selected blocks: the visited blocks ascending (those that
// some row names among the cached whole blocks, and every block from the
// context's last one on) and, per visited block, one bit per row that reads
// its cached tokens.
constexpr int kPlanThreads2 = 256;
__global__ void __launch_bounds__(kPlanThreads2) tree_plan_kernel(const TreeLaunch p) {
  __shared__ uint32_t bits[kMaxBlocksPerRow / 32];
  __shared__ int rank[kMaxBlocksPerRow / 32 + 1];
  __shared__ int s_part[kPlanThreads2 / 32];
  const int q = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = p.batch.num_reqs;
  bool ok = p.batch.cu_seqlens_q[0] == 0 && p.batch.cu_seqlens_q[R] == p.batch.num_rows;
  for (int i = tid; i < R; i += kPlanThreads2)
    ok &= p.batch.cu_seqlens_q[i + 1] >= p.batch.cu_seqlens_q[i];
  if (!__syncthreads_and(ok)) return;  // the main kernel reports it
  const TreeReq rq = tree_request(p, q);
  if (rq.bad || rq.qlen <= 0) return;
  const int words = (rq.nb + 31) / 32, whole = rq.ctx / kBlock;
  bool bad = false;
  for (int b = tid; b < rq.nb; b += kPlanThreads2) {
    const int page = p.batch.block_table[(long long)q * p.batch.bt_stride + b];
    bad |= page < 0 || page >= p.batch.num_pages;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) p.list_count[q] = -1;
    return;
  }
  for (int w = tid; w < words; w += kPlanThreads2) {
    uint32_t x = 0;
    for (int b = 32 * w; b < min(32 * w + 32, rq.nb); ++b)
      if (b >= whole) x |= 1u << (b & 31);
    bits[w] = x;
  }
  __syncthreads();
  const long long picks = (long long)rq.qlen * p.topk;
  const int32_t* sel = p.topk_idx + (long long)rq.q0 * p.topk;
  for (long long i = tid; i < picks; i += kPlanThreads2) {
    const int b = sel[i];
    if (b >= 0 && b < whole) atomicOr(&bits[b >> 5], 1u << (b & 31));
  }
  __syncthreads();
  // exclusive popcount prefix over the words
  int base = 0;
  for (int w0 = 0; w0 < words; w0 += kPlanThreads2) {
    const int w = w0 + tid;
    const int n = w < words ? __popc(bits[w]) : 0;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_part[warp] = x;
    __syncthreads();
    int before = base;
    for (int i = 0; i < kPlanThreads2 / 32; ++i) {
      if (i < warp) before += s_part[i];
      base += s_part[i];
    }
    if (w < words) rank[w] = before + x - n;
    __syncthreads();
  }
  int32_t* list = p.list_blk + (long long)q * p.list_cap;
  uint32_t* rows = p.list_rows + (long long)q * p.list_cap * p.list_words;
  const int count = min(base, p.list_cap);  // (the capacity holds any union)
  if (tid == 0) p.list_count[q] = count;
  for (int i = tid; i < count * p.list_words; i += kPlanThreads2) rows[i] = 0u;
  for (int w = tid; w < words; w += kPlanThreads2) {
    uint32_t x = bits[w];
    for (int at = rank[w]; x && at < count; ++at, x &= x - 1) list[at] = 32 * w + __ffs(x) - 1;
  }
  __syncthreads();
  for (long long i = tid; i < picks; i += kPlanThreads2) {
    const int b = sel[i], j = (int)(i / p.topk);
    if (b < 0 || b >= whole) continue;
    const int at = rank[b >> 5] + __popc(bits[b >> 5] & ((1u << (b & 31)) - 1u));
    if (at < count) atomicOr(rows + (long long)at * p.list_words + (j >> 5), 1u << (j & 31));
  }
}

cudaError_t launch_merge(const TreeLaunch& p, int grid, int tile_rows, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  // (a unit holds a row x head at least)
  cfg.gridDim = dim3((unsigned)max(1ll, min(6ll * grid, (long long)p.batch.num_rows * p.num_heads)));
  cfg.blockDim = dim3(kMgThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel, p, grid, tile_rows);
}

template <bool FP8, bool PTH, int MW>
cudaError_t launch_main(const TreeLaunch& p, cudaStream_t stream) {
  using C = TaCfg<FP8, MW>;
  CUtensorMap qmap, kmap, vmap;
  memset(&qmap, 0, sizeof(qmap));
  const CUtensorMapDataType t = FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const long long toks = max(1ll, (long long)p.batch.num_pages) * kBlock;
  const int box = FP8 ? 128 : 64, pitch = kHeadDim * (FP8 ? 1 : 2);
  if (!encode_map_2d(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.q, kHeadDim,
                     (long long)p.batch.num_rows * p.num_heads, kHeadDim * 2, 64, C::kM) ||
      !encode_map_2d(&kmap, t, p.k, kHeadDim, toks, pitch, box, kStageTok) ||
      !encode_map_2d(&vmap, t, p.v, kHeadDim, toks, pitch, box, kStageTok))
    return cudaErrorInvalidValue;
  auto kern = tree_attn_kernel<FP8, PTH, MW>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e != cudaSuccess) return e;
  const int grid = min(device_sm_count(), kMaxMainCtas);
  kern<<<grid, kTaThreads, C::kBytes, stream>>>(p, qmap, kmap, vmap);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_merge(p, grid, C::kM, stream);
}

// Up to 32 rows x heads per request (one token of up to 16 heads, two of 16) warp MMA,
// which starts sooner; above, the 5th-generation tensor cores, whose tiles of 128 rows
// cost the same however few are used.  The rule goes by the batch's largest request.
// 16 requests of 16384 tokens, us, this kernel / tree_attn_tc.cu (the stream of K and V
// would take 20 for bf16, 10 for e4m3):
//   rows x heads      16        32          64          128
//   bf16            33.9 /  39.7 / 40.7  61.0 / 40.9  87.0 / 44.3
//   e4m3            31.4 /  40.4 / 46.6  62.3 / 46.9  96.8 / 51.1
//   e4m3, scales    33.1 /  44.8 / 55.7  66.8 / 57.4   107 / 63.1
// What is above the stream here is its start and the merge (11 us for one request of 700
// tokens), ~14 blocks a CTA, and with 32 rows the products, two tiles of 16 rows by eight
// warps that read every fragment of K and V from shared memory twice.
// bf16 pools with a scale per token, which the latter does not take, stay here (35.2,
// 43.4, 67.5, 100).
// The tile is the smallest that holds a request's rows, so that short trees do not
// carry empty rows through the products (one token of 16 heads: tile 16).
template <bool FP8, bool PTH>
cudaError_t launch_tile(const TreeLaunch& p, cudaStream_t stream) {
  const int m = p.max_rows * p.num_heads;
  if (m <= 16) return launch_main<FP8, PTH, 1>(p, stream);
  if (m <= 32) return launch_main<FP8, PTH, 2>(p, stream);
  if constexpr (!FP8 && PTH) {
    return m <= 64 ? launch_main<FP8, PTH, 4>(p, stream) : launch_main<FP8, PTH, 8>(p, stream);
  } else {
    const int grid = min(device_sm_count(), kMaxMainCtas);
    const cudaError_t e = launch_tree_attn_tc(p, grid, stream);
    return e != cudaSuccess ? e : launch_merge(p, grid, 256, stream);
  }
}

}  // namespace

// Rows of a partial, at most: the tensor-core kernel takes pairs of 128-row tiles.
int tree_part_rows(int max_rows, int num_heads) {
  const int m = max_rows * num_heads;
  return m <= 16 ? 16 : m <= 32 ? 32 : 256;
}

cudaError_t launch_tree_plan(const TreeLaunch& p, cudaStream_t stream) {
  tree_plan_kernel<<<p.batch.num_reqs, kPlanThreads2, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_tree_attn(const TreeLaunch& p, cudaStream_t stream) {
  if (p.topk_idx) {
    const cudaError_t e = launch_tree_plan(p, stream);
    if (e != cudaSuccess) return e;
  }
  const bool pth = p.scale_mode == MSA_SCALE_PER_TOKEN_HEAD;
  if (p.kv_fp8) return pth ? launch_tile<true, true>(p, stream) : launch_tile<true, false>(p, stream);
  return pth ? launch_tile<false, true>(p, stream) : launch_tile<false, false>(p, stream);
}

}  // namespace msa
