// evict.cu -- eviction from the cache: the tokens a request keeps under a
// budget, and the in-place move of kept tokens (which also commits the
// accepted path of a draft tree).
//
// Selection.  Orderable 32-bit keys of the masses (NaN lowest, -0 = +0), a
// radix selection of the need-th largest by digits of 11, 11 and 10 bits, then
// an ordered pass that keeps keys above it and the first of those equal to it.
// One thread-block cluster per request; each CTA reads its share of the tokens
// once, into registers (large shares into shared memory), a warp a contiguous run
// of them.  The masses are 4 bytes a token, so the time is not bandwidth but the
// chain of histograms and cluster barriers: each pass counts in shared memory, adds
// its counts that are not zero to every CTA of the cluster, and needs one barrier;
// tokens of weight zero, often a large part, are counted by ballot instead of 32
// adds to one bin.
// Measured: 64 requests of 4096..32768 tokens 22 us (the masses and lists would
// stream in 0.6), one of 500009 tokens 36 us.
#include "tree_common.cuh"

namespace msa {
namespace {

constexpr int kEvBins = 2048;
constexpr int kEvMaxCluster = 16;
constexpr uint32_t kZeroKey = 0x80000000u;    // of a weight of 0
constexpr uint32_t kForcedKey = 0xffffffffu;  // above every weight's: always kept

__device__ __forceinline__ bool bad_pages(const msa_cache_view& c, int r, int nb, int nt) {
  bool bad = false;
#pragma unroll 4
  for (int b = threadIdx.x; b < nb; b += nt) {
    const int page = __ldg(c.block_table + (long long)r * c.bt_stride + b);
    bad |= page < 0 || page >= c.num_pages;
  }
  return __syncthreads_or(bad) != 0;
}

__device__ __forceinline__ void red_dsmem_add(uint32_t addr, int v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// grid: (cluster, requests), one cluster per request.  KEYS: keys a thread
// holds in registers (a CTA's share has at most its threads * KEYS tokens);
// kInShared: in shared memory; 0: none, they are read again in every pass.  Shares
// that fit registers: 22 us there, 30 in shared memory, 44 read again (64 requests
// of up to 32768 tokens); beyond: 36 in shared memory, 74 read again (500009 tokens).
constexpr int kInShared = -1;
constexpr int kSharedKeys = 44 * 1024;
template <int KEYS>
struct EvCfg {
  static constexpr int kThreads = KEYS > 0 ? 512 : 1024;
};

template <int KEYS>
__global__ void __launch_bounds__(EvCfg<KEYS>::kThreads, KEYS > 0 ? 2 : 1)
    evict_select_kernel(const EvictLaunch p) {
  constexpr int kEvThreads = EvCfg<KEYS>::kThreads, kEvWarps = kEvThreads / 32;
  constexpr int kBinsPer = kEvBins / kEvThreads;
  extern __shared__ uint32_t s_key[];  // KEYS == kInShared
  // counts of this CTA, and of the cluster, for each digit
  __shared__ int hist[2][kEvBins];
  __shared__ int total[3][kEvBins];
  __shared__ int s_scan[kEvWarps], s_digit, s_left, s_bad, s_count[2];
  __shared__ int s_wa[kEvWarps], s_we[kEvWarps];
  const int r = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, C = gridDim.x;
  const unsigned all = 0xffffffffu;
  const msa_cache_view& cv = p.cache;
  int32_t* keep = p.keep + (long long)r * p.budget;
  const int L = cv.lens[r];
  const bool malformed = L < 0 || (long long)L > (long long)kBlock * cv.bt_stride;
  for (int i = tid; i < 3 * kEvBins; i += kEvThreads) {
    (&total[0][0])[i] = 0;
    if (i < 2 * kEvBins) (&hist[0][0])[i] = 0;
  }
  if (tid == 0) s_bad = 0;
  // every CTA of the cluster runs and is cleared before another adds to it
  if (C > 1) joined_cluster_sync();
  else __syncthreads();

  // ---- this warp's run of tokens, [w0, w1): whole groups of 32
  const int per = malformed ? 0 : (L + C - 1) / C;
  const int sub = (per + kEvWarps * 32 - 1) / (kEvWarps * 32) * 32;
  const long long first = ((long long)rank * kEvWarps + warp) * sub;
  const int w0 = malformed ? 0 : (int)min((long long)L, first), w1 = malformed ? 0 : min(L, w0 + sub);
  const int lo = p.first, hi = L - p.recent;  // those that are ranked: [lo, hi)
  const int need = p.budget - p.first - p.recent;
  const int32_t* bt = cv.block_table + (long long)r * cv.bt_stride;
  bool bad = false;
  // The keys of tokens [t, t + 32 n) of the warp's run, n <= 16: the pages of
  // all of them at once, a lane each, then the weights at once (a bad page
  // reads page 0's, and is noted; there is none without pages).
  constexpr int most = KEYS > 0 ? (KEYS < 16 ? KEYS : 16) : KEYS == kInShared ? 16 : 1;
  auto load = [&](int t, int n, auto put) {
    if (cv.num_pages == 0) {  // no page: every token's is bad
      bad |= t < w1;
      for (int i = 0; i < n; ++i) put(i, 0u);
      return;
    }
    int page = 0;
    if (lane < n && t + 32 * lane < w1) {
      page = __ldg(bt + (t + 32 * lane) / kBlock);
      if (page < 0 || page >= cv.num_pages) {
        bad = true;
        page = 0;
      }
    }
    // (all loads unconditional and before the first use, so that they are in
    // flight together; beyond the run they read a slot of a page that is there)
    float m[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < most)
        m[i] = __ldg(p.mass + (long long)__shfl_sync(all, page, i) * kBlock + (t + 32 * i + lane) % kBlock);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int at = t + 32 * i + lane;
      if (i < most && i < n) put(i, at < lo || at >= hi ? kForcedKey : score_key(m[i]));
    }
  };
  uint32_t keys[KEYS > 0 ? KEYS : 1];
  uint32_t* run = s_key + warp * sub + lane;  // this lane's column of the warp's run
  if constexpr (KEYS > 0) {
    load(w0, KEYS, [&](int i, uint32_t k) { keys[i] = k; });
  } else {
    for (int t = w0; t < w1; t += 32 * most)
      load(t, min(most, (w1 - t + 31) / 32), [&](int i, uint32_t k) {
        if (KEYS == kInShared) run[t - w0 + 32 * i] = k;
      });
  }
  // f(t, key) for each of this thread's tokens, whole warps at a time
  auto each = [&](auto f) {
    if constexpr (KEYS > 0) {
#pragma unroll
      for (int i = 0; i < KEYS; ++i) {
        if (w0 + 32 * i >= w1) break;
        f(w0 + 32 * i + lane, keys[i]);
      }
    } else if constexpr (KEYS == kInShared) {
#pragma unroll 4
      for (int t = w0; t < w1; t += 32) f(t + lane, run[t - w0]);
    } else {
      for (int t = w0; t < w1; t += 32)
        load(t, 1, [&](int, uint32_t k) { f(t + lane, k); });
    }
  };
  if (__any_sync(all, bad) && lane == 0) {
    for (int c = 0; c < C; ++c) st_dsmem_s32(mapa_shared(smem_u32(&s_bad), c), 1);
  }

  uint32_t prefix = 0;
  int left = need;  // how many of the keys that match the prefix are kept
  const bool rank_them = !malformed && need > 0 && L > p.budget;
  // The cluster's counts are added up in every CTA, or, in a large cluster, in
  // the first alone, which tells the others the digit (16 adds for each of up
  // to 2048 counts took 10 K cycles in the second pass).
  const int holders = C <= 4 ? C : 1;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, up = pass == 1 ? 21 : 10;
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    if (rank_them) {
      if (pass == 2) {  // the first digit's counts again
        for (int i = tid; i < kEvBins; i += kEvThreads) hist[0][i] = 0;
        __syncthreads();
      }
      int zeros = 0;
      each([&](int t, uint32_t k) {
        const bool in = t < w1 && (pass == 0 ? k != kForcedKey : (k >> up) == (prefix >> up));
        if (pass > 0 && !__any_sync(all, in)) return;
        const bool zero = in && k == kZeroKey;
        zeros += __popc(__ballot_sync(all, zero));
        if (in && !zero) atomicAdd(&hist[pass & 1][(k >> shift) & mask], 1);
      });
      if (zeros && lane == 0) atomicAdd(&hist[pass & 1][(kZeroKey >> shift) & mask], zeros);
      __syncthreads();
      for (int i = tid; i < kEvBins; i += kEvThreads) {
        const int n = hist[pass & 1][i];
        if (n) {
          const uint32_t at = smem_u32(&total[pass][i]);
          for (int c = 0; c < holders; ++c) red_dsmem_add(mapa_shared(at, c), n);
        }
      }
    }
    if (C > 1) joined_cluster_sync();
    else __syncthreads();
    if (pass == 0) {
      // (every CTA's pages have been looked at)
      const uint32_t why = malformed ? MSA_DEV_MALFORMED : s_bad ? MSA_DEV_BAD_PAGE : 0u;
      const int kl = why ? 0 : min(L, p.budget);
      const int everyone = C * kEvThreads, me = rank * kEvThreads + tid;
      if (me == 0) {
        p.keep_len[r] = why ? -1 : kl;
        if (why) atomicOr(p.status, why);
      }
      for (int i = kl + me; i < p.budget; i += everyone) keep[i] = -1;
      if (!why && L <= p.budget)
        for (int i = me; i < L; i += everyone) keep[i] = i;
      if (why || L <= p.budget) {
        // no CTA leaves while another may still add to it
        if (C > 1) joined_cluster_sync();
        return;
      }
    }
    if (!rank_them) continue;
    // the digit, from the largest down
    if (rank < holders) {
    int n[kBinsPer], sum = 0;
#pragma unroll
    for (int k = 0; k < kBinsPer; ++k) {
      n[k] = total[pass][kEvBins - 1 - (kBinsPer * tid + k)];
      sum += n[k];
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(all, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    int at = inc - sum;
    for (int w = 0; w < warp; ++w) at += s_scan[w];
#pragma unroll
    for (int k = 0; k < kBinsPer; ++k) {
      if (at < left && at + n[k] >= left) {
        s_digit = kEvBins - 1 - (kBinsPer * tid + k);
        s_left = left - at;
      }
      at += n[k];
    }
    }
    if (holders < C) {
      if (rank == 0) {
        __syncthreads();
        if (tid < C) {
          st_dsmem_s32(mapa_shared(smem_u32(&s_digit), tid), s_digit);
          st_dsmem_s32(mapa_shared(smem_u32(&s_left), tid), s_left);
        }
      }
      joined_cluster_sync();
    } else {
      __syncthreads();
    }
    prefix |= (uint32_t)s_digit << shift;
    left = s_left;
  }

  // ---- ordered pass: count what each warp keeps and what equals the border,
  // then write behind the others
  const uint32_t border = need > 0 ? prefix : kForcedKey - 1;
  auto classify = [&](int t, uint32_t k, unsigned& ba, unsigned& be) {
    ba = __ballot_sync(all, t < w1 && k > border);
    be = __ballot_sync(all, t < w1 && k == border && need > 0);
  };
  int n_above = 0, n_eq = 0;
  each([&](int t, uint32_t k) {
    unsigned ba, be;
    classify(t, k, ba, be);
    n_above += __popc(ba);
    n_eq += __popc(be);
  });
  if (lane == 0) {
    s_wa[warp] = n_above;
    s_we[warp] = n_eq;
  }
  __syncthreads();
  int above = 0, eq = 0, above_cta = 0, eq_cta = 0;
#pragma unroll
  for (int w = 0; w < kEvWarps; ++w) {
    if (w < warp) {
      above += s_wa[w];
      eq += s_we[w];
    }
    above_cta += s_wa[w];
    eq_cta += s_we[w];
  }
  if (C > 1) {
    if (tid == 0) {
      s_count[0] = above_cta;
      s_count[1] = eq_cta;
    }
    joined_cluster_sync();
    // lane c reads CTA c's counts (C <= 16)
    int a = 0, e = 0;
    if (lane < rank) {
      a = ld_dsmem_s32(mapa_shared(smem_u32(&s_count[0]), lane));
      e = ld_dsmem_s32(mapa_shared(smem_u32(&s_count[1]), lane));
    }
    above += __reduce_add_sync(all, a);
    eq += __reduce_add_sync(all, e);
  }
  each([&](int t, uint32_t k) {
    unsigned ba, be;
    classify(t, k, ba, be);
    const unsigned below = (1u << lane) - 1u;
    const int eq_at = eq + __popc(be & below);
    // kept before this token: those above the border, and the first `left` equal to it
    if ((ba >> lane & 1u) || ((be >> lane & 1u) && eq_at < left))
      keep[above + __popc(ba & below) + min(eq_at, left)] = t;
    above += __popc(ba);
    eq += __popc(be);
  });
  // no CTA leaves while another reads its counts
  if (C > 1) joined_cluster_sync();
}

// ------------------------------------------------------------------- move

// In place and in parallel without a second buffer: the list ascends, so a
// token only moves down (destination i <= source).  Taken in chunks of
// consecutive destinations, a chunk's destinations lie below every later
// chunk's sources; so whoever reads a whole chunk before any of it is written
// never overwrites a token that is still to be read.  The pools are cut into
// columns of a token's row (of 256 bytes; with 128 the same within 2%), and a cluster
// of CTAs moves one column of one request, a barrier of the cluster between a chunk's
// reads and its writes: no two clusters touch the same bytes.  32 x 4096 tokens of K, V,
// index keys and masses, 203 MB read and written, take 52 us (3.9 TB/s, 58% of a copy's
// rate): a CTA has 16 KB of a chunk in flight and 16 KB of the next, and each of the 16
// chunks ends in a barrier.  A single request has four CTAs to each column and nothing
// else to fill the GPU with: 16384 tokens in 85 us, where their 25 MB would stream in 4.
constexpr int kCpThreads = 256;
constexpr int kCpColumn = 256;  // bytes of a column
constexpr int kCpParts = 4;     // CTAs of a cluster (long lists)
constexpr int kCpPages = 2048;  // page numbers held in shared memory

// Arrival at the cluster's barrier once this thread's loads have come back (x
// depends on all of them).  Nothing has to be published: the barrier only keeps
// writes behind reads, and a releasing arrival would wait for the last chunk's
// stores each time.
__device__ __forceinline__ void loads_done_cluster_sync(uint32_t x) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %0, 0x9e3779b9;\n\t@p nanosleep.u32 0;\n\t}" ::"r"(x)
      : "memory");
  __syncwarp();  // (a lane may have had nothing to load)
  asm volatile(
      "barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::
          : "memory");
}

__device__ __forceinline__ uint32_t fold(uint32_t x) { return x; }
__device__ __forceinline__ uint32_t fold(const uint4& v) { return v.x ^ v.y ^ v.z ^ v.w; }

// A thread takes V pieces of a token's column (piece sub + lanes * v), so that a
// token's address is worked out once per V.  The chunks are pipelined: while one
// is written, the next one's data and the list entries of the one after it are
// in flight (reads of later chunks may run ahead at will; only writes must wait
// for earlier reads).
template <typename T, int V, int S>
__device__ __forceinline__ void move_column(const CompactLaunch& p, int r, int base, int n,
                                            uint8_t* pool, int row, int col, int width,
                                            const int* s_page, int part, int parts) {
  const int lanes = width / ((int)sizeof(T) * V);  // threads per token
  const int sub = threadIdx.x % lanes, tok = threadIdx.x / lanes, toks = kCpThreads / lanes;
  const int32_t* bt = p.cache.block_table + (long long)r * p.cache.bt_stride;
  const int32_t* keep = p.keep + (long long)r * p.keep_stride;
  uint8_t* mine = pool + col + sub * (int)sizeof(T);
  const int step = lanes * (int)sizeof(T);
  auto at = [&](int pos) -> uint8_t* {
    const int b = pos / kBlock;
    const int page = b < kCpPages ? s_page[b] : __ldg(bt + b);
    return mine + ((long long)page * kBlock + pos % kBlock) * row;
  };
  const int chunk = toks * S * parts;
  const bool on = tok < toks;
  // list entries of a chunk; a token that stays where it is counts as absent
  auto entries = [&](int c0, int (&k)[S]) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int i = c0 + (s * parts + part) * toks + tok;
      k[s] = -1;
      if (on && i < n) {
        const int e = __ldg(keep + i);
        if (e != i) k[s] = e;
      }
    }
  };
  auto fetch = [&](const int (&k)[S], T (&v)[S][V]) {
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (k[s] >= 0) {
        const uint8_t* src = at(base + k[s]);
#pragma unroll
        for (int x = 0; x < V; ++x) v[s][x] = *reinterpret_cast<const T*>(src + x * step);
      }
  };
  int ka[S], kb[S], kc[S];
  T va[S][V] = {}, vb[S][V] = {};
  entries(0, ka);
  entries(chunk, kb);
  fetch(ka, va);
  for (int c0 = 0; c0 < n; c0 += chunk) {
    entries(c0 + 2 * chunk, kc);
    fetch(kb, vb);
    // every thread has read this chunk before any of it is overwritten
    if (parts > 1) {
      uint32_t x = 0;
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int y = 0; y < V; ++y) x ^= fold(va[s][y]);
      loads_done_cluster_sync(x);
    } else {
      __syncthreads();
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (ka[s] >= 0) {
        uint8_t* dst = at(base + c0 + (s * parts + part) * toks + tok);
#pragma unroll
        for (int x = 0; x < V; ++x) *reinterpret_cast<T*>(dst + x * step) = va[s][x];
      }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      ka[s] = kb[s];
      kb[s] = kc[s];
#pragma unroll
      for (int x = 0; x < V; ++x) va[s][x] = vb[s][x];
    }
  }
}

__global__ void __launch_bounds__(kCpThreads) kv_compact_kernel(const CompactLaunch p, int parts) {
  __shared__ int s_page[kCpPages], s_first;
  const int r = blockIdx.y, tid = threadIdx.x;
  const int n = p.keep_len[r];
  if (n <= 0) return;
  const int L = p.cache.lens[r], base = p.base ? p.base[r] : 0;
  uint32_t bad = 0;
  if (L < 0 || (long long)L > (long long)kBlock * p.cache.bt_stride) bad = MSA_DEV_MALFORMED;
  else if (n > p.keep_stride || base < 0 || base >= L) bad = MSA_DEV_BAD_TABLE;
  if (!bad) {
    const int32_t* keep = p.keep + (long long)r * p.keep_stride;
    bool list_bad = false;
#pragma unroll 8
    for (int i = tid; i < n; i += kCpThreads) {
      const int k = __ldg(keep + i), before = __ldg(keep + max(i - 1, 0));
      list_bad |= (i > 0 && k <= before) || k < 0 || k >= L - base;
    }
    if (__syncthreads_or(list_bad)) bad = MSA_DEV_BAD_TABLE;
  }
  if (!bad && bad_pages(p.cache, r, (L + kBlock - 1) / kBlock, kCpThreads)) bad = MSA_DEV_BAD_PAGE;
  if (!bad && p.cache.refs) {  // pages that tokens move into: from the first that does not stay on
    if (tid == 0) s_first = n;
    __syncthreads();
    int first = n;
    for (int i = tid; i < n && first == n; i += kCpThreads)
      if (__ldg(p.keep + (long long)r * p.keep_stride + i) != i) first = i;
    if (first < n) atomicMin(&s_first, first);
    __syncthreads();
    bool shared = false;
    if (s_first < n)
      for (int b = (base + s_first) / kBlock + tid; b <= (base + n - 1) / kBlock; b += kCpThreads)
        shared |= __ldg(p.cache.refs + __ldg(p.cache.block_table + (long long)r * p.cache.bt_stride + b)) > 1;
    if (__syncthreads_or(shared)) bad = MSA_DEV_BAD_TABLE;
  }
  if (bad) {
    if (tid == 0 && blockIdx.x == 0) atomicOr(p.status, bad);
    return;
  }
  for (int b = tid; b < min(kCpPages, (L + kBlock - 1) / kBlock); b += kCpThreads)
    s_page[b] = p.cache.block_table[(long long)r * p.cache.bt_stride + b];
  __syncthreads();
  // this CTA's column, and its part of it
  int x = blockIdx.x / parts;
  const int part = blockIdx.x % parts;
  for (int i = 0; i < kCompactPools; ++i) {
    const int row = p.pool[i].row;
    if (!p.pool[i].base) continue;
    const int cols = (row + kCpColumn - 1) / kCpColumn;
    if (x < cols) {
      const int col = x * kCpColumn, width = min(kCpColumn, row - col);
      uint8_t* pool = p.pool[i].base;
      if (row % 16 != 0) move_column<uint32_t, 1, 4>(p, r, base, n, pool, row, col, width, s_page, part, parts);
      else if (width % 64 == 0) move_column<uint4, 4, 1>(p, r, base, n, pool, row, col, width, s_page, part, parts);
      else move_column<uint4, 1, 4>(p, r, base, n, pool, row, col, width, s_page, part, parts);
      return;
    }
    x -= cols;
  }
}

}  // namespace

// CTAs per request: as many as leave each 2048 tokens or more while the grid
// fits the GPU at once; 16 (beyond the portable 8) where the device can place
// such a cluster.  64 requests of up to 32768 tokens: 30 us with one CTA each, 22
// with two and with four; one of 500009: 898 us with one, 459 with two, 240 with four,
// 129 with eight, 36 with sixteen (whose shares fit shared memory).
template <int KEYS>
cudaError_t launch_evict(const EvictLaunch& p, int C, long long share, cudaStream_t stream,
                         bool* placed) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, p.cache.num_reqs);
  constexpr int kEvThreads = EvCfg<KEYS>::kThreads;
  cfg.blockDim = dim3(kEvThreads);
  cfg.stream = stream;
  if (KEYS == kInShared) {
    // (a share, rounded up to 32 tokens a warp)
    cfg.dynamicSmemBytes = ((size_t)((share + kEvThreads - 1) / kEvThreads) * kEvThreads) * 4;
    const cudaError_t e = cudaFuncSetAttribute(
        evict_select_kernel<KEYS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedKeys * 4);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  *placed = true;
  if (C > 8) {
    const cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<KEYS>,
                                               cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    int fit = 0;
    if (cudaOccupancyMaxActiveClusters(&fit, evict_select_kernel<KEYS>, &cfg) != cudaSuccess || fit < 1) {
      cudaGetLastError();
      *placed = false;
      return cudaSuccess;
    }
  }
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<KEYS>, p);
}

cudaError_t launch_evict_select(const EvictLaunch& p, cudaStream_t stream) {
  const long long most = (long long)p.cache.bt_stride * kBlock;
  int C = 1;
  while (C < kEvMaxCluster && most >= 4096ll * C && (long long)p.cache.num_reqs * C <= device_sm_count())
    C *= 2;
  for (;; C /= 2) {
    const long long share = (most + C - 1) / C;
    bool placed;
    cudaError_t e;
    if (share <= 16 * EvCfg<16>::kThreads) e = launch_evict<16>(p, C, share, stream, &placed);
    else if (share <= kSharedKeys) e = launch_evict<kInShared>(p, C, share, stream, &placed);
    else e = launch_evict<0>(p, C, share, stream, &placed);
    if (placed) return e;
  }
}

cudaError_t launch_kv_compact(const CompactLaunch& p, cudaStream_t stream) {
  int cols = 0;
  for (int i = 0; i < kCompactPools; ++i)
    if (p.pool[i].base) cols += (p.pool[i].row + kCpColumn - 1) / kCpColumn;
  if (cols == 0) return cudaSuccess;
  // A short list (an accepted path) is a few chunks of 64 tokens at most, for one CTA:
  // 16 paths of up to 8 rows 3.8 us, with the cluster 5.6; 32 x 4096 tokens 78 us with
  // one CTA, 52 with four
  const int parts = p.keep_stride > 256 ? kCpParts : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cols * parts, p.cache.num_reqs);
  cfg.blockDim = dim3(kCpThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_compact_kernel, p, parts);
}

}  // namespace msa
