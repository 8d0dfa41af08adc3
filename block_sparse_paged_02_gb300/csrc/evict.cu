// evict.cu -- eviction from the cache: the tokens a request keeps under a
// budget, and the in-place move of kept tokens (which also commits the
// accepted path of a draft tree).
//
// Selection.  Orderable 32-bit keys of the masses (NaN lowest, -0 = +0), a
// radix selection of the need-th largest by digits of 11, 11 and 10 bits, then
// an ordered pass that keeps keys above it and the first of those equal to it.
// One thread-block cluster per request: each CTA reads its share of the tokens
// once, keeps the keys in shared memory for the later passes, and the cluster
// adds up its histograms through distributed shared memory.  The masses are
// 4 bytes a token, so the pass over memory is short and the time is the chain
// of cluster barriers and histogram scans, not bandwidth.
#include "tree_common.cuh"

namespace msa {
namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvBins = 2048;
constexpr int kEvKeys = 52 * 1024;  // keys that a CTA's shared memory holds
constexpr int kEvMaxCluster = 16;

__device__ __forceinline__ bool bad_pages(const msa_cache_view& c, int r, int nb, int nt) {
  bool bad = false;
  for (int b = threadIdx.x; b < nb; b += nt) {
    const int page = c.block_table[(long long)r * c.bt_stride + b];
    bad |= page < 0 || page >= c.num_pages;
  }
  return __syncthreads_or(bad) != 0;
}

// inclusive sum over the CTA's threads; *total: the sum over all.  scratch: 33 ints
__device__ __forceinline__ int cta_scan(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int x = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += n;
    }
    scratch[lane] = x;
  }
  __syncthreads();
  *total = scratch[31];
  const int before = warp ? scratch[warp - 1] : 0;
  __syncthreads();
  return before + v;
}

// grid: (cluster, requests), one cluster per request
__global__ void __launch_bounds__(kEvThreads, 1) evict_select_kernel(const EvictLaunch p, int cap) {
  extern __shared__ uint32_t s_key[];  // [cap]
  __shared__ int hist[kEvBins];
  __shared__ int s_scan[33];
  __shared__ int s_digit, s_left, s_above, s_eq;
  __shared__ int s_wa[32], s_we[32];
  const int r = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, C = gridDim.x;
  const msa_cache_view& cv = p.cache;
  int32_t* keep = p.keep + (long long)r * p.budget;
  const int L = cv.lens[r];
  uint32_t bad = 0;
  if (L < 0 || (long long)L > (long long)kBlock * cv.bt_stride) bad = MSA_DEV_MALFORMED;
  else if (bad_pages(cv, r, (L + kBlock - 1) / kBlock, kEvThreads)) bad = MSA_DEV_BAD_PAGE;
  const int kl = bad ? 0 : min(L, p.budget);
  const int all = C * kEvThreads, me = rank * kEvThreads + tid;
  if (me == 0) {
    p.keep_len[r] = bad ? -1 : kl;
    if (bad) atomicOr(p.status, bad);
  }
  for (int i = kl + me; i < p.budget; i += all) keep[i] = -1;
  if (bad) return;
  if (L <= p.budget) {
    for (int i = me; i < L; i += all) keep[i] = i;
    return;
  }
  // this CTA's tokens: whole blocks, [t0, t1)
  const int nb = (L + kBlock - 1) / kBlock;
  const int per = (nb + C - 1) / C * kBlock;
  const int t0 = min(L, rank * per), t1 = min(L, t0 + per);
  const int lo = p.first, hi = L - p.recent;  // those that are ranked: [lo, hi)
  const int need = p.budget - p.first - p.recent;
  const int32_t* bt = cv.block_table + (long long)r * cv.bt_stride;
  const bool held = per <= cap;
  auto load_key = [&](int t) {
    return score_key(__ldg(p.mass + (long long)__ldg(bt + t / kBlock) * kBlock + t % kBlock));
  };
  auto key_at = [&](int t) { return held ? s_key[t - t0] : load_key(t); };
  if (held && need > 0) {
#pragma unroll 4
    for (int t = t0 + tid; t < t1; t += kEvThreads) s_key[t - t0] = load_key(t);
  }
  const int a = max(lo, t0), b = min(hi, t1);
  uint32_t prefix = 0;
  int left = need;  // how many of the keys that match the prefix are kept
  if (need > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      for (int i = tid; i < kEvBins; i += kEvThreads) hist[i] = 0;
      __syncthreads();
      for (int t = a + tid; t < b; t += kEvThreads) {
        const uint32_t k = key_at(t);
        const int up = pass == 1 ? 21 : 10;  // the digits already fixed lie above
        if (pass == 0 || (k >> up) == (prefix >> up)) atomicAdd(&hist[(k >> shift) & mask], 1);
      }
      if (C > 1) cluster_sync();
      else __syncthreads();
      // the cluster's counts of two bins per thread, largest digit first
      int n[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int bin = kEvBins - 1 - (2 * tid + k);
        if (C > 1) {
          const uint32_t at = smem_u32(&hist[bin]);
          for (int c = 0; c < C; ++c) n[k] += ld_dsmem_s32(mapa_shared(at, c));
        } else {
          n[k] = hist[bin];
        }
      }
      int total;
      const int upto = cta_scan(n[0] + n[1], s_scan, &total);
      const int before = upto - n[0] - n[1];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int x = k ? before + n[0] : before;
        if (x < left && x + n[k] >= left) {
          s_digit = kEvBins - 1 - (2 * tid + k);
          s_left = left - x;
        }
      }
      __syncthreads();
      prefix |= (uint32_t)s_digit << shift;
      left = s_left;
      // no CTA clears its counts while another still reads them
      if (C > 1) cluster_sync();
      else __syncthreads();
    }
  }
  // ordered pass: a warp takes a contiguous part of the CTA's tokens, counts
  // what it keeps and what equals the border, then writes behind the others
  const int sub = (per / 32 + 31) / 32 * 32;
  const int w0 = min(t1, t0 + warp * sub), w1 = min(t1, w0 + sub);
  auto classify = [&](int t, bool& above, bool& eq) {
    above = eq = false;
    if (t < w1) {
      if (t < lo || t >= hi) above = true;
      else if (need > 0) {
        const uint32_t k = key_at(t);
        above = k > prefix;
        eq = k == prefix;
      }
    }
  };
  int n_above = 0, n_eq = 0;
  for (int t = w0; t < w1; t += 32) {
    bool above, eq;
    classify(t + lane, above, eq);
    n_above += __popc(__ballot_sync(0xffffffffu, above));
    n_eq += __popc(__ballot_sync(0xffffffffu, eq));
  }
  if (lane == 0) {
    s_wa[warp] = n_above;
    s_we[warp] = n_eq;
  }
  __syncthreads();
  int above_before = 0, eq_before = 0, above_cta = 0, eq_cta = 0;
  for (int w = 0; w < 32; ++w) {
    if (w < warp) {
      above_before += s_wa[w];
      eq_before += s_we[w];
    }
    above_cta += s_wa[w];
    eq_cta += s_we[w];
  }
  if (C > 1) {
    if (tid == 0) {
      s_above = above_cta;
      s_eq = eq_cta;
    }
    cluster_sync();
    for (int c = 0; c < rank; ++c) {
      above_before += ld_dsmem_s32(mapa_shared(smem_u32(&s_above), c));
      eq_before += ld_dsmem_s32(mapa_shared(smem_u32(&s_eq), c));
    }
  }
  for (int t = w0; t < w1; t += 32) {
    bool above, eq;
    classify(t + lane, above, eq);
    const unsigned be = __ballot_sync(0xffffffffu, eq), ba = __ballot_sync(0xffffffffu, above);
    const unsigned below = (1u << lane) - 1u;
    const int eq_at = eq_before + __popc(be & below);
    // kept before this token: those above the border, and the first `left` equal to it
    if (above || (eq && eq_at < left))
      keep[above_before + __popc(ba & below) + min(eq_at, left)] = t + lane;
    above_before += __popc(ba);
    eq_before += __popc(be);
  }
  // no CTA leaves while another reads its counts
  if (C > 1) cluster_sync();
}

// ------------------------------------------------------------------- move

// In place and in parallel without a second buffer: the list ascends, so a
// token only moves down (destination i <= source).  Taken in chunks of
// consecutive destinations, a chunk's destinations lie below every later
// chunk's sources; so a CTA that reads a whole chunk before it writes it
// never overwrites a token that it still has to read.  The pools are cut into
// columns of a token's row, and each CTA moves one column of one request:
// no two CTAs touch the same bytes.
constexpr int kCpThreads = 256;
constexpr int kCpColumn = 64;   // bytes of a column
constexpr int kCpSteps = 4;     // tokens per thread and chunk
constexpr int kCpPages = 2048;  // page numbers held in shared memory

// The chunks are pipelined: while one is written, the next one's data and the
// list entries of the one after it are in flight (reads of later chunks may
// run ahead at will; only writes must wait for earlier reads).
template <typename T>
__device__ __forceinline__ void move_column(const CompactLaunch& p, int r, int base, int n,
                                            uint8_t* pool, int row, int col, int width,
                                            const int* s_page) {
  const int per = width / (int)sizeof(T);  // threads per token
  const int sub = threadIdx.x % per, tok = threadIdx.x / per, toks = kCpThreads / per;
  const int32_t* bt = p.cache.block_table + (long long)r * p.cache.bt_stride;
  const int32_t* keep = p.keep + (long long)r * p.keep_stride;
  auto at = [&](int pos) -> T* {
    const int b = pos / kBlock;
    const long long page = b < kCpPages ? s_page[b] : __ldg(bt + b);
    return reinterpret_cast<T*>(pool + (page * kBlock + pos % kBlock) * row + col) + sub;
  };
  const int chunk = toks * kCpSteps;
  const bool on = tok < toks;
  // list entries of a chunk; a token that stays where it is counts as absent
  auto entries = [&](int c0, int (&k)[kCpSteps]) {
#pragma unroll
    for (int s = 0; s < kCpSteps; ++s) {
      const int i = c0 + s * toks + tok;
      k[s] = -1;
      if (on && i < n) {
        const int e = __ldg(keep + i);
        if (e != i) k[s] = e;
      }
    }
  };
  auto fetch = [&](const int (&k)[kCpSteps], T (&v)[kCpSteps]) {
#pragma unroll
    for (int s = 0; s < kCpSteps; ++s)
      if (k[s] >= 0) v[s] = *at(base + k[s]);
  };
  auto store = [&](int c0, const int (&k)[kCpSteps], const T (&v)[kCpSteps]) {
#pragma unroll
    for (int s = 0; s < kCpSteps; ++s)
      if (k[s] >= 0) *at(base + c0 + s * toks + tok) = v[s];
  };
  int ka[kCpSteps], kb[kCpSteps], kc[kCpSteps];
  T va[kCpSteps], vb[kCpSteps];
  entries(0, ka);
  entries(chunk, kb);
  fetch(ka, va);
  for (int c0 = 0; c0 < n; c0 += chunk) {
    entries(c0 + 2 * chunk, kc);
    fetch(kb, vb);
    // every thread has read this chunk (its data is needed below) before any
    // of it is overwritten
    __syncthreads();
    store(c0, ka, va);
#pragma unroll
    for (int s = 0; s < kCpSteps; ++s) {
      ka[s] = kb[s];
      kb[s] = kc[s];
      va[s] = vb[s];
    }
  }
}

__global__ void __launch_bounds__(kCpThreads) kv_compact_kernel(const CompactLaunch p) {
  __shared__ int s_page[kCpPages];
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
    for (int i = tid; i < n; i += kCpThreads) {
      const int k = keep[i], before = i > 0 ? keep[i - 1] : -1;
      list_bad |= k <= before || k < 0 || k >= L - base;
    }
    if (__syncthreads_or(list_bad)) bad = MSA_DEV_BAD_TABLE;
  }
  if (!bad && bad_pages(p.cache, r, (L + kBlock - 1) / kBlock, kCpThreads)) bad = MSA_DEV_BAD_PAGE;
  if (bad) {
    if (tid == 0 && blockIdx.x == 0) atomicOr(p.status, bad);
    return;
  }
  for (int b = tid; b < min(kCpPages, (L + kBlock - 1) / kBlock); b += kCpThreads)
    s_page[b] = p.cache.block_table[(long long)r * p.cache.bt_stride + b];
  __syncthreads();
  // this CTA's column
  int x = blockIdx.x;
  for (int i = 0; i < kCompactPools; ++i) {
    const int row = p.pool[i].row;
    if (!p.pool[i].base) continue;
    const int cols = (row + kCpColumn - 1) / kCpColumn;
    if (x < cols) {
      const int col = x * kCpColumn, width = min(kCpColumn, row - col);
      if (row % 16 == 0) move_column<uint4>(p, r, base, n, p.pool[i].base, row, col, width, s_page);
      else move_column<uint32_t>(p, r, base, n, p.pool[i].base, row, col, width, s_page);
      return;
    }
    x -= cols;
  }
}

}  // namespace

// CTAs per request: enough that one holds about 4096 tokens, while the grid
// fits the GPU about twice; 16 (beyond the portable 8) where the device can
// place such a cluster.
cudaError_t launch_evict_select(const EvictLaunch& p, cudaStream_t stream) {
  const long long most = (long long)p.cache.bt_stride * kBlock;
  const int sms = device_sm_count();
  int C = 1;
  while (C < kEvMaxCluster && most > 4096ll * C && (long long)p.cache.num_reqs * C * 2 <= 2ll * sms) C *= 2;
  for (;; C /= 2) {
    const long long per = (most / kBlock + C - 1) / C * kBlock;
    const int cap = (int)min(per, (long long)kEvKeys);
    const size_t bytes = (size_t)cap * 4;
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kEvKeys * 4);
    if (e != cudaSuccess) return e;
    if (C > 8) {
      e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C, p.cache.num_reqs);
    cfg.blockDim = dim3(kEvThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (C > 8) {
      int fit = 0;
      if (cudaOccupancyMaxActiveClusters(&fit, evict_select_kernel, &cfg) != cudaSuccess || fit < 1) {
        cudaGetLastError();
        continue;
      }
    }
    return cudaLaunchKernelEx(&cfg, evict_select_kernel, p, cap);
  }
}

cudaError_t launch_kv_compact(const CompactLaunch& p, cudaStream_t stream) {
  int cols = 0;
  for (int i = 0; i < kCompactPools; ++i)
    if (p.pool[i].base) cols += (p.pool[i].row + kCpColumn - 1) / kCpColumn;
  if (cols == 0) return cudaSuccess;
  kv_compact_kernel<<<dim3(cols, p.cache.num_reqs), kCpThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace msa
