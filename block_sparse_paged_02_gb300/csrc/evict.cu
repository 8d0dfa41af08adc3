// evict.cu -- eviction from the cache: the tokens a request keeps under a
// budget, and the in-place move of kept tokens (which also commits the
// accepted path of a draft tree).
//
// Selection.  Orderable 32-bit keys of the masses (NaN lowest, -0 = +0), a
// radix selection of the need-th largest by 8-bit digits, then one ordered
// pass that keeps keys above it and the first of those equal to it.
#include "tree_common.cuh"

namespace msa {
namespace {

constexpr int kEvThreads = 1024;

__device__ __forceinline__ bool bad_pages(const msa_cache_view& c, int r, int nb, int nt) {
  bool bad = false;
  for (int b = threadIdx.x; b < nb; b += nt) {
    const int page = c.block_table[(long long)r * c.bt_stride + b];
    bad |= page < 0 || page >= c.num_pages;
  }
  return __syncthreads_or(bad) != 0;
}

__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(const EvictLaunch p) {
  __shared__ int hist[256];
  __shared__ int s_digit, s_above;
  __shared__ int s_keep[32], s_eq[32];
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const msa_cache_view& cv = p.cache;
  int32_t* keep = p.keep + (long long)r * p.budget;
  const int L = cv.lens[r];
  uint32_t bad = 0;
  if (L < 0 || (long long)L > (long long)kBlock * cv.bt_stride) bad = MSA_DEV_MALFORMED;
  else if (bad_pages(cv, r, (L + kBlock - 1) / kBlock, kEvThreads)) bad = MSA_DEV_BAD_PAGE;
  const int kl = bad ? 0 : min(L, p.budget);
  if (tid == 0) {
    p.keep_len[r] = bad ? -1 : kl;
    if (bad) atomicOr(p.status, bad);
  }
  for (int i = kl + tid; i < p.budget; i += kEvThreads) keep[i] = -1;
  if (bad) return;
  if (L <= p.budget) {
    for (int i = tid; i < L; i += kEvThreads) keep[i] = i;
    return;
  }
  const int lo = p.first, hi = L - p.recent;  // the others: [lo, hi)
  const int need = p.budget - p.first - p.recent;
  const int32_t* bt = cv.block_table + (long long)r * cv.bt_stride;
  auto key_at = [&](int t) { return score_key(p.mass[(long long)bt[t / kBlock] * kBlock + t % kBlock]); };
  uint32_t prefix = 0;
  int left = need;  // how many of the keys that match the prefix are kept
  for (int shift = 24; need > 0 && shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kEvThreads) hist[i] = 0;
    __syncthreads();
    for (int t = lo + tid; t < hi; t += kEvThreads) {
      const uint32_t k = key_at(t);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int n = 0, d = 255;
      for (; d > 0 && n + hist[d] < left; --d) n += hist[d];
      s_digit = d;
      s_above = n;
    }
    __syncthreads();
    prefix |= (uint32_t)s_digit << shift;
    left -= s_above;
    __syncthreads();
  }
  // ordered pass
  int n_keep = 0, n_eq = 0;
  for (int base = 0; base < L; base += kEvThreads) {
    const int t = base + tid;
    bool above = false, eq = false;
    if (t < L) {
      if (t < lo || t >= hi) above = true;
      else if (need > 0) {
        const uint32_t k = key_at(t);
        above = k > prefix;
        eq = k == prefix;
      }
    }
    const unsigned be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) s_eq[warp] = __popc(be);
    __syncthreads();
    int eq_before = n_eq, eq_all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) eq_before += s_eq[w];
      eq_all += s_eq[w];
    }
    eq_before += __popc(be & ((1u << lane) - 1u));
    const bool take = above || (eq && eq_before < left);
    const unsigned bk = __ballot_sync(0xffffffffu, take);
    if (lane == 0) s_keep[warp] = __popc(bk);
    __syncthreads();
    int before = n_keep, all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += s_keep[w];
      all += s_keep[w];
    }
    if (take) keep[before + __popc(bk & ((1u << lane) - 1u))] = t;
    n_keep += all;
    n_eq += eq_all;
  }
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
constexpr int kCpColumn = 64;  // bytes of a column
constexpr int kCpSteps = 8;    // tokens per thread and chunk

template <typename T>
__device__ __forceinline__ void move_column(const CompactLaunch& p, int r, int base, int n,
                                            uint8_t* pool, int row, int col, int width) {
  const int per = width / (int)sizeof(T);  // threads per token
  const int sub = threadIdx.x % per, tok = threadIdx.x / per, toks = kCpThreads / per;
  const bool on = tok < toks;
  const int32_t* bt = p.cache.block_table + (long long)r * p.cache.bt_stride;
  const int32_t* keep = p.keep + (long long)r * p.keep_stride;
  auto at = [&](int pos) -> T* {
    return reinterpret_cast<T*>(pool + ((long long)bt[pos / kBlock] * kBlock + pos % kBlock) * row + col) + sub;
  };
  for (int c0 = 0; c0 < n; c0 += toks * kCpSteps) {
    T v[kCpSteps];
    bool moves[kCpSteps];
#pragma unroll
    for (int s = 0; s < kCpSteps; ++s) {
      const int i = c0 + s * toks + tok;
      moves[s] = false;
      if (on && i < n) {
        const int k = keep[i];
        moves[s] = k != i;
        if (moves[s]) v[s] = *at(base + k);
      }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kCpSteps; ++s)
      if (moves[s]) *at(base + c0 + s * toks + tok) = v[s];
  }
}

__global__ void __launch_bounds__(kCpThreads) kv_compact_kernel(const CompactLaunch p) {
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
  // this CTA's column
  int x = blockIdx.x;
  for (int i = 0; i < kCompactPools; ++i) {
    const int row = p.pool[i].row;
    if (!p.pool[i].base) continue;
    const int cols = (row + kCpColumn - 1) / kCpColumn;
    if (x < cols) {
      const int col = x * kCpColumn, width = min(kCpColumn, row - col);
      if (row % 16 == 0) move_column<uint4>(p, r, base, n, p.pool[i].base, row, col, width);
      else move_column<uint32_t>(p, r, base, n, p.pool[i].base, row, col, width);
      return;
    }
    x -= cols;
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictLaunch& p, cudaStream_t stream) {
  evict_select_kernel<<<p.cache.num_reqs, kEvThreads, 0, stream>>>(p);
  return cudaGetLastError();
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
