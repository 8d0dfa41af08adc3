// pages.cu -- the sharing of pages: the tables and reference counts of the requests
// that go on after a step (msa_page_fork), and the copies it asks for (msa_page_copy).
//
// The fork is one thread-block cluster, so that its passes meet at cluster barriers
// inside one launch: (1) refs copied, everything checked, children of each old request
// counted; (2) each old request's pages gain children - 1 holders (a partial last page
// only those children that do not grow), so that requests with one child touch no
// count, and those behind the request's tokens lose one; (3) of the requests that go on
// writing a partial page that nobody else holds, the lowest keeps it: every CTA finds
// these for itself in a table in shared memory, as it does the pages needed per request
// and their prefix sum, and counts the free pages of its slice; (4) tables, and the
// lowest free pages, found in order by a scan.  Counts are integers, so their order does
// not matter.
//
// 64 requests of 4 beams each, contexts to 8192, take 11.0 us (graph).  Their tables and
// counts are some 60 KB: it is bound by latency, the cluster barriers and the chains of
// dependent loads between them.
#include "prompt_common.cuh"

namespace msa {
namespace {

// (clusters of 8, 4, 2 and 1 CTAs: 10.9, 13.1, 16.9 and 22.7 us when it was chosen, before the wait
// for every CTA's start: the counts and the tables are shared out, the barriers stay)
constexpr int kFkThreads = 1024, kFkWarps = kFkThreads / 32, kFkCtas = 8;
constexpr unsigned kAll = 0xffffffffu;

constexpr int kFkRows = kMaxReqs / kFkThreads;  // new requests of a thread

// Shared memory behind the fixed part: children[R] (then place[N]), off[N + 1], and the
// table of pages that may be kept, keys[slots] and lowest[slots]
struct FkShared {
  int warp[2][kFkWarps];
  int flags[kFkCtas], free_pages[kFkCtas];
};
__host__ __device__ __forceinline__ int fk_slots(int n) {
  int s = 64;
  while (s < 2 * n) s *= 2;
  return s;
}
__host__ __device__ __forceinline__ int fk_longer(int r, int n) { return r > n ? r : n; }
size_t fk_bytes(int r, int n) { return sizeof(FkShared) + 4ull * (fk_longer(r, n) + n + 1 + 2 * fk_slots(n)); }

// A new request: its parent, tokens, growth, and the partial page it would write on (-1: none)
struct FkNew {
  int parent, n, grow, last;
  __device__ __forceinline__ int have() const { return (n + kBlock - 1) / kBlock; }
  __device__ __forceinline__ int full() const { return n / kBlock; }
  __device__ __forceinline__ int blocks() const { return (n + grow + kBlock - 1) / kBlock; }
};

// sum over the block of v; s_warp is free again after the next barrier
__device__ __forceinline__ int block_sum(int v, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = __reduce_add_sync(kAll, v);
  if (lane == 0) s_warp[warp] = v;
  __syncthreads();
  return __reduce_add_sync(kAll, s_warp[lane]);
}
// exclusive sum; the total in *sum
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  const int w = s_warp[lane];
  *sum = __reduce_add_sync(kAll, w);
  const int before = __reduce_add_sync(kAll, lane < warp ? w : 0);
  return before + x - v;
}

__global__ void __cluster_dims__(kFkCtas, 1, 1) __launch_bounds__(kFkThreads, 1)
    page_fork_kernel(const __grid_constant__ ForkLaunch p) {
  extern __shared__ __align__(16) uint8_t fk_smem[];
  cluster_started();  // (waited for behind part (1), whose loads take longer)
  FkShared& s = *reinterpret_cast<FkShared*>(fk_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x;
  const int R = p.from.num_reqs, N = p.to.num_reqs, P = p.from.num_pages, slots = fk_slots(N);
  int* children = reinterpret_cast<int*>(&s + 1);  // of an old request: all, and those that grow << 16
  // of a new request: its parent << 16 | whether it copies a page << 15 | blocks shared
  int* place = children;
  int* off = children + fk_longer(R, N);           // first new page of a new request; the total behind them
  int* keys = off + N + 1;
  int* lowest = keys + slots;
  int32_t* refs = p.to.refs;
  const int gwarp = rank * kFkWarps + warp;
  constexpr int kGridWarps = kFkCtas * kFkWarps;
  // pages of this CTA: [p0, p1), whole groups of four but for the last
  const int slice = ((P + kFkCtas - 1) / kFkCtas + 3) & ~3;
  const int p0 = (int)min((long long)P, (long long)rank * slice), p1 = (int)min((long long)P, (long long)p0 + slice);

  const auto copy_refs = [&]() {
    for (int i = p0 + 4 * tid; i < p1; i += 4 * kFkThreads) {
      if (i + 4 <= p1) {
        *reinterpret_cast<int4*>(refs + i) = __ldg(reinterpret_cast<const int4*>(p.refs + i));
      } else {
        for (int k = i; k < p1; ++k) refs[k] = __ldg(p.refs + k);
      }
    }
  };
  // a value of every CTA to every CTA's `to` array, and a cluster barrier
  const auto exchange = [&](int* to, int value) {
    if (tid < kFkCtas) st_dsmem_s32(mapa_shared(smem_u32(to + rank), tid), value);
    __syncthreads();
    joined_cluster_sync();
  };
  const auto refuse = [&](uint32_t bits) {
    for (int i = rank * kFkThreads + tid; i < N; i += kFkCtas * kFkThreads) {
      p.to.lens[i] = -1;
      if (p.to.blocks) p.to.blocks[i] = -1;
      p.to.copy_src[i] = p.to.copy_dst[i] = -1;
      p.to.copy_tokens[i] = 0;
    }
    if (rank == 0 && tid == 0) atomicOr(p.status, bits);
  };

  // ---- (1) checks and the children of each old request (every CTA counts them all)
  // Warps of the cluster to old requests: several a request when these are few.  The loads go out
  // in stages, each one's in flight together: lengths, parents; pages; their counts.
  const int wpo = max(1, kGridWarps / max(1, R)), wpn = max(1, kGridWarps / max(1, N));
  const int r0 = gwarp / wpo, b0 = (gwarp % wpo) * 32 + lane;
  const int n0 = r0 < R ? __ldg(p.from.lens + r0) : 0;
  const bool fits0 = n0 >= 0 && n0 <= (long long)kBlock * p.from.bt_stride;
  // pages that an old request holds: those of its tokens, and maybe more
  const int h0 = r0 < R && p.from.blocks ? __ldg(p.from.blocks + r0) : fits0 ? (n0 + kBlock - 1) / kBlock : 0;
  const auto held = [&](int r, int have) { return r == r0 ? h0 : p.from.blocks ? __ldg(p.from.blocks + r) : have; };
  FkNew x[kFkRows];
  uint32_t wrong = 0;
#pragma unroll
  for (int k = 0; k < kFkRows; ++k) {
    const int i = tid + k * kFkThreads;
    x[k].parent = -1;
    x[k].n = x[k].grow = 0;
    x[k].last = -1;
    if (i >= N) continue;
    x[k].parent = __ldg(p.parent + i);
    x[k].grow = p.grow ? __ldg(p.grow + i) : 0;
    if (x[k].parent < -1 || x[k].parent >= R || x[k].grow < 0) {
      wrong |= MSA_DEV_MALFORMED;
      x[k].parent = -1;
    }
  }
  for (int i = tid; i < R; i += kFkThreads) children[i] = 0;
  for (int i = tid; i < slots; i += kFkThreads) {
    keys[i] = -1;
    lowest[i] = N;
  }
  int page0 = 0;  // of block b0 of request r0
  if (fits0 && h0 <= p.from.bt_stride && b0 < h0) page0 = __ldg(p.from.block_table + (long long)r0 * p.from.bt_stride + b0);
  copy_refs();
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kFkRows; ++k) {
    if (tid + k * kFkThreads >= N) continue;
    if (x[k].parent >= 0) {
      x[k].n = __ldg(p.from.lens + x[k].parent);
      atomicAdd(&children[x[k].parent], 1 + (x[k].grow > 0 ? 1 << 16 : 0));
    }
    if (x[k].n < 0 || x[k].n > (long long)kBlock * p.from.bt_stride ||
        (long long)x[k].n + x[k].grow > (long long)kBlock * p.to.bt_stride) {
      wrong |= MSA_DEV_MALFORMED;
    } else if (x[k].grow > 0 && x[k].n % kBlock) {
      x[k].last = __ldg(p.from.block_table + (long long)x[k].parent * p.from.bt_stride + x[k].full());
    }
  }
  for (int r = r0; r < R; r += kGridWarps / wpo) {
    const int n = r == r0 ? n0 : __ldg(p.from.lens + r);
    if (n < 0 || n > (long long)kBlock * p.from.bt_stride) {
      wrong |= MSA_DEV_MALFORMED;
      continue;
    }
    const int have = (n + kBlock - 1) / kBlock, nb = held(r, have);
    if (nb < have || nb > p.from.bt_stride) {
      wrong |= MSA_DEV_MALFORMED;
      continue;
    }
    for (int b = b0; b < nb; b += 32 * wpo) {
      const int page = r == r0 && b == b0 ? page0 : __ldg(p.from.block_table + (long long)r * p.from.bt_stride + b);
      if (page < 0 || page >= P) wrong |= MSA_DEV_BAD_PAGE;
      else if (__ldg(p.refs + page) < 1) wrong |= MSA_DEV_BAD_TABLE;
    }
  }
  wrong = __reduce_or_sync(kAll, wrong);
  if (lane == 0) s.warp[0][warp] = (int)wrong;
  __syncthreads();
  wrong = __reduce_or_sync(kAll, (uint32_t)s.warp[0][lane]);
  cluster_wait_started();
  exchange(s.flags, (int)wrong);
  wrong = __reduce_or_sync(kAll, lane < kFkCtas ? (uint32_t)s.flags[lane] : 0u);
  if (wrong) {
    refuse(wrong);
    return;
  }

  // ---- (2) holders gained and lost
  for (int r = r0; r < R; r += kGridWarps / wpo) {
    const int all = children[r] & 0xffff, grown = children[r] >> 16;
    if (all == 1 && grown == 0 && !p.from.blocks) continue;
    const int n = r == r0 ? n0 : __ldg(p.from.lens + r), full = n / kBlock, have = (n + kBlock - 1) / kBlock;
    const int nb = held(r, have);
    for (int b = b0; b < nb; b += 32 * wpo) {
      const int d = (b < full ? all : b < have ? all - grown : 0) - 1;
      if (d == 0) continue;
      atomicAdd(refs + (r == r0 && b == b0 ? page0 : __ldg(p.from.block_table + (long long)r * p.from.bt_stride + b)), d);
    }
  }
  __syncthreads();
  joined_cluster_sync();

  // ---- (3) who keeps a partial page: the lowest of those that go on writing one without holders
  const auto slot_of = [&](int page) { return (int)(((uint32_t)page * 2654435761u) >> 8) & (slots - 1); };
  bool wants[kFkRows];
#pragma unroll
  for (int k = 0; k < kFkRows; ++k) {
    const int page = x[k].last;
    wants[k] = page >= 0 && __ldcg(refs + page) <= 0;
    if (!wants[k]) continue;
    int at = slot_of(page);
    while (true) {  // (half the table stays empty)
      const int was = atomicCAS(&keys[at], -1, page);
      if (was == -1 || was == page) break;
      at = (at + 1) & (slots - 1);
    }
    atomicMin(&lowest[at], tid + k * kFkThreads);
  }
  __syncthreads();
  // pages needed and their prefix sum (every CTA for all), free pages of the slice
  int total = 0, kept_here = 0;
#pragma unroll
  for (int k = 0; k < kFkRows; ++k) {
    if (k * kFkThreads >= N) break;
    const int i = tid + k * kFkThreads;
    int need = 0;
    if (i < N) {
      const int page = x[k].last;
      bool keeps = wants[k];
      if (keeps) {
        int at = slot_of(page);
        while (keys[at] != page) at = (at + 1) & (slots - 1);
        keeps = lowest[at] == i;
      }
      wants[k] = keeps;
      const bool copy = page >= 0 && !keeps;
      if (keeps && page >= p0 && page < p1 && __ldcg(refs + page) == 0) ++kept_here;
      need = x[k].blocks() - x[k].have() + (copy ? 1 : 0);
      place[i] = max(x[k].parent, 0) << 16 | (copy ? 1 << 15 | x[k].full() : x[k].have());
      if (i % kFkCtas == rank) {
        p.to.lens[i] = x[k].n;
        if (p.to.blocks) p.to.blocks[i] = x[k].blocks();
        p.to.copy_src[i] = copy ? page : -1;
        p.to.copy_tokens[i] = copy ? x[k].n % kBlock : 0;
        if (!copy) p.to.copy_dst[i] = -1;
      }
    }
    int sum;
    const int before = block_scan(need, s.warp[k & 1], &sum);
    if (i < N) off[i] = total + before;
    total += sum;
  }
  if (tid == 0) off[N] = total;
  int zeros = -kept_here;
  for (int i = p0 + tid; i < p1; i += kFkThreads) zeros += __ldcg(refs + i) == 0;
  __syncthreads();
  exchange(s.free_pages, block_sum(zeros, s.warp[0]));
  const int free_of = lane < kFkCtas ? s.free_pages[lane] : 0;
  int at = __reduce_add_sync(kAll, lane < rank ? free_of : 0);
  if ((int)__reduce_add_sync(kAll, free_of) < total) {
    copy_refs();
    refuse(MSA_DEV_NO_PAGES);
    return;
  }

  // ---- (4) tables
#pragma unroll
  for (int k = 0; k < kFkRows; ++k)
    if (wants[k] && x[k].last >= p0 && x[k].last < p1) refs[x[k].last] = 1;
  __syncthreads();  // (before the slice's free pages are looked for)
  for (int i = gwarp / wpn; i < N; i += kGridWarps / wpn) {
    const int parent = place[i] >> 16, shared = place[i] & 0x7fff;
    for (int b = (gwarp % wpn) * 32 + lane; b < shared; b += 32 * wpn)
      p.to.block_table[(long long)i * p.to.bt_stride + b] =
          __ldg(p.from.block_table + (long long)parent * p.from.bt_stride + b);
  }
  for (int i0 = p0, turn = 0; i0 < p1 && at < total; i0 += kFkThreads, turn ^= 1) {
    const int page = i0 + tid;
    const bool free_page = page < p1 && __ldcg(refs + page) == 0;
    int sum;
    const int k = at + block_scan(free_page ? 1 : 0, s.warp[turn], &sum);
    if (free_page && k < total) {
      int lo = 0, hi = N - 1;  // the last request whose first new page is k or before
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= k) lo = mid; else hi = mid - 1;
      }
      const int j = k - off[lo];
      p.to.block_table[(long long)lo * p.to.bt_stride + (place[lo] & 0x7fff) + j] = page;
      if (j == 0 && (place[lo] >> 15 & 1)) p.to.copy_dst[lo] = page;
      refs[page] = 1;
    }
    at += sum;
  }
}

// ------------------------------------------------------------------ copies

// 16 bytes a thread and load.  120 pages in 40 layers of e4m3 with scales, 245 MB both ways, in
// one launch: 40.9 us (6.0 TB/s, 88 % of the copy rate: bound by memory).  In two launches it took
// 43.4, with 256 and 512 threads 44.8 and 67.7, with 2 loads of a thread in flight in place of 4
// 46.3, with 8 60.2 (the last four at two launches, 2 and 8 loads at 256 threads).  96 pages of
// one layer: 3.2 us (3.7 with 2 loads), a launch and two dependent loads.
constexpr int kCpThreads = 128;

// One array's part of one page per CTA
__global__ void __launch_bounds__(kCpThreads) page_copy_kernel(const __grid_constant__ CopyLaunch p) {
  const int i = blockIdx.x / p.num_pools;
  const CopyPool pool = p.pool[blockIdx.x % p.num_pools];
  const int tokens = __ldg(p.tokens + i), src = __ldg(p.src + i), dst = __ldg(p.dst + i);
  if (tokens <= 0) return;
  uint32_t wrong = 0;
  if (tokens > kBlock) wrong |= MSA_DEV_MALFORMED;
  if (src < 0 || src >= p.num_pages || dst < 0 || dst >= p.num_pages) wrong |= MSA_DEV_BAD_PAGE;
  if (wrong) {
    if (threadIdx.x == 0) atomicOr(p.status, wrong);
    return;
  }
  const long long page = (long long)kBlock * pool.row;
  const uint8_t* a = pool.base + src * page;
  uint8_t* b = pool.base + dst * page;
  const int bytes = tokens * pool.row, whole = bytes / 16;
  constexpr int kLoads = 4;
  for (int j = threadIdx.x; j < whole; j += kLoads * kCpThreads) {
    uint4 v[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
      if (j + k * kCpThreads < whole) v[k] = __ldcs(reinterpret_cast<const uint4*>(a) + j + k * kCpThreads);
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
      if (j + k * kCpThreads < whole) reinterpret_cast<uint4*>(b)[j + k * kCpThreads] = v[k];
  }
  // (rows of scales and weights are multiples of 4 bytes)
  const int rest = (bytes - 16 * whole) / 4;
  if ((int)threadIdx.x < rest)
    reinterpret_cast<uint32_t*>(b + 16 * whole)[threadIdx.x] =
        reinterpret_cast<const uint32_t*>(a + 16 * whole)[threadIdx.x];
}

}  // namespace

cudaError_t launch_page_fork(const ForkLaunch& p, cudaStream_t stream) {
  const size_t bytes = fk_bytes(p.from.num_reqs, p.to.num_reqs);
  if (bytes > 48 * 1024) {
    // (what any call may need: the limit is the process's, and another thread's call sets it too)
    const cudaError_t e = cudaFuncSetAttribute(page_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)fk_bytes(kMaxReqs, kMaxReqs));
    if (e != cudaSuccess) return e;
  }
  page_fork_kernel<<<kFkCtas, kFkThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_page_copy(const CopyLaunch& p, cudaStream_t stream) {
  page_copy_kernel<<<p.num_copies * p.num_pools, kCpThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace msa
