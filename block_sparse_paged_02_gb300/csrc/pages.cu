// pages.cu -- the sharing of pages: the tables and reference counts of the requests
// that go on after a step (msa_page_fork), and the copies it asks for (msa_page_copy).
//
// The fork is one thread-block cluster, so that its passes meet at cluster barriers
// inside one launch: (1) refs copied, everything checked, children of each old request
// counted; (2) each old request's pages gain children - 1 holders (a partial last page
// only those children that do not grow), so that requests with one child touch no
// count; (3) of the requests that go on writing a partial page that nobody else holds,
// the lowest keeps it (an atomic minimum of a negative number in its count); (4) pages
// needed per request and their prefix sum, free pages per CTA; (5) the lowest free
// pages found in order by ballots and written to the tables.  Counts are integers, so
// their order does not matter.
#include "prompt_common.cuh"

namespace msa {
namespace {

constexpr int kFkThreads = 1024, kFkWarps = kFkThreads / 32, kFkCtas = 8;
constexpr unsigned kAll = 0xffffffffu;

struct FkShared {
  int children[kMaxReqs];   // of an old request: all, and those that grow << 16
  int off[kMaxReqs + 1];    // first new page of a new request; the total behind them
  int warp[kFkWarps];
  int flags[kFkCtas], free_pages[kFkCtas];
};

// A new request: its tokens, blocks held, full ones, the page it would write on with
// (-1: none), blocks with its growth; wrong: status bits
struct FkNew {
  int n, have, full, last, blocks;
  bool partial;  // its last page is partial and it grows
  uint32_t wrong;
};

__device__ __forceinline__ FkNew fk_new(const ForkLaunch& p, int i) {
  FkNew x;
  x.n = x.have = x.full = x.blocks = 0;
  x.last = -1;
  x.partial = false;
  x.wrong = 0;
  const int parent = __ldg(p.parent + i), grow = p.grow ? __ldg(p.grow + i) : 0;
  if (parent < -1 || parent >= p.from.num_reqs || grow < 0) {
    x.wrong = MSA_DEV_MALFORMED;
    return x;
  }
  if (parent >= 0) x.n = __ldg(p.from.lens + parent);
  const long long most = (long long)x.n + grow;
  if (x.n < 0 || x.n > (long long)kBlock * p.from.bt_stride || most > (long long)kBlock * p.to.bt_stride) {
    x.wrong = MSA_DEV_MALFORMED;
    return x;
  }
  x.have = (x.n + kBlock - 1) / kBlock;
  x.full = x.n / kBlock;
  x.blocks = (int)((most + kBlock - 1) / kBlock);
  x.partial = grow > 0 && x.have > x.full;
  if (x.partial) x.last = __ldg(p.from.block_table + (long long)parent * p.from.bt_stride + x.full);
  return x;
}

// exclusive sum over the block; the total in *sum
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kFkWarps; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  *sum = all;
  return before + x - v;
}

__global__ void __cluster_dims__(kFkCtas, 1, 1) __launch_bounds__(kFkThreads, 1)
    page_fork_kernel(const __grid_constant__ ForkLaunch p) {
  __shared__ FkShared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x;
  const int R = p.from.num_reqs, N = p.to.num_reqs, P = p.from.num_pages;
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
    cluster_sync();
  };
  const auto refuse = [&](uint32_t bits) {
    for (int i = rank * kFkThreads + tid; i < N; i += kFkCtas * kFkThreads) {
      p.to.lens[i] = -1;
      p.to.copy_src[i] = p.to.copy_dst[i] = -1;
      p.to.copy_tokens[i] = 0;
    }
    if (rank == 0 && tid == 0) atomicOr(p.status, bits);
  };

  // ---- (1) checks and the children of each old request (every CTA counts them all)
  for (int i = tid; i < R; i += kFkThreads) s.children[i] = 0;
  __syncthreads();
  uint32_t wrong = 0;
  for (int i = tid; i < N; i += kFkThreads) {
    const FkNew x = fk_new(p, i);
    wrong |= x.wrong;
    const int parent = __ldg(p.parent + i);
    if (!x.wrong && parent >= 0)
      atomicAdd(&s.children[parent], 1 + (p.grow && __ldg(p.grow + i) > 0 ? 1 << 16 : 0));
  }
  copy_refs();
  // warps of the cluster to old requests: several a request when these are few
  const int wpo = max(1, kGridWarps / max(1, R)), wpn = max(1, kGridWarps / max(1, N));
  for (int r = gwarp / wpo; r < R; r += kGridWarps / wpo) {
    const int n = __ldg(p.from.lens + r);
    if (n < 0 || n > (long long)kBlock * p.from.bt_stride) {
      wrong |= MSA_DEV_MALFORMED;
      continue;
    }
    const int nb = (n + kBlock - 1) / kBlock;
    for (int b = (gwarp % wpo) * 32 + lane; b < nb; b += 32 * wpo) {
      const int page = __ldg(p.from.block_table + (long long)r * p.from.bt_stride + b);
      if (page < 0 || page >= P) wrong |= MSA_DEV_BAD_PAGE;
      else if (__ldg(p.refs + page) < 1) wrong |= MSA_DEV_BAD_TABLE;
    }
  }
  wrong = __reduce_or_sync(kAll, wrong);
  if (lane == 0) s.warp[warp] = (int)wrong;
  __syncthreads();
  wrong = 0;
  for (int w = 0; w < kFkWarps; ++w) wrong |= (uint32_t)s.warp[w];
  exchange(s.flags, (int)wrong);
  wrong = 0;
  for (int c = 0; c < kFkCtas; ++c) wrong |= (uint32_t)s.flags[c];
  if (wrong) {
    refuse(wrong);
    return;
  }

  // ---- (2) holders gained and lost
  for (int r = gwarp / wpo; r < R; r += kGridWarps / wpo) {
    const int n = __ldg(p.from.lens + r), full = n / kBlock, nb = (n + kBlock - 1) / kBlock;
    const int all = s.children[r] & 0xffff, grown = s.children[r] >> 16;
    for (int b = (gwarp % wpo) * 32 + lane; b < nb; b += 32 * wpo) {
      const int d = (b < full ? all : all - grown) - 1;
      if (d) atomicAdd(refs + __ldg(p.from.block_table + (long long)r * p.from.bt_stride + b), d);
    }
  }
  __syncthreads();
  cluster_sync();

  // ---- (3) who keeps a partial page
  for (int i = rank * kFkThreads + tid; i < N; i += kFkCtas * kFkThreads) {
    const FkNew x = fk_new(p, i);
    if (x.partial && __ldcg(refs + x.last) <= 0) atomicMin(refs + x.last, -(N - i));
  }
  __syncthreads();
  cluster_sync();

  // ---- (4) new pages per request (every CTA for all), free pages
  const auto keeps = [&](const FkNew& x, int i) { return x.partial && __ldcg(refs + x.last) == -(N - i); };
  int total = 0;
  for (int i0 = 0; i0 < N; i0 += kFkThreads) {
    const int i = i0 + tid;
    int need = 0;
    if (i < N) {
      const FkNew x = fk_new(p, i);
      const bool copy = x.partial && !keeps(x, i);
      need = x.blocks - x.have + (copy ? 1 : 0);
      if (i % kFkCtas == rank) {
        p.to.lens[i] = x.n;
        p.to.copy_src[i] = copy ? x.last : -1;
        p.to.copy_tokens[i] = copy ? x.n % kBlock : 0;
        if (!copy) p.to.copy_dst[i] = -1;
      }
    }
    int sum;
    const int before = block_scan(need, s.warp, &sum);
    if (i < N) s.off[i] = total + before;
    total += sum;
  }
  if (tid == 0) s.off[N] = total;
  int zeros = 0;
  for (int i = p0 + tid; i < p1; i += kFkThreads) zeros += __ldcg(refs + i) == 0;
  zeros = __reduce_add_sync(kAll, zeros);
  __syncthreads();
  if (lane == 0) s.warp[warp] = zeros;
  __syncthreads();
  int mine = 0;
  for (int w = 0; w < kFkWarps; ++w) mine += s.warp[w];
  exchange(s.free_pages, mine);
  int at = 0, avail = 0;
  for (int c = 0; c < kFkCtas; ++c) {
    if (c < rank) at += s.free_pages[c];
    avail += s.free_pages[c];
  }
  if (avail < total) {
    copy_refs();
    refuse(MSA_DEV_NO_PAGES);
    return;
  }

  // ---- (5) tables
  for (int i = gwarp / wpn; i < N; i += kGridWarps / wpn) {
    const FkNew x = fk_new(p, i);
    const int parent = __ldg(p.parent + i);
    // (a kept page's count is negative until it becomes 1 below, a copied one's is not)
    const int count = s.off[i + 1] - s.off[i];
    const bool copy = count > x.blocks - x.have;
    const int shared = copy ? x.full : x.have;
    for (int b = (gwarp % wpn) * 32 + lane; b < shared; b += 32 * wpn)
      p.to.block_table[(long long)i * p.to.bt_stride + b] =
          __ldg(p.from.block_table + (long long)parent * p.from.bt_stride + b);
    if (x.partial && !copy && gwarp % wpn == 0 && lane == 0) refs[x.last] = 1;
  }
  for (int i0 = p0; i0 < p1 && at < total; i0 += kFkThreads) {
    const int page = i0 + tid;
    const bool free_page = page < p1 && __ldcg(refs + page) == 0;
    int sum;
    const int k = at + block_scan(free_page ? 1 : 0, s.warp, &sum);
    if (free_page && k < total) {
      int lo = 0, hi = N - 1;  // the last request whose first new page is k or before
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.off[mid] <= k) lo = mid; else hi = mid - 1;
      }
      const FkNew x = fk_new(p, lo);
      const bool copy = s.off[lo + 1] - s.off[lo] > x.blocks - x.have;
      const int j = k - s.off[lo];
      p.to.block_table[(long long)lo * p.to.bt_stride + (copy ? x.full : x.have) + j] = page;
      if (copy && j == 0) p.to.copy_dst[lo] = page;
      refs[page] = 1;
    }
    at += sum;
  }
}

// ------------------------------------------------------------------ copies

constexpr int kCpThreads = 256;

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
  page_fork_kernel<<<kFkCtas, kFkThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_page_copy(const CopyLaunch& p, cudaStream_t stream) {
  page_copy_kernel<<<p.num_copies * p.num_pools, kCpThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace msa
