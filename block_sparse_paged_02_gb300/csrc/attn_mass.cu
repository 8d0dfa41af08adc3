// attn_mass.cu -- the attention weight that a step's rows gave each cached
// token, added up over rows and heads into a paged array.
//
// Mathematics.  w_t = sum over (row, head) that see t of 2^(s - lse), both in
// log2 units, with the row's lse known from the attention: one product Q K^T
// and a sum over the rows, no second pass.  A token belongs to one CTA, which
// adds its rows in a fixed order: no atomics, the same bits every time.
//
// The keys are the rows of the product (S^T = K Q^T on warp MMA, m16n8k16):
// a warp keeps its 16 tokens' keys in registers for all the rows, the sum
// over a row's heads is a sum over accumulator columns, and only the last
// four partial sums cross lanes.
#include <string.h>

#include "tree_common.cuh"

namespace msa {
namespace {

constexpr int kMaThreads = 256;
constexpr int kQRows = 64;  // rows x heads per pass over Q

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <bool FP8>
struct MassCfg {
  static constexpr int kPage = kBlock * kHeadDim * (FP8 ? 1 : 2);
  static constexpr int kSmQ = kPage;                       // [2 halves][64 rows][128 B], swizzled
  static constexpr int kSmLse = kSmQ + kQRows * 256;
  static constexpr int kSmBar = kSmLse + kQRows * 4;
  static constexpr int kSmScan = kSmBar + 16;
  static constexpr int kBytes = kSmScan + 40 * 8 + 1024;
};

__device__ __forceinline__ long long mass_weight(int qlen, int heads) {
  return (qlen * heads + kQRows - 1) / kQRows;  // passes over Q per block
}

template <bool FP8>
__global__ void __launch_bounds__(kMaThreads, FP8 ? 4 : 3)
    attn_mass_kernel(const TreeLaunch p, const __grid_constant__ CUtensorMap kmap) {
  using C = MassCfg<FP8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::kSmBar);
  float* s_lse = reinterpret_cast<float*>(smem + C::kSmLse);
  long long* s_ll = reinterpret_cast<long long*>(smem + C::kSmScan);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int H = p.num_heads;
  if (tid == 0) {
    mbar_init(bar, 1);
    fence_barrier_init();
  }
  const TreeSlice sl = tree_slice<kMaThreads>(
      p,
      [&](int q) -> long long {
        TreeReq r = tree_request(p, q);
        if (r.qlen <= 0) return 0;
        const int n = tree_visits(p, q, r);
        return r.bad ? 1 : n * mass_weight(r.qlen, H);
      },
      s_ll);
  __syncthreads();
  if (!sl.tiled) {
    if (tid == 0 && blockIdx.x == 0) atomicOr(p.status, MSA_DEV_MALFORMED);
    return;
  }
  if (sl.begin >= sl.end) return;
  float scale2 = p.softmax_scale * kTreeLog2e;
  if (p.scale_mode == MSA_SCALE_SCALAR) scale2 *= __ldg(p.k_scale);
  const bool pth = p.scale_mode == MSA_SCALE_PER_TOKEN_HEAD;
  long long pre = sl.pre;
  uint32_t phase = 0;
  const uint32_t q_s = smem_u32(smem + C::kSmQ);

  for (int q = sl.q; q < p.batch.num_reqs && pre < sl.end; ++q) {
    TreeReq rq = tree_request(p, q);
    if (rq.qlen <= 0) continue;
    const int nv = tree_visits(p, q, rq);  // 1 for a poisoned request
    const long long w = rq.bad ? 1 : mass_weight(rq.qlen, H);
    const long long first = pre;
    pre += nv * w;
    if (!rq.bad) {
      // a bad page anywhere leaves the whole request as it is
      bool bad = false;
      for (int b = tid; b < rq.nb; b += kMaThreads) {
        const int page = p.batch.block_table[(long long)q * p.batch.bt_stride + b];
        bad |= page < 0 || page >= p.batch.num_pages;
      }
      if (__syncthreads_or(bad)) rq.bad = MSA_DEV_BAD_PAGE;
    }
    if (rq.bad) {
      if (tid == 0) atomicOr(p.status, rq.bad);
      continue;
    }
    // blocks whose first item lies in the slice
    const int i0 = (int)((max(sl.begin, first) - first + w - 1) / w);
    const int i1 = (int)min((long long)nv, (sl.end - first + w - 1) / w);
    const int rows = rq.qlen * H, seq = rq.ctx + rq.qlen;
    for (int i = i0; i < i1; ++i) {
      const int b = p.topk_idx ? p.list_blk[(long long)q * p.list_cap + i] : i;
      const int page = p.batch.block_table[(long long)q * p.batch.bt_stride + b];
      const bool cached_all = !p.topk_idx || b >= rq.ctx / kBlock;
      const uint32_t* sel =
          cached_all ? nullptr : p.list_rows + ((long long)q * p.list_cap + i) * p.list_words;
      const bool mixed = !cached_all || kBlock * b + kBlock > rq.ctx;
      __syncthreads();  // the previous block's keys have been read
      if (tid == 0) {
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(bar, C::kPage);
        tma_load_2d(smem, &kmap, 0, page * kBlock, bar);
        if constexpr (!FP8) tma_load_2d(smem + C::kPage / 2, &kmap, 64, page * kBlock, bar);
      }
      const bool there = mbar_wait(bar, phase);
      phase ^= 1;
      if (!__syncthreads_and(there)) {
        if (tid == 0) atomicOr(p.status, MSA_DEV_TIMEOUT);
        return;
      }
      // ---- this warp's 16 tokens as the A operand
      uint32_t ka[8][4];
      const int t0 = kBlock * b + 16 * warp;
      if constexpr (FP8) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const uint8_t* kr = smem + (16 * warp + g + 8 * hh) * kHeadDim;
          const uint4 a = lds128(kr + (((2 * c) ^ g) << 4)), d = lds128(kr + (((2 * c + 1) ^ g) << 4));
          const uint32_t w8[8] = {a.x, a.y, a.z, a.w, d.x, d.y, d.z, d.w};
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            ka[kk][hh] = e4m3x2_to_f16x2((uint16_t)(w8[kk] & 0xffffu));
            ka[kk][2 + hh] = e4m3x2_to_f16x2((uint16_t)(w8[kk] >> 16));
          }
        }
      } else {
        const int row = 16 * warp + (lane & 15);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const int ch = 2 * kk + (lane >> 4);
          ldsm4(smem_u32(smem) + (ch >> 3) * (C::kPage / 2) + row * 128 + (((ch & 7) ^ (row & 7)) << 4),
                ka[kk]);
        }
      }
      const long long slot = (long long)page * kBlock + 16 * warp;
      float f[2] = {scale2, scale2};
      if (pth) {
        f[0] *= __ldg(p.k_scale + slot + g);
        f[1] *= __ldg(p.k_scale + slot + g + 8);
      }
      float acc[2] = {0.f, 0.f};
      for (int r0 = 0; r0 < rows; r0 += kQRows) {
        const int n = min(kQRows, rows - r0);
        __syncthreads();
        for (int x = tid; x < kQRows * 16; x += kMaThreads) {  // 16-byte chunks of Q
          const int row = x >> 4, ch = x & 15;
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (row < n)
            v = __ldg(reinterpret_cast<const uint4*>(p.q + ((long long)rq.q0 * H + r0 + row) * kHeadDim) + ch);
          if constexpr (FP8) {
            v.x = pack_f16x2(bf16lo(v.x), bf16hi(v.x));
            v.y = pack_f16x2(bf16lo(v.y), bf16hi(v.y));
            v.z = pack_f16x2(bf16lo(v.z), bf16hi(v.z));
            v.w = pack_f16x2(bf16lo(v.w), bf16hi(v.w));
          }
          *reinterpret_cast<uint4*>(smem + C::kSmQ + (ch >> 3) * (kQRows * 128) + row * 128 +
                                    (((ch & 7) ^ (row & 7)) << 4)) = v;
        }
        if (tid < kQRows) {
          // a row that saw nothing (lse -inf) or lies past the end gives nothing
          const float l = tid < n ? __ldg(p.lse + (long long)rq.q0 * H + r0 + tid) : -INFINITY;
          s_lse[tid] = l == -INFINITY ? INFINITY : l * kTreeLog2e;
        }
        __syncthreads();
        for (int u = 0; u < (n + 7) / 8; ++u) {
          float s[4] = {0.f, 0.f, 0.f, 0.f};
          const int row = 8 * u + (FP8 ? g : (lane & 7));
          if constexpr (FP8) {
            const uint8_t* qr = smem + C::kSmQ + (c >> 1) * (kQRows * 128) + row * 128;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint4 v = lds128(qr + (((4 * (c & 1) + x) ^ (row & 7)) << 4));
              mma16816<true>(s, ka[2 * x], v.x, v.y);
              mma16816<true>(s, ka[2 * x + 1], v.z, v.w);
            }
          } else {
#pragma unroll
            for (int kp = 0; kp < 4; ++kp) {
              uint32_t v[4];
              const int ch = 4 * kp + (lane >> 3);
              ldsm4(q_s + (ch >> 3) * (kQRows * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4), v);
              mma16816<false>(s, ka[2 * kp], v[0], v[1]);
              mma16816<false>(s, ka[2 * kp + 1], v[2], v[3]);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int m = 8 * u + 2 * c + e;
            const float l = s_lse[m];
            uint32_t vis = 0xffffu;
            if (l == INFINITY) {
              vis = 0;
            } else if (mixed) {
              const int j = (r0 + m) / H;
              vis = tree_vis16(p, rq.q0 + j, j, rq.ctx, rq.qlen, t0, tree_row_selects(sel, j));
            }
            const float p0 = exp2f(fmaf(s[e], f[0], -l)), p1 = exp2f(fmaf(s[2 + e], f[1], -l));
            acc[0] += (vis >> g) & 1u ? p0 : 0.f;
            acc[1] += (vis >> (g + 8)) & 1u ? p1 : 0.f;
          }
        }
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        acc[hh] += __shfl_xor_sync(0xffffffffu, acc[hh], 1);
        acc[hh] += __shfl_xor_sync(0xffffffffu, acc[hh], 2);
        const int t = t0 + g + 8 * hh;
        if (c == 0 && t < seq) {
          float* m = p.mass + slot + g + 8 * hh;
          *m = t < rq.ctx ? *m + acc[hh] : acc[hh];
        }
      }
    }
  }
}

template <bool FP8>
cudaError_t launch_mass(const TreeLaunch& p, cudaStream_t stream) {
  using C = MassCfg<FP8>;
  CUtensorMap kmap;
  const CUtensorMapDataType t = FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!encode_map_2d(&kmap, t, p.k, kHeadDim, max(1ll, (long long)p.batch.num_pages) * kBlock,
                     kHeadDim * (FP8 ? 1 : 2), FP8 ? 128 : 64, kBlock))
    return cudaErrorInvalidValue;
  auto kern = attn_mass_kernel<FP8>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e != cudaSuccess) return e;
  kern<<<device_sm_count() * (FP8 ? 4 : 3), kMaThreads, C::kBytes, stream>>>(p, kmap);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_mass(const TreeLaunch& p, cudaStream_t stream) {
  if (p.topk_idx) {
    const cudaError_t e = launch_tree_plan(p, stream);
    if (e != cudaSuccess) return e;
  }
  return p.kv_fp8 ? launch_mass<true>(p, stream) : launch_mass<false>(p, stream);
}

}  // namespace msa
