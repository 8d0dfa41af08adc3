// attn_tc.cuh -- the softmax side of attention on the 5th-generation tensor
// cores, one thread per row (tensor-memory lane), 64 logits at a time: maxima,
// exponentials written back as 16-bit P, a P V added by hand where V holds
// values that must not reach every row, and the layout of what they read.
// Shared by the draft-tree attention and the whole-prompt attention.
#pragma once

#include "tcgen05.cuh"
#include "tree_common.cuh"

namespace msa {
namespace {

constexpr int kHalf = 128 * 128;  // 128 rows x 128 B: one swizzle-atom column of a tile
constexpr int kTile = 2 * kHalf;  // 128 x 128 bf16
constexpr int kRaw = 128 * 128;   // 128 x 128 e4m3

// blocks whose scales are held: the factors of the logits, the v scales, log2 of their
// magnitudes; then the largest and the smallest of these of each 32 tokens
constexpr int kScales = 4;
constexpr int kSoV = 128, kSoLog = 2 * 128, kSoRange = 3 * 128, kScaleWords = 3 * 128 + 8;
// With a scale per token P is kept relative to max(s + log2 |v scale|).  Where the 64
// tokens' scales lie within 2^kNear, max(s) + max(log2 |v scale|) stands for it, at most that
// much above: the exact maximum needs a second word per token from shared memory for every
// row (2 requests of 33 rows x 12 heads over 131K tokens: 107 us with it everywhere, 102 so).
constexpr float kNear = 4.f;

template <int N>
__device__ __forceinline__ void regs_fewer() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// largest of N logits and acc (of their negations when NEG), those with a set
// bit only when MASKED, each times its token's factor ks when PTH, plus lv when EXACT
template <bool NEG, bool MASKED, bool PTH, bool EXACT = false, int N>
__device__ __forceinline__ float row_max(const uint32_t (&r)[N], float acc, uint32_t vis0,
                                         uint32_t vis1, const float* ks,
                                         const float* lv = nullptr) {
  float g[8] = {acc, acc, acc, acc, acc, acc, acc, acc};
#pragma unroll
  for (int t = 0; t < N; t += 2) {
    float a = __uint_as_float(r[t]), b = __uint_as_float(r[t + 1]);
    if (PTH) {
      const float2 k = *reinterpret_cast<const float2*>(ks + t);
      mul2v(a, b, k.x, k.y);
    }
    if (EXACT) {
      a += lv[t];
      b += lv[t + 1];
    }
    if (NEG) {
      a = -a;
      b = -b;
    }
    if (MASKED) {
      const uint32_t vis = t < 32 ? vis0 : vis1;
      a = (vis >> (t & 31)) & 1u ? a : -INFINITY;
      b = (vis >> ((t + 1) & 31)) & 1u ? b : -INFINITY;
    }
    g[(t >> 1) & 7] = fmax3(g[(t >> 1) & 7], a, b);
  }
  return fmax3(fmax3(g[0], g[1], g[2]), fmax3(g[3], g[4], g[5]), fmaxf(g[6], g[7]));
}

// P = 2^(s * scale2 - m) of N logits as 16-bit pairs into the N / 2 columns at pa
// (with PTH the token's ks in the place of scale2, which SCALED logits carry already, and P
// times its vs); returns the fp32 sum of the 2^...
template <bool MASKED, bool FP8, bool PTH, bool SCALED = false, int N>
__device__ __forceinline__ float row_exp(const uint32_t (&r)[N], uint32_t pa, float scale2, float m,
                                         uint32_t vis0, uint32_t vis1, const float* ks,
                                         const float* vs) {
  // (eight sums: with four, the packed adds' latency bound the softmax, 900
  // cycles for a warp's 64 columns against 390)
  float l[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int q = 0; q < N / 32; ++q) {
    uint32_t w[16];
    float4 four = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const int t = 32 * q + i;
      float a = __uint_as_float(r[t]), b = __uint_as_float(r[t + 1]);
      if (SCALED) {
        add2(a, b, -m, -m);
      } else if (PTH) {
        const float2 k = *reinterpret_cast<const float2*>(ks + t);
        fma2p(a, b, k.x, k.y, -m);
      } else {
        fma2(a, b, scale2, -m);
      }
      a = ex2_ftz(a);
      b = ex2_ftz(b);
      const uint32_t v = q ? vis1 : vis0;
      if (MASKED) {
        a = (v >> i) & 1u ? a : 0.f;
        b = (v >> (i + 1)) & 1u ? b : 0.f;
      }
      add2(l[i & 6], l[(i & 6) + 1], a, b);
      if (PTH) {
        float2 x;
        if (SCALED) {
          if ((i & 2) == 0) four = *reinterpret_cast<const float4*>(vs + t);
          x = (i & 2) == 0 ? make_float2(four.x, four.y) : make_float2(four.z, four.w);
        } else {
          x = *reinterpret_cast<const float2*>(vs + t);
        }
        mul2v(a, b, x.x, x.y);
        if (MASKED) {  // (the scale of a token that the row does not see may be anything)
          a = (v >> i) & 1u ? a : 0.f;
          b = (v >> (i + 1)) & 1u ? b : 0.f;
        }
      }
      w[i >> 1] = FP8 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
    }
    tc::tmem_st16(pa + 16 * q, w);
  }
  return ((l[0] + l[1]) + (l[2] + l[3])) + ((l[4] + l[5]) + (l[6] + l[7]));
}

// O += P V of a block for the row of this thread, the tokens with a set bit of vis
// alone; P of the first 64 tokens (times f0) at pa, of the others kNext behind it, and O at oa in
// tensor memory, V at v, `words` x 32 tokens; O starts with it when fresh
template <bool FP8, int kNext = 32>
__device__ __noinline__ void pv_by_hand(uint32_t oa, uint32_t pa, const uint8_t* v, uint4 vis4,
                                        int words, float f0, bool fresh) {
  tc::tmem_wait_st();
#pragma unroll 1
  for (int c = 0; c < 128; c += 16) {
    uint32_t o[16];
    if (!fresh) tc::tmem_ld16(oa + c, o);
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = fresh ? 0.f : __uint_as_float(o[i]);
#pragma unroll 1
    for (int w = 0; w < words; ++w) {
      uint32_t pr[16];
      tc::tmem_ld16(pa + 16 * w + (w < 2 ? 0 : kNext - 32), pr);
      const uint32_t vis = w == 0 ? vis4.x : w == 1 ? vis4.y : w == 2 ? vis4.z : vis4.w;
      const float f = w < 2 ? f0 : 1.f;
#pragma unroll
      for (int t = 0; t < 32; ++t) {
        if ((vis >> t) & 1u) {
          const int tok = 32 * w + t;
          const uint8_t* row = v + (c >> 6) * kHalf + tok * 128;
          float x;
          if (FP8) {
            const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&pr[t >> 1]));
            x = t & 1 ? h.y : h.x;
          } else {
            x = t & 1 ? bf16hi(pr[t >> 1]) : bf16lo(pr[t >> 1]);
          }
          x *= f;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint4 q = lds128(row + (((((c >> 3) & 7) + k) ^ (tok & 7)) << 4));
            const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float2 y;
              if (FP8) y = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
              else y = make_float2(bf16lo(u[i]), bf16hi(u[i]));
              acc[8 * k + 2 * i] += x * y.x;
              acc[8 * k + 2 * i + 1] += x * y.y;
            }
          }
        }
      }
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(acc[i]);
    tc::tmem_st16(oa + c, o);
  }
}

}  // namespace
}  // namespace msa
