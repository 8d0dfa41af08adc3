// qk_rope.cu -- norm, rotation and insertion of the new tokens in one pass: the
// queries and keys of every head normed (y = x (mean x^2 + eps)^-1/2 (w + shift))
// and rotated by position, queries handed on in bf16, keys, values and index keys
// written into the paged pools by the rules of kv_insert.cu.
//
// A vector of 128 values belongs to 16 lanes, 8 values each (a 16-byte load); a
// lane keeps the same dims for every vector of its row, so the row's cosines and
// sines are read once.  The sum of squares and the largest magnitude (scales of
// e4m3) are butterflies over the 16 lanes; rotation of halves takes the partner's
// values by shuffles, rotation of neighbours stays in the lane.  Everything is
// fp32 between the load and the one rounding at the end.
#include "prompt_common.cuh"

namespace msa {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  x[0] = bf16lo(r.x); x[1] = bf16hi(r.x); x[2] = bf16lo(r.y); x[3] = bf16hi(r.y);
  x[4] = bf16lo(r.z); x[5] = bf16hi(r.z); x[6] = bf16lo(r.w); x[7] = bf16hi(r.w);
}

// WPR warps share a row
template <int WPR>
__global__ void __launch_bounds__(kWarps * 32) qk_rope_kernel(const __grid_constant__ RopeLaunch p, int rows_per_cta) {
  __shared__ int s_le[kWarps];
  const msa_batch& b = p.batch;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane & 15;
  const unsigned full = 0xffffffffu;
  const int R = b.num_reqs, first_row = blockIdx.x * rows_per_cta;
  const int end_row = min(b.num_rows, first_row + rows_per_cta);

  // the first row's request, and whether cu_seqlens_q tiles the rows
  bool tiled = true;
  int le = 0;
  for (int q = tid; q < R; q += kWarps * 32) {
    const int c0 = b.cu_seqlens_q[q], c1 = b.cu_seqlens_q[q + 1];
    tiled &= c1 >= c0 && (q > 0 || c0 == 0) && (q < R - 1 || c1 == b.num_rows);
    le += c0 <= first_row;
  }
  le = __reduce_add_sync(full, le);
  if (lane == 0) s_le[warp] = le;
  tiled = __syncthreads_and(tiled) != 0;
  int q = -1;
  for (int w = 0; w < kWarps; ++w) q += s_le[w];

  const int half = p.rotary >> 1, steps = p.rotary >> 4;  // pairs; lanes of a half
  const int H = p.q.heads, Hk = p.k.heads, Hi = p.idx_k.heads, Di = p.idx_k.dim;
  const int nvec = H + 2 * Hk + 2 * Hi;
  int checked = -1, q0 = 0, qlen = 0, ctx = 0, nb = 0;
  uint32_t bad = tiled ? 0u : MSA_DEV_MALFORMED;

  for (int r = first_row + warp / WPR; r < end_row; r += kWarps / WPR) {
    if (tiled) {
      while (true) {  // the row's request: the first from q on that ends behind it
        const int at = q + 1 + lane;
        const unsigned past = __ballot_sync(full, at <= R && b.cu_seqlens_q[at] <= r);
        q += __popc(past);
        if (past != full) break;
      }
      if (q != checked) {
        checked = q;
        bad = request_lengths(b, q, &q0, &qlen, &ctx, &nb);
        bool odd = false;
        if (!bad) {
          const int32_t* table = b.block_table + (long long)q * b.bt_stride;
#pragma unroll 8
          for (int i = lane; i < nb; i += 32) {
            const int page = __ldg(table + i);
            odd |= page < 0 || page >= b.num_pages;
          }
        }
        if (__any_sync(full, odd)) bad = MSA_DEV_BAD_PAGE;
      }
    }
    uint32_t wrong = bad;
    int pos = ctx + (r - q0), rot = pos;
    if (p.rotary && !wrong) {
      if (p.positions) rot = __ldg(p.positions + r);
      if (rot < 0 || rot >= p.max_pos) wrong = MSA_DEV_BAD_POS;
    }
    long long token = 0;
    float cs[8], sn[8];  // of the lane's pairs (four when neighbours rotate)
    if (wrong) {
      if (lane == 0 && warp % WPR == 0) atomicOr(p.status, wrong);
    } else {
      token = (long long)__ldg(b.block_table + (long long)q * b.bt_stride + pos / kBlock) * kBlock + pos % kBlock;
      if (8 * l < p.rotary) {
        const float* t = p.cos_sin + (long long)rot * p.rotary + (p.near ? 4 * l : 8 * l < half ? 8 * l : 8 * l - half);
        const float4 c0 = __ldg(reinterpret_cast<const float4*>(t));
        const float4 s0 = __ldg(reinterpret_cast<const float4*>(t + half));
        cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w;
        sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w;
        if (!p.near) {
          const float4 c1 = __ldg(reinterpret_cast<const float4*>(t + 4));
          const float4 s1 = __ldg(reinterpret_cast<const float4*>(t + half + 4));
          cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
          sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
        }
      }
      if (p.mass && lane == 0 && warp % WPR == 0) p.mass[token] = 0.f;
    }
    for (int v0 = 2 * (warp % WPR); v0 < nvec; v0 += 2 * WPR) {
      // the half warp's vector: kind 0 q, 1 k, 2 v, 3 index q, 4 index k
      const int i = v0 + (lane >> 4);
      int kind = 0, h = i;
      if (h >= H) { h -= H; kind = 1; }
      if (kind == 1 && h >= Hk) { h -= Hk; kind = 2; }
      if (kind == 2 && h >= Hk) { h -= Hk; kind = 3; }
      if (kind == 3 && h >= Hi) { h -= Hi; kind = 4; }
      const RopeVec& x = kind == 0 ? p.q : kind == 1 ? p.k : kind == 2 ? p.v : kind == 3 ? p.idx_q : p.idx_k;
      const bool on = i < nvec && 8 * l < (kind < 3 ? kHeadDim : Di);
      if (wrong) {  // queries of a row that is not inserted
        uint16_t* out = kind == 0 ? p.q_out : kind == 3 ? p.idx_q_out : nullptr;
        if (on && out)
          *reinterpret_cast<uint4*>(out + ((long long)r * x.heads + h) * x.dim + 8 * l) = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      uint4 raw = make_uint4(0u, 0u, 0u, 0u), wr = make_uint4(0u, 0u, 0u, 0u);
      const uint16_t* norm = on ? x.norm : nullptr;
      if (on) raw = *reinterpret_cast<const uint4*>(x.src + (long long)r * x.stride + (long long)h * x.dim + 8 * l);
      if (norm) wr = __ldg(reinterpret_cast<const uint4*>(norm + 8 * l));
      float y[8];
      unpack8(raw, y);
      if (__any_sync(full, norm != nullptr)) {
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) ss += y[k] * y[k];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(full, ss, o);
        if (norm) {
          const float f = rsqrtf(ss / (float)x.dim + p.eps);
          float w[8];
          unpack8(wr, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = y[k] * f * (w[k] + p.shift);
        }
      }
      const bool turn = kind != 2 && 8 * l < p.rotary;
      if (p.near) {
        if (turn) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = y[2 * k], c = y[2 * k + 1];
            y[2 * k] = a * cs[k] - c * sn[k];
            y[2 * k + 1] = c * cs[k] + a * sn[k];
          }
        }
      } else if (p.rotary) {
        const bool low = l < steps;
        const int from = turn ? (low ? l + steps : l - steps) : l;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float o = __shfl_sync(full, y[k], from, 16);
          if (turn) y[k] = y[k] * cs[k] + (low ? -o : o) * sn[k];
        }
      }
      // where it goes
      const bool key = kind == 1 || kind == 2;
      const bool coded = on && (key ? p.kv_fp8 : kind == 4 && p.idx_fp8);
      float* scale = nullptr;  // written per token and head
      float s = 1.f;
      if (coded && key && p.scale_mode == MSA_SCALE_SCALAR) s = __ldg(kind == 1 ? p.k_scale : p.v_scale);
      if (coded && key && p.scale_mode == MSA_SCALE_PER_TOKEN_HEAD) scale = kind == 1 ? p.k_scale : p.v_scale;
      if (coded && !key) scale = p.idx_scale;
      if (__any_sync(full, scale != nullptr)) {
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(y[k]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(full, m, o));
        if (scale) {
          s = m > 0.f ? __fdiv_rn(m, 448.f) : 1.f;
          if (l == 0) scale[token * x.heads + h] = s;
        }
      }
      if (!on) continue;
      const long long at = (token * x.heads + h) * x.dim + 8 * l;
      if (coded) {
        uint8_t* dst = (kind == 1 ? p.k_cache : kind == 2 ? p.v_cache : p.idx_cache) + at;
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = __fdiv_rn(y[k], s);
        *reinterpret_cast<uint2*>(dst) = make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
        continue;
      }
      const uint4 w = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                 pack_bf16x2(y[6], y[7]));
      uint8_t* dst;
      if (kind == 0) dst = reinterpret_cast<uint8_t*>(p.q_out + ((long long)r * H + h) * kHeadDim + 8 * l);
      else if (kind == 3) dst = reinterpret_cast<uint8_t*>(p.idx_q_out + ((long long)r * Hi + h) * Di + 8 * l);
      else dst = (kind == 1 ? p.k_cache : kind == 2 ? p.v_cache : p.idx_cache) + 2 * at;
      *reinterpret_cast<uint4*>(dst) = w;
    }
  }
}

template <int WPR>
cudaError_t launch(const RopeLaunch& p, int rows_per_cta, cudaStream_t stream) {
  const int grid = (int)(((long long)p.batch.num_rows + rows_per_cta - 1) / rows_per_cta);
  qk_rope_kernel<WPR><<<grid, kWarps * 32, 0, stream>>>(p, rows_per_cta);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_rope_insert(const RopeLaunch& p, cudaStream_t stream) {
  const int n = p.batch.num_rows, sms = device_sm_count();
  if (n <= 4 * sms) return launch<8>(p, 1, stream);
  if (n <= 16 * sms) return launch<4>(p, 2, stream);
  return launch<1>(p, 16, stream);
}

}  // namespace msa
