// qk_rope.cu -- norm, rotation and insertion of the new tokens in one pass: the
// queries and keys of every head normed (y = x (mean x^2 + eps)^-1/2 (w + shift))
// and rotated by position, queries handed on in bf16, keys, values and index keys
// written into the paged pools by the rules of kv_insert.cu.
//
// A vector of 128 values belongs to 8 lanes, two chunks of 8 values each (two
// 16-byte loads), one of 64 values to 4 lanes.  Rotation of halves pairs chunk c with
// chunk c + rotary / 16, so a lane holds both values of its pairs and rotation
// needs no exchange; the sum of squares and the largest magnitude (scales of e4m3)
// are butterflies over the vector's lanes.  Everything is fp32 between the load and
// the one rounding at the end.
//
// A warp takes four query heads at a time; what is left of a row (odd query heads,
// keys, values, index vectors) goes through a second form that picks source, weights
// and destination by lane group.  Weights, cosines and sines lie in shared memory:
// held in registers they cost the occupancy that hides the loads (12.6 K rows, below:
// 36 us at two CTAs an SM, 31.4 at four).  A warp of many rows asks for the next four
// heads before it turns these (31.2 us without, 28.5 with).
//
// Measured (graph, 16 heads, bf16 pools, two index heads of 64, rotary 64): one row 4.4
// us, 64 rows over e4m3 with scales 5.3, both a launch and a chain of loads; 12.6 K
// rows of neighbours' rotation 28.5 us, 133 MB at 4.7 TB/s (69 % of the copy rate), over
// e4m3 29.7, with scales 30.1: bound by load latency, 3 rows to each of seven warps (the
// eighth has none), each a chain of angles, heads, rest.
//
// A request's pages are all looked at before one of its rows is written, by every warp
// that has such a row, so the time grows with the context: one row behind 8 K tokens 4.7
// us, 131 K 5.2, 1 M 11.5; 64 rows behind 8 K each 5.0, 131 K 5.6; 4096 rows of one
// request behind 0, 131 K, 500 K and 1 M tokens 10.1, 11.1, 13.8 and 17.5.
#include "prompt_common.cuh"

namespace msa {
namespace {

constexpr int kWarps = 8;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// a pair at a time: c += a * b, a * b
__device__ __forceinline__ void fma_pair(float& c0, float& c1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%0, %1};\n\tfma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "+f"(c0), "+f"(c1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void mul_pair(float& c0, float& c1, float b0, float b1) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(c0), "+f"(c1)
      : "f"(b0), "f"(b1));
}

// A lane's 16 values of a vector: chunk a, then chunk b
struct Lane16 {
  float x[16];
  __device__ __forceinline__ void unpack(const uint4& a, const uint4& b) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[2 * k] = bf16lo(w[k]);
      x[2 * k + 1] = bf16hi(w[k]);
    }
  }
  // eight values from k on, by f times eight weights in shared memory
  __device__ __forceinline__ void scale8(int k, float f, const float* w) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      float4 y = *reinterpret_cast<const float4*>(w + i);
      mul_pair(y.x, y.y, f, f);
      mul_pair(y.z, y.w, f, f);
      mul_pair(x[k + i], x[k + i + 1], y.x, y.y);
      mul_pair(x[k + i + 2], x[k + i + 3], y.z, y.w);
    }
  }
  __device__ __forceinline__ float squares() const {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 16; k += 2) fma_pair(s[k & 2], s[(k & 2) + 1], x[k], x[k + 1], x[k], x[k + 1]);
    return (s[0] + s[1]) + (s[2] + s[3]);
  }
  __device__ __forceinline__ float largest() const {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) m = fmaxf(m, fabsf(x[k]));
    return m;
  }
  // pairs (k, 8 + k) by eight cosines and sines in shared memory
  __device__ __forceinline__ void rotate_halves(const float* cs, const float* sn) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 c4 = *reinterpret_cast<const float4*>(cs + i), s4 = *reinterpret_cast<const float4*>(sn + i);
      const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const int y = i + k;
        float a0 = x[y], a1 = x[y + 1], b0 = x[8 + y], b1 = x[9 + y];
        mul_pair(a0, a1, c[k], c[k + 1]);
        mul_pair(b0, b1, c[k], c[k + 1]);
        fma_pair(a0, a1, x[8 + y], x[9 + y], -s[k], -s[k + 1]);
        fma_pair(b0, b1, x[y], x[y + 1], s[k], s[k + 1]);
        x[y] = a0; x[y + 1] = a1; x[8 + y] = b0; x[9 + y] = b1;
      }
    }
  }
  // the four pairs of neighbours from value `at` on
  template <int at>
  __device__ __forceinline__ void rotate_near(const float* cs, const float* sn) {
    const float4 c4 = *reinterpret_cast<const float4*>(cs), s4 = *reinterpret_cast<const float4*>(sn);
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = x[at + 2 * k], b = x[at + 2 * k + 1];
      x[at + 2 * k] = a * c[k] - b * s[k];
      x[at + 2 * k + 1] = b * c[k] + a * s[k];
    }
  }
  // of place l among the vector's n lanes, by the table's row
  __device__ __forceinline__ void rotate(const float* row, int l, int n, int pairs, bool near) {
    const float* sn = row + 8 * pairs;
    if (near) {
      if (l < 2 * pairs) rotate_near<0>(row + 4 * l, sn + 4 * l);
      if (l + n < 2 * pairs) rotate_near<8>(row + 4 * (l + n), sn + 4 * (l + n));
    } else if (l < pairs) {
      rotate_halves(row + 8 * l, sn + 8 * l);
    }
  }
  __device__ __forceinline__ uint4 bf16(int k) const {
    return make_uint4(pack_bf16x2(x[k], x[k + 1]), pack_bf16x2(x[k + 2], x[k + 3]),
                      pack_bf16x2(x[k + 4], x[k + 5]), pack_bf16x2(x[k + 6], x[k + 7]));
  }
};

// sum / maximum over groups of `lanes` lanes (8 or 4)
__device__ __forceinline__ float group_sum(float v, bool eight) {
  v += __shfl_xor_sync(kAll, v, 1);
  v += __shfl_xor_sync(kAll, v, 2);
  const float o = __shfl_xor_sync(kAll, v, 4);
  return eight ? v + o : v;
}
__device__ __forceinline__ float group_max(float v, bool eight) {
  v = fmaxf(v, __shfl_xor_sync(kAll, v, 1));
  v = fmaxf(v, __shfl_xor_sync(kAll, v, 2));
  const float o = __shfl_xor_sync(kAll, v, 4);
  return eight ? fmaxf(v, o) : v;
}

// First dims of a lane's chunks: place l among the vector's n lanes.  Halves: `pairs` lanes
// hold the two values of their pairs, the others chunks that do not rotate; neighbours: chunks n
// apart.  A load or store of a vector's lanes covers whole sectors either way.
__device__ __forceinline__ int chunk_a(int l, int pairs, bool near) {
  return 8 * (near || l < pairs ? l : pairs + l);
}
__device__ __forceinline__ int chunk_b(int l, int n, int pairs, bool near) {
  return 8 * (near || l >= pairs ? l + n : l + pairs);
}

// WPR warps share a row; their other rows follow it
template <int WPR>
__global__ void __launch_bounds__(kWarps * 32, 4) qk_rope_kernel(const __grid_constant__ RopeLaunch p, int rows_per_cta) {
  __shared__ int s_le[kWarps];
  // the four kinds' weights, and each warp's row of the table (registers are short)
  __shared__ __align__(16) float s_w[4][kHeadDim], s_cs[kWarps][kHeadDim];
  constexpr int kTeams = kWarps / WPR;
  const msa_batch& b = p.batch;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane & 7, group = lane >> 3;
  const int R = b.num_reqs, first_row = blockIdx.x * rows_per_cta;
  const int each = (rows_per_cta + kTeams - 1) / kTeams;  // rows of a team
  const int team_row = first_row + warp / WPR * each;
  const int end_row = min(b.num_rows, min(first_row + rows_per_cta, team_row + each));

  // the first row's request, and whether cu_seqlens_q tiles the rows
  bool tiled = true;
  int le = 0;
  for (int q = tid; q < R; q += kWarps * 32) {
    const int c0 = b.cu_seqlens_q[q], c1 = b.cu_seqlens_q[q + 1];
    tiled &= c1 >= c0 && (q > 0 || c0 == 0) && (q < R - 1 || c1 == b.num_rows);
    le += c0 <= first_row;
  }
  for (int i = tid; i < 4 * kHeadDim; i += kWarps * 32) {
    const int kind = i / kHeadDim, d = i % kHeadDim;
    const RopeVec* x = kind == 0 ? &p.q : kind == 1 ? &p.k : kind == 2 ? &p.idx_q : &p.idx_k;
    if (x->norm && d < x->dim) s_w[kind][d] = __uint_as_float((uint32_t)__ldg(x->norm + d) << 16) + p.shift;
  }
  le = __reduce_add_sync(kAll, le);
  if (lane == 0) s_le[warp] = le;
  tiled = __syncthreads_and(tiled) != 0;
  int q = -1;
  for (int w = 0; w < kWarps; ++w) q += s_le[w];

  const bool near = p.near != 0;
  const int pairs = p.rotary >> 4;  // lanes that rotate halves
  const int H = p.q.heads, Hk = p.k.heads, Hi = p.idx_k.heads, Di = p.idx_k.dim;
  const int quads = H >> 2;                               // steps of four query heads
  const int per_slot = Di == 64 ? 2 : 1;                  // index vectors of 8 lanes
  const int islots = (Hi + per_slot - 1) / per_slot, rest = (H & 3) + 2 * Hk + 2 * islots;
  const int steps = quads + ((rest + 3) >> 2);
  const int ca = chunk_a(l, pairs, near), cb = chunk_b(l, 8, pairs, near);
  int q_end = -1, q0 = 0, qlen = 0, ctx = 0, nb = 0;
  uint32_t bad = tiled ? 0u : MSA_DEV_MALFORMED;

  for (int r = team_row; r < end_row; ++r) {
    if (tiled && r >= q_end) {
      while (true) {  // the row's request: the first from q on that ends behind it
        const int at = q + 1 + lane;
        const unsigned past = __ballot_sync(kAll, at <= R && b.cu_seqlens_q[at] <= r);
        q += __popc(past);
        if (past != kAll) break;
      }
      bad = request_lengths(b, q, &q0, &qlen, &ctx, &nb);
      q_end = q0 + qlen;
      bool odd = false;
      if (!bad) {
        const int32_t* table = b.block_table + (long long)q * b.bt_stride;
#pragma unroll 8
        for (int i = lane; i < nb; i += 32) {
          const int page = __ldg(table + i);
          odd |= page < 0 || page >= b.num_pages;
        }
      }
      if (__any_sync(kAll, odd)) bad = MSA_DEV_BAD_PAGE;
    }
    uint32_t wrong = bad;
    const int pos = ctx + (r - q0);
    int rot = pos;
    if (p.rotary && !wrong) {
      if (p.positions) rot = __ldg(p.positions + r);
      if (rot < 0 || rot >= p.max_pos) wrong = MSA_DEV_BAD_POS;
    }
    if (wrong) {  // not inserted; its queries are 0
      if (warp % WPR == 0) {
        if (lane == 0) atomicOr(p.status, wrong);
        uint4* out = reinterpret_cast<uint4*>(p.q_out + (long long)r * H * kHeadDim);
        for (int i = lane; i < H * kHeadDim / 8; i += 32) out[i] = make_uint4(0u, 0u, 0u, 0u);
        out = reinterpret_cast<uint4*>(p.idx_q_out + (long long)r * Hi * Di);
        for (int i = lane; i < Hi * Di / 8; i += 32) out[i] = make_uint4(0u, 0u, 0u, 0u);
      }
      continue;
    }
    const float* table = p.cos_sin + (long long)rot * p.rotary;
    float* mine = s_cs[warp];
    // (the first heads are asked for before the angles are waited for, where a warp takes
    // several; with one the angles go first)
    const uint16_t* src = p.q.src + (long long)r * p.q.stride + group * kHeadDim;
    uint4 na = make_uint4(0u, 0u, 0u, 0u), nc = na;
    if (WPR < kWarps && warp % WPR < quads) {
      na = *reinterpret_cast<const uint4*>(src + warp % WPR * 4 * kHeadDim + ca);
      nc = *reinterpret_cast<const uint4*>(src + warp % WPR * 4 * kHeadDim + cb);
    }
    __syncwarp();  // the row before has been turned
    if (4 * lane < p.rotary)
      *reinterpret_cast<float4*>(mine + 4 * lane) = __ldg(reinterpret_cast<const float4*>(table) + lane);
    __syncwarp();

    // ---- four query heads at a time
    uint16_t* dst = p.q_out + ((long long)r * H + group) * kHeadDim;
    for (int s0 = warp % WPR; s0 < quads; s0 += WPR) {
      const int at = s0 * 4 * kHeadDim;
      Lane16 v;
      if (WPR == kWarps) {
        na = *reinterpret_cast<const uint4*>(src + at + ca);
        nc = *reinterpret_cast<const uint4*>(src + at + cb);
      }
      v.unpack(na, nc);
      if (WPR < kWarps && s0 + WPR < quads) {
        na = *reinterpret_cast<const uint4*>(src + at + 4 * WPR * kHeadDim + ca);
        nc = *reinterpret_cast<const uint4*>(src + at + 4 * WPR * kHeadDim + cb);
      }
      if (p.q.norm) {
        const float f = rsqrtf(group_sum(v.squares(), true) * (1.f / kHeadDim) + p.eps);
        v.scale8(0, f, s_w[0] + ca);
        v.scale8(8, f, s_w[0] + cb);
      }
      v.rotate(mine, l, 8, pairs, near);
      *reinterpret_cast<uint4*>(dst + at + ca) = v.bf16(0);
      *reinterpret_cast<uint4*>(dst + at + cb) = v.bf16(8);
    }
    // ---- the rest, a vector (two index vectors of 64) to a group of 8 lanes
    int s0 = warp % WPR;
    if (s0 < quads) s0 += (quads - s0 + WPR - 1) / WPR * WPR;
    for (int step = s0; step < steps; step += WPR) {
      const int page = __ldg(b.block_table + (long long)q * b.bt_stride + pos / kBlock);
      const long long token = (long long)page * kBlock + pos % kBlock;
      // kind 0 q, 1 k, 2 v, 3 index q, 4 index k
      int h = 4 * (step - quads) + group, kind = 0;
      const bool any = h < rest;
      if (h >= (H & 3)) { h -= H & 3; kind = 1; }
      if (kind == 1 && h >= Hk) { h -= Hk; kind = 2; }
      if (kind == 2 && h >= Hk) { h -= Hk; kind = 3; }
      if (kind == 3 && h >= islots) { h -= islots; kind = 4; }
      if (kind == 0) h += 4 * quads;
      const RopeVec* x = kind == 0 ? &p.q : kind == 1 ? &p.k : kind == 2 ? &p.v : kind == 3 ? &p.idx_q : &p.idx_k;
      const bool eight = kind < 3 || Di == kHeadDim;
      if (!eight) h = 2 * h + (l >> 2);
      const int m = eight ? l : l & 3, heads = x->heads, dim = eight ? kHeadDim : 64;  // place among the vector's lanes
      const bool on = any && h < heads;
      const int a = chunk_a(m, pairs, near), c = chunk_b(m, eight ? 8 : 4, pairs, near);
      const uint16_t* norm = on ? x->norm : nullptr;
      uint4 ra = make_uint4(0u, 0u, 0u, 0u), rb = ra;
      if (on) {
        const uint16_t* from = x->src + (long long)r * x->stride + (long long)h * dim;
        ra = *reinterpret_cast<const uint4*>(from + a);
        rb = *reinterpret_cast<const uint4*>(from + c);
      }
      Lane16 v;
      v.unpack(ra, rb);
      if (__any_sync(kAll, norm != nullptr)) {
        const float f = rsqrtf(group_sum(v.squares(), eight) * (eight ? 1.f / 128 : 1.f / 64) + p.eps);
        if (norm) {
          const float* w = s_w[kind < 2 ? kind : kind - 1];
          v.scale8(0, f, w + a);
          v.scale8(8, f, w + c);
        }
      }
      if (on && kind != 2) v.rotate(mine, m, eight ? 8 : 4, pairs, near);
      // where it goes
      const bool key = kind == 1 || kind == 2;
      const bool coded = on && (key ? p.kv_fp8 != 0 : kind == 4 && p.idx_fp8);
      float* scale = nullptr;  // written per token and head
      float s = 1.f;
      if (coded && key && p.scale_mode == MSA_SCALE_SCALAR) s = __ldg(kind == 1 ? p.k_scale : p.v_scale);
      if (coded && key && p.scale_mode == MSA_SCALE_PER_TOKEN_HEAD) scale = kind == 1 ? p.k_scale : p.v_scale;
      if (coded && !key) scale = p.idx_scale;
      if (__any_sync(kAll, scale != nullptr)) {
        const float top = group_max(v.largest(), eight);
        if (scale) {
          s = top > 0.f ? __fdiv_rn(top, 448.f) : 1.f;
          if (m == 0) scale[token * heads + h] = s;
        }
      }
      if (p.mass && step == quads && lane == 0) p.mass[token] = 0.f;
      if (!on) continue;
      const long long at = (token * heads + h) * dim;
      if (coded) {
        uint8_t* to = (kind == 1 ? p.k_cache : kind == 2 ? p.v_cache : p.idx_cache) + at;
#pragma unroll
        for (int k = 0; k < 16; ++k) v.x[k] = __fdiv_rn(v.x[k], s);
        *reinterpret_cast<uint2*>(to + a) = make_uint2(e4m3x4(v.x[0], v.x[1], v.x[2], v.x[3]), e4m3x4(v.x[4], v.x[5], v.x[6], v.x[7]));
        *reinterpret_cast<uint2*>(to + c) = make_uint2(e4m3x4(v.x[8], v.x[9], v.x[10], v.x[11]), e4m3x4(v.x[12], v.x[13], v.x[14], v.x[15]));
        continue;
      }
      uint16_t* to;
      if (kind == 0) to = p.q_out + ((long long)r * H + h) * kHeadDim;
      else if (kind == 3) to = p.idx_q_out + ((long long)r * Hi + h) * Di;
      else to = reinterpret_cast<uint16_t*>(kind == 1 ? p.k_cache : kind == 2 ? p.v_cache : p.idx_cache) + at;
      *reinterpret_cast<uint4*>(to + a) = v.bf16(0);
      *reinterpret_cast<uint4*>(to + c) = v.bf16(8);
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

// Warps to a row: few rows are shared out, many are not, as each of a row's warps repeats
// its checks and brings its cosines.  us for 64, 304, 608, 1216, 2432, 4864, 9728 rows:
//   8 warps  4.6  4.8  5.1  8.9  15.8  28.6  57.2
//   2        5.9  5.9  5.9  6.7   8.5  14.4  30.1
//   1        7.1  7.1  7.0  7.3   8.7  12.2  22.8
cudaError_t launch_qk_rope_insert(const RopeLaunch& p, cudaStream_t stream) {
  const int n = p.batch.num_rows, sms = device_sm_count();
  if (n <= 4 * sms) return launch<8>(p, 1, stream);
  if (n <= 16 * sms) return launch<2>(p, 4, stream);
  // (whole waves of four CTAs an SM, of at most 8 rows a warp)
  const int waves = (int)((n + 4ll * sms * 8 * kWarps - 1) / (4ll * sms * 8 * kWarps));
  return launch<1>(p, (int)((n + 4ll * sms * waves - 1) / (4ll * sms * waves)), stream);
}

}  // namespace msa
