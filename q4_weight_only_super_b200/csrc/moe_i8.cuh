// A whole mixture-of-experts layer for a few tokens over int8 expert weights (one fp32
// scale per output channel), in two kernels:
//
//   p_tj, e_tj = softmax over the top-k logits of token t, and their experts
//   h_tj       = silu(g) * u,  g, u = s_gate_up[e] * (W_gate_up[e] X_t)      (kernel 1)
//   Y_t        = residual_t + sum_j p_tj * s_down[e] * (W_down[e] h_tj)      (kernel 2)
//
// A few tokens select experts whose weights are each read for one or two rows: the weight
// bytes bound the layer, so the activations stay bf16 (nothing would be saved by 8-bit
// ones) and the weights go from global memory into registers in long contiguous runs, are
// converted there to bf16 (exact) and multiplied by mma.sync m16n8k16 with fp32 sums.
//
//  * MMA operands without shuffles: K may be permuted as long as both operands agree, so
//    lane (g, i) of a warp takes 16 contiguous bytes of weight row g, k = 64c + 16i .., as
//    its A fragments of four MMAs, and the same 16 activations of token g as its B ones.
//  * Kernel 1: a unit is 8 gate rows and the 8 matching up rows of one expert (an MMA's 16
//    rows, so a gate and its up value meet in one lane) times up to 8 of its tokens. Units
//    go round-robin over the CTAs; the four warps of a CTA split K.
//  * h leaves kernel 1 as three bf16 planes (h = h0 + h1 + h2, 8 of
//    its 24 bits each, exact); kernel 2 adds three MMAs into the same sums.
//  * Kernel 2: a CTA owns 16 output columns and runs over all experts that were selected,
//    so the combine needs no exchange between CTAs and no atomics: each warp adds its
//    experts' rows, weighted, to its own sums in shared memory, which are added in warp
//    order at the end. The result is deterministic.
//  * Routing (a warp per token) runs in every CTA of kernel 1; CTA 0 leaves the list of
//    (expert, rows) groups and the rows' tokens and weights for kernel 2.
#pragma once
#include "common.cuh"
#include "gemm_tc.cuh"
#include "moe.cuh"

namespace q4k {

constexpr int kMi8MaxM = 32;
constexpr int kMi8MaxRows = kMi8MaxM * kMaxTopk;  // (token, slot) pairs
constexpr int kMi8Warps1 = 4;   // kernel 1: warps of a CTA, splitting K
constexpr int kMi8Warps2 = 16;  // kernel 2: warps of a CTA, splitting the experts
constexpr int kMi8Batch = 8;    // 64-wide pieces of K that a lane holds in registers

// The plan that kernel 1 leaves for kernel 2 at the start of the workspace.
struct Mi8Plan {
  int32_t groups;
  int32_t pad[3];
  int32_t group_expert[kMi8MaxRows];  // a group: up to 8 rows of one expert
  int32_t group_row[kMi8MaxRows];     // its first row | number of rows << 16
  int32_t row_token[kMi8MaxRows];     // rows sorted by (expert, token)
  float row_weight[kMi8MaxRows];
};

struct Mi8Params {
  const float* logits;
  const int8_t* Wgu;
  const float* sgu;
  const int8_t* Wd;
  const float* sd;
  const uint16_t* X;
  const float* residual;  // may be null; may be Y
  float* Y;
  Mi8Plan* plan;
  uint16_t* h;  // [rows][3][F] bf16
  int M, E, topk, H, F;
};

inline size_t mi8_ws_bytes(int M, int topk, int F) {
  return ((sizeof(Mi8Plan) + 255) & ~(size_t)255) + (size_t)M * topk * 3 * (size_t)F * 2;
}

// Order of the logits as unsigned keys: -inf .. +inf, a NaN below them all, 0 for none.
__device__ __forceinline__ uint32_t mi8_key(float v) { return v != v ? 1u : order_key(v); }

// Top-k of one token by a whole warp: lane j < topk returns the j-th expert (higher logit
// first, equal logits by the lower id) and its softmax weight over the selected ones.
template <int PL>
__device__ __forceinline__ void mi8_topk(const float* __restrict__ row, int E, int topk, int lane, int* id, float* w) {
  uint32_t key[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = i * 32 + lane;
    key[i] = e < E ? mi8_key(row[e]) : 0u;
  }
  uint32_t my_key = 0;
  *id = 0;
  for (int k = 0; k < topk; ++k) {
    uint32_t best = 0;
    int bi = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (key[i] > best) {
        best = key[i];
        bi = i;
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const uint32_t e = __reduce_min_sync(0xffffffffu, best == top ? (uint32_t)(bi * 32 + lane) : 0xffffffffu);
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (e == (uint32_t)(i * 32 + lane)) key[i] = 0;
    if (lane == k) {
      my_key = top;
      *id = (int)e;
    }
  }
  const float v = my_key == 1u ? __uint_as_float(0x7FC00000u) : key_value(my_key);
  const float v0 = __shfl_sync(0xffffffffu, v, 0);
  const float ek = lane < topk ? expf(v - v0) : 0.f;
  float den = ek;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  *w = ek / den;
}

// Four int8 of a word to four bf16, exact: with b = q + 128 in the low mantissa bits of
// 0x43xx the value is 256 + q for q < 0 and 2q + 256 otherwise (the top bit of b reaches the
// exponent); less 256 that is q, or 2q, and the smaller of it and its half is q.
__device__ __forceinline__ void i8x4_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t b = w ^ 0x80808080u;
  const uint32_t p0 = __byte_perm(b, 0x43434343u, 0x4140), p1 = __byte_perm(b, 0x43434343u, 0x4342);
  const __nv_bfloat162 c = __floats2bfloat162_rn(256.f, 256.f), half = __floats2bfloat162_rn(0.5f, 0.5f);
  const __nv_bfloat162 g0 = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&p0), c);
  const __nv_bfloat162 g1 = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&p1), c);
  const __nv_bfloat162 r0 = __hmin2(g0, __hmul2(g0, half)), r1 = __hmin2(g1, __hmul2(g1, half));
  lo = *reinterpret_cast<const uint32_t*>(&r0);
  hi = *reinterpret_cast<const uint32_t*>(&r1);
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One 64-wide piece of K: A from rows g (u) and g + 8 (v) of 16 bytes a lane, B planes.
template <int PLANES>
__device__ __forceinline__ void mi8_piece(float (&acc)[4], const uint4& u, const uint4& v, const uint4 (&b)[PLANES][2]) {
  const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t a0, a1, a2, a3;
    i8x4_bf16(uw[j], a0, a2);
    i8x4_bf16(vw[j], a1, a3);
#pragma unroll
    for (int pl = PLANES - 1; pl >= 0; --pl) {
      const uint4& q = b[pl][j >> 1];
      mma_bf16(acc, a0, a1, a2, a3, j & 1 ? q.z : q.x, j & 1 ? q.w : q.y);
    }
  }
}

__device__ __forceinline__ uint4 zero4() { return make_uint4(0u, 0u, 0u, 0u); }

template <int PL>
__global__ void __launch_bounds__(32 * kMi8Warps1, 4)
mi8_gate_up_kernel(Mi8Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ unsigned tmask[32 * PL];          // tokens that selected expert e
  __shared__ int s_id[kMi8MaxRows];            // [token][slot]
  __shared__ float s_w[kMi8MaxRows];
  __shared__ int start[32 * PL];               // expert's first row
  __shared__ int g_expert[kMi8MaxRows], g_row[kMi8MaxRows];
  __shared__ int s_token[kMi8MaxRows];         // row -> token
  __shared__ int s_groups;
  __shared__ float red[2][kMi8Warps1][16][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  // ---- routing: who goes where ----
  for (int e = threadIdx.x; e < 32 * PL; e += blockDim.x) tmask[e] = 0u;
  __syncthreads();
  for (int t = warp; t < p.M; t += kMi8Warps1) {
    int id;
    float w;
    mi8_topk<PL>(p.logits + (int64_t)t * p.E, p.E, p.topk, lane, &id, &w);
    if (lane < p.topk) {
      s_id[t * p.topk + lane] = id;
      s_w[t * p.topk + lane] = w;
      atomicOr(&tmask[id], 1u << t);
    }
  }
  __syncthreads();
  if (warp == 0) {  // groups of up to 8 rows, experts in order
    int rows = 0, groups = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int c = __popc(tmask[e0 + lane]), n = (c + 7) / 8;
      int rc = c, rn = n;  // inclusive scans
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, rc, o), b = __shfl_up_sync(0xffffffffu, rn, o);
        if (lane >= o) {
          rc += a;
          rn += b;
        }
      }
      start[e0 + lane] = rows + rc - c;
      for (int i = 0; i < n; ++i) {
        g_expert[groups + rn - n + i] = e0 + lane;
        g_row[groups + rn - n + i] = (rows + rc - c + 8 * i) | min(8, c - 8 * i) << 16;
      }
      rows += __shfl_sync(0xffffffffu, rc, 31);
      groups += __shfl_sync(0xffffffffu, rn, 31);
    }
    if (lane == 0) s_groups = groups;
  }
  __syncthreads();
  const int groups = s_groups;
  for (int f = threadIdx.x; f < p.M * p.topk; f += blockDim.x) {
    const int t = f / p.topk, e = s_id[f];
    const int row = start[e] + __popc(tmask[e] & ((1u << t) - 1u));
    s_token[row] = t;
    if (blockIdx.x == 0) {
      p.plan->row_token[row] = t;
      p.plan->row_weight[row] = s_w[f];
    }
  }
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < groups; i += blockDim.x) {
      p.plan->group_expert[i] = g_expert[i];
      p.plan->group_row[i] = g_row[i];
    }
    if (threadIdx.x == 0) p.plan->groups = groups;
  }
  __syncthreads();

  // ---- units: (group, 8 gate rows + 8 up rows) ----
  const int tiles = p.F / 8;
  const int units = groups * tiles;
  const int g = lane >> 2, i4 = lane & 3;
  const int pieces = (p.H + 63) / 64;                      // 64-wide pieces of K
  const int pairs = (pieces + 1) / 2;                      // the warps take 128-byte pairs in turn
  const int batches = (pairs + kMi8Warps1 * (kMi8Batch / 2) - 1) / (kMi8Warps1 * (kMi8Batch / 2));
  uint4 au[kMi8Batch], av[kMi8Batch];
  // k offset of this lane's 16 values of piece j of batch b
  auto kof = [&](int b, int j) { return (((b * (kMi8Batch / 2) + (j >> 1)) * kMi8Warps1 + warp) * 2 + (j & 1)) * 64 + 16 * i4; };
  auto rows_of = [&](int u) {
    const int grp = u / tiles, f0 = (u % tiles) * 8;
    return p.Wgu + ((int64_t)g_expert[grp] * 2 * p.F + f0 + g) * p.H;
  };
  auto load = [&](const int8_t* w, int b, int j) {
    const int k = kof(b, j);
    au[j] = k < p.H ? ldg_stream_u4(w + k) : zero4();
    av[j] = k < p.H ? ldg_stream_u4(w + (int64_t)p.F * p.H + k) : zero4();
  };
  int u = blockIdx.x, buf = 0;
  if (u < units) {
    const int8_t* w = rows_of(u);
#pragma unroll
    for (int j = 0; j < kMi8Batch; ++j) load(w, 0, j);
  }
  for (; u < units; u += gridDim.x, buf ^= 1) {
    const int grp = u / tiles, f0 = (u % tiles) * 8;
    const int row0 = g_row[grp] & 0xFFFF, nrows = g_row[grp] >> 16, e = g_expert[grp];
    const uint16_t* x = p.X + (int64_t)(g < nrows ? s_token[row0 + g] : 0) * p.H;
    const int un = u + gridDim.x;
    const int8_t* w_cur = rows_of(u);
    const int8_t* w_next = un < units ? rows_of(un) : nullptr;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int b = 0; b < batches; ++b) {
      const bool last = b + 1 == batches;
#pragma unroll
      for (int j = 0; j < kMi8Batch; ++j) {
        const int k = kof(b, j);
        uint4 bx[1][2];
        const bool in = g < nrows && k < p.H;
        bx[0][0] = in ? __ldg(reinterpret_cast<const uint4*>(x + k)) : zero4();
        bx[0][1] = in ? __ldg(reinterpret_cast<const uint4*>(x + k + 8)) : zero4();
        mi8_piece<1>(acc, au[j], av[j], bx);
        if (!last)
          load(w_cur, b + 1, j);
        else if (w_next)
          load(w_next, 0, j);
      }
    }
    float(*r)[8] = red[buf][warp];
    r[g][2 * i4] = acc[0];
    r[g][2 * i4 + 1] = acc[1];
    r[g + 8][2 * i4] = acc[2];
    r[g + 8][2 * i4 + 1] = acc[3];
    __syncthreads();
    if (threadIdx.x < 64) {  // (f, row): 8 neighbouring threads write 8 neighbouring f
      const int f = threadIdx.x & 7, c = threadIdx.x >> 3;
      if (c < nrows) {
        float gs = 0.f, us = 0.f;
#pragma unroll
        for (int wv = 0; wv < kMi8Warps1; ++wv) {
          gs += red[buf][wv][f][c];
          us += red[buf][wv][f + 8][c];
        }
        const float* s = p.sgu + (int64_t)e * 2 * p.F + f0 + f;
        const float hv = silu_mul(gs * s[0], us * s[p.F]);
        uint16_t* h = p.h + (int64_t)(row0 + c) * 3 * p.F + f0 + f;
        float rest = hv;
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) {
          // truncated, so that 3 x 8 bits hold all 24 of h and the first plane cannot overflow
          const __nv_bfloat16 b = __float2bfloat16_rz(rest);
          h[(int64_t)pl * p.F] = __bfloat16_as_ushort(b);
          rest = isfinite(hv) ? rest - __bfloat162float(b) : 0.f;  // inf, NaN: the first plane alone
        }
      }
    }
  }
}

__global__ void __launch_bounds__(32 * kMi8Warps2, 1)
mi8_down_kernel(Mi8Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float sums[kMi8Warps2][kMi8MaxM][16 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, i4 = lane & 3;
  const int n0 = blockIdx.x * 16;
  for (int i = lane; i < kMi8MaxM * 17; i += 32) (&sums[warp][0][0])[i] = 0.f;
  __syncwarp();
  const int groups = p.plan->groups;
  const int pieces = (p.F + 63) / 64;
  // items: (group, part of K); parts > 1 only when there are fewer groups than warps
  const int parts = groups >= kMi8Warps2 ? 1 : max(1, min(kMi8Warps2 / max(groups, 1), pieces));
  for (int it = warp; it < groups * parts; it += kMi8Warps2) {
    const int grp = it / parts, part = it % parts;
    const int e = p.plan->group_expert[grp], gr = p.plan->group_row[grp];
    const int row0 = gr & 0xFFFF, nrows = gr >> 16;
    const int c0 = pieces * part / parts, c1 = pieces * (part + 1) / parts;
    const int8_t* w = p.Wd + ((int64_t)e * p.H + n0 + g) * p.F;
    const uint16_t* h = p.h + (int64_t)(row0 + min(g, nrows - 1)) * 3 * p.F;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int cb = c0; cb < c1; cb += kMi8Batch) {
      uint4 au[kMi8Batch], av[kMi8Batch];
#pragma unroll
      for (int j = 0; j < kMi8Batch; ++j) {
        const int k = (cb + j) * 64 + 16 * i4;
        const bool in = cb + j < c1 && k < p.F;
        au[j] = in ? ldg_stream_u4(w + k) : zero4();
        av[j] = in ? ldg_stream_u4(w + 8 * (int64_t)p.F + k) : zero4();
      }
#pragma unroll
      for (int j = 0; j < kMi8Batch; ++j) {
        if (cb + j >= c1) break;
        const int k = (cb + j) * 64 + 16 * i4;
        uint4 b[3][2];
        const bool in = g < nrows && k < p.F;
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) {
          b[pl][0] = in ? *reinterpret_cast<const uint4*>(h + (int64_t)pl * p.F + k) : zero4();
          b[pl][1] = in ? *reinterpret_cast<const uint4*>(h + (int64_t)pl * p.F + k + 8) : zero4();
        }
        mi8_piece<3>(acc, au[j], av[j], b);
      }
    }
    const float s0 = p.sd[(int64_t)e * p.H + n0 + g], s1 = p.sd[(int64_t)e * p.H + n0 + g + 8];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = 2 * i4 + c;
      if (r < nrows) {
        const int t = p.plan->row_token[row0 + r];
        const float pw = p.plan->row_weight[row0 + r];
        sums[warp][t][g] += pw * (s0 * acc[c]);
        sums[warp][t][g + 8] += pw * (s1 * acc[2 + c]);
      }
    }
    __syncwarp();
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.M * 16; i += blockDim.x) {
    const int t = i >> 4, n = i & 15;
    float y = 0.f;
    for (int wv = 0; wv < kMi8Warps2; ++wv) y += sums[wv][t][n];
    const int64_t at = (int64_t)t * p.H + n0 + n;
    p.Y[at] = p.residual ? p.residual[at] + y : y;
  }
}

}  // namespace q4k
