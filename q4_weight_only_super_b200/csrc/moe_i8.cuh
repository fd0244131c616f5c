// A whole mixture-of-experts layer for a few tokens over int8 expert weights (one fp32
// scale per output channel), in two kernels:
//
//   p_tj, e_tj = softmax over the top-k logits of token t, and their experts
//   h_tj       = silu(g) * u,  g, u = s_gate_up[e] * (W_gate_up[e] X_t)      (kernel 1)
//   Y_t        = residual_t + sum_j p_tj * s_down[e] * (W_down[e] h_tj)      (kernel 2)
//
// A few tokens select experts whose weights are each read for one or two rows, so the
// layer is bound by reading the weights, and nothing would be saved by activations of 8
// bits. But the tensor cores take int8 weights as they are only with int8 activations:
// a row of activations is therefore held as 24-bit fixed point, one scale per row, in three
// signed base-256 digits, each a column of its own in the MMA:
//   x = v / S,  v = rint(x S) = 65536 d0 + 256 d1 + d2,
//   W x = (65536 (W d0) + 256 (W d1) + W d2) / S     with int32 sums, exact.
// That keeps what fp32 sums would (X: S is a power of two, so a bf16 value within 2^14 of
// its row's largest is exact; h: to 2^-23 of its row's largest), costs no instruction per
// weight, and makes the sums independent of their order.
// Measured (128 experts, top-8, H = 2048, F = 768): 19.9 / 59.5 / 115 us for 1 / 8 / 32 tokens,
// 1.9 / 4.1 / 4.6 TB/s of the weights that have to be read; the streams themselves run at 5.5 to
// 5.9 TB/s, the rest is routing, the hand-over between the kernels and the last sums. mma.sync
// kernels that converted the weights to bf16 in registers took 26 / 90 / 188 us, bound by
// ~100 to 180 instructions per KB of weights and by latency.
//   warp 0      TMA producer: 128 weight rows x 128 bytes of K per stage (128-byte swizzle).
//   warp 1      TMEM; one lane issues tcgen05.mma kind::i8 (M=128, N = 4 columns per row of
//               activations: three digits and one that nobody reads, rounded up to 16).
//   warps 2-5   epilogue: a thread owns a weight row (output channel).
//   warps 6-9   digits: each takes every fourth stage, reads the rows' 128 activations from
//               L2 and writes their digits in the layout that the MMA reads.
// Kernel 1: a unit is one expert's 64 gate and the matching 64 up rows (16 of each per warp
// of the epilogue, one shuffle brings a pair together); units go round-robin over the CTAs.
// h leaves as fp32 with the largest magnitude of every 16 of a row. Kernel 2: a CTA owns
// 128 output columns and every split-th group: the weighted rows are summed in shared
// memory, and the CTAs of a column tile, one cluster's, add theirs in a fixed order through
// distributed shared memory (no atomics on results: deterministic).
// Both kernels know the whole routing: each cluster routes the tokens, a warp
// per token, and shares what it finds; kernel 2 then starts its weight stream before kernel
// 1 has ended (programmatic dependent launch) and waits for it only before it reads h.
// Every wait is bounded; on expiry the kernel latches Q4K_ERR_DEVICE_TIMEOUT, stops all
// roles, drains its own copies (bounded), frees TMEM and returns.
#pragma once
#include "common.cuh"
#include "gemm_tc.cuh"
#include "i8_gemm.cuh"
#include "moe.cuh"

namespace q4k {

constexpr int kMi8MaxM = 32;
constexpr int kMi8MaxRows = kMi8MaxM * kMaxTopk;  // (token, slot) pairs
constexpr int kMi8Warps = 10;
constexpr int kMi8DigitWarps = 4;
constexpr int kMi8Cluster[2] = {4, 8};  // CTAs of a cluster, which share the routing (kernel 1, 2)
constexpr int kMi8GroupRows = 8;  // rows of a group at most
constexpr int kMi8MaxStages = 10;
constexpr float kMi8Top = 8355711.f;  // 127 * 65536 + 127 * 256 + 127: the largest three digits hold

struct Mi8Params {
  const float* logits;
  const float* sgu;
  const float* sd;
  const uint16_t* X;
  const float* residual;  // may be null; may be Y
  float* Y;
  float* h;        // [rows][F], rows sorted by (expert, token)
  uint32_t* hmax;  // [rows][hparts]: bits of the largest |h| of each 16
  int M, E, topk, H, F;
  int hparts;  // 4 per tile of kernel 1
  int nb;      // columns that a stage has room for: 4 per row of a group, rounded up to 16
  int stages, tstride, tmem_cols;
  int split;   // kernel 2: CTAs that share a column tile, taking the experts in turn: 1, 2, 4, 8
};

inline int mi8_tiles(int F) { return (F + 63) / 64; }

// h, hmax
inline size_t mi8_ws_h(int M, int topk, int F) { return (size_t)M * topk * F * 4; }
inline size_t mi8_ws_bytes(int M, int topk, int F) {
  return mi8_ws_h(M, topk, F) + (size_t)M * topk * 16 * (size_t)mi8_tiles(F);
}

// Order of the logits as unsigned keys: -inf .. +inf, a NaN below them all, 0 for none.
__device__ __forceinline__ uint32_t mi8_key(float v) { return v != v ? 1u : order_key(v); }

// Top-k of one token by a whole warp, from PL logits per lane (expert 32 i + lane) as keys:
// the j-th expert (higher logit first, equal logits by the lower id) goes to id[j], its key
// to keys[j]. Ranks are counted, not found round by round (a round of warp-wide reductions
// measured ~380 cycles): the topk-th largest of the 32 lanes' own maxima bounds the topk-th
// key of all from below, the few keys that reach it are collected, and each of them counts
// those before it. list: room for 32 PL entries of this warp's own, 16-byte aligned.
template <int PL>
__device__ __forceinline__ void mi8_topk(const uint32_t (&key)[PL], int topk, int lane, uint64_t* list, uint16_t* id,
                                         uint32_t* keys) {
  uint32_t m = key[0];
#pragma unroll
  for (int i = 1; i < PL; ++i) m = max(m, key[i]);
  // distinct, and off by less than the 5 bits that the bound gives away below
  m = (m & ~31u) | (31u - lane);
  uint32_t* maxima = reinterpret_cast<uint32_t*>(list);
  maxima[lane] = m;
  __syncwarp();
  int rank = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint4 o = reinterpret_cast<const uint4*>(maxima)[j];
    rank += (o.x > m) + (o.y > m) + (o.z > m) + (o.w > m);
  }
  const uint32_t bound = __shfl_sync(0xffffffffu, m, __ffs(__ballot_sync(0xffffffffu, rank == topk - 1)) - 1) & ~31u;
  int count = 0;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const bool in = key[i] != 0 && key[i] >= bound;
    const unsigned who = __ballot_sync(0xffffffffu, in);  // (also: every lane has read the maxima)
    if (in) list[count + __popc(who & ((1u << lane) - 1u))] = (uint64_t)key[i] << 32 | (0xffffffffu - (32 * i + lane));
    count += __popc(who);
  }
  __syncwarp();
  for (int c = lane; c < count; c += 32) {
    const uint64_t mine = list[c];
    int before = 0;
    // (the list is in the order of the ids: among many equal logits topk steps decide)
    for (int j = 0; j < count && before < topk; ++j) before += list[j] > mine;
    if (before < topk) {
      id[before] = (uint16_t)(0xffffffffu - (uint32_t)mine);
      keys[before] = (uint32_t)(mine >> 32);
    }
  }
  __syncwarp();
}

// Scale of a row whose largest magnitude has these bits, and 1 / scale; a row of zeros: 0
// and 0; a row with an infinity or a NaN: 0 and NaN, so that its products are NaN.
// TWO: a power of two (0.25 .. 0.5 of the digits' range).
template <bool TWO>
__device__ __forceinline__ float2 mi8_scale(uint32_t bits) {
  if (bits >= 0x7F800000u) return make_float2(0.f, __uint_as_float(0x7FC00000u));
  if (bits == 0) return make_float2(0.f, 0.f);
  if (TWO) {
    // amax in [2^e, 2^(e+1)): S = 2^(21 - e), kept normal (below 2^-105 the digits lose range, no more)
    const int e = max((int)(bits >> 23) - 127, -105);
    const int s = min(21 - e, 126);
    return make_float2(__uint_as_float((uint32_t)(127 + s) << 23), __uint_as_float((uint32_t)(127 - s) << 23));
  }
  const float amax = fmaxf(__uint_as_float(bits), 0x1p-100f);
  return make_float2(kMi8Top / amax, amax / kMi8Top);
}

// The routing of all tokens, as every CTA of both kernels holds it: rows sorted by
// (expert, token), cut into groups of up to kMi8GroupRows rows of one expert.
template <int PL>
struct Mi8Route {
  unsigned tmask[32 * PL];   // tokens that selected expert e
  uint16_t start[32 * PL];   // e's first row
  uint16_t id[kMi8MaxRows];  // [token][slot]
  uint32_t w[kMi8MaxRows];   // the logits' keys, then the weights' bits
  uint16_t group_expert[kMi8MaxRows];
  int group_row[kMi8MaxRows];  // first row | number of rows << 16
  uint16_t row_token[kMi8MaxRows];
  float row_weight[kMi8MaxRows];
  int groups;
};

// Stores to, and an OR into, the variable at this place in the shared memory of CTA `rank`
// of the cluster.
__device__ __forceinline__ uint32_t map_cluster(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void st_cluster(uint32_t* p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_cluster(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint16_t* p, uint32_t rank, uint16_t v) {
  asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(map_cluster(p, rank)), "h"(v) : "memory");
}
__device__ __forceinline__ void or_cluster(unsigned* p, uint32_t rank, unsigned v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.or.b32 %0, [%1], %2;" : "=r"(old) : "r"(map_cluster(p, rank)), "r"(v) : "memory");
}

// Every CTA needs the whole routing, but were every CTA to read all logits (and, for their
// scales, all of X), 148 SMs would ask a few L2 slices for the same lines: 6 us for 32
// tokens of 128 experts, and as much for X. So the CTAs of a cluster route a share of the
// tokens each, a warp per token, and write what they find into each other's shared memory.
// SCALES: also the tokens' scales into `scale`. scratch: 32 PL entries of 8 bytes per warp.
// The masks are cleared, and that is known to the whole cluster, before.
template <int PL, int C, bool SCALES>
__device__ __forceinline__ void mi8_route(const Mi8Params& p, Mi8Route<PL>& r, float2* scale, uint8_t* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)(blockIdx.x % C);
  uint64_t* list = reinterpret_cast<uint64_t*>(scratch) + warp * 32 * PL;
#pragma unroll 1
  for (int t = rank + C * warp; t < p.M; t += C * kMi8Warps) {
    uint32_t key[PL];
#pragma unroll
    for (int j = 0; j < PL; ++j) key[j] = 32 * j + lane < p.E ? mi8_key(__ldcg(p.logits + (int64_t)t * p.E + 32 * j + lane)) : 0u;
    uint16_t* id = r.id + t * p.topk;
    uint32_t* w = r.w + t * p.topk;
    mi8_topk<PL>(key, p.topk, lane, list, id, w);
    // softmax over the selected: lane j has the j-th, the sum in a fixed butterfly order
    const uint32_t k = w[min(lane, p.topk - 1)], k0 = w[0];
    // a NaN logit weighs nothing, as -inf does; with nothing but NaN, v0 is NaN
    const float v = k == 1u ? -INFINITY : key_value(k), v0 = k0 == 1u ? __uint_as_float(0x7FC00000u) : key_value(k0);
    const float ek = lane < p.topk ? expf(v - v0) : 0.f;
    float den = ek;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (lane < p.topk) {
      const uint16_t e = id[lane];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        st_cluster(id + lane, c, e);
        st_cluster(w + lane, c, __float_as_uint(ek / den));
        or_cluster(&r.tmask[e], c, 1u << t);
      }
    }
  }
  if (SCALES) {  // by other warps than route the tokens, as far as there are
#pragma unroll 1
    for (int t = rank + C * ((warp + kMi8Warps / 2) % kMi8Warps); t < p.M; t += C * kMi8Warps) {
      uint32_t m = 0;
#pragma unroll 8
      for (int k = 8 * lane; k < p.H; k += 256) {
        const uint4 x = ldg_u4(p.X + (int64_t)t * p.H + k);
        m = __vmaxu2(__vmaxu2(m, __vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu)),
                     __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
      }
      const float2 sc = mi8_scale<true>(__reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16)) << 16);
      if (lane < C) {
        st_cluster(reinterpret_cast<uint32_t*>(&scale[t].x), lane, __float_as_uint(sc.x));
        st_cluster(reinterpret_cast<uint32_t*>(&scale[t].y), lane, __float_as_uint(sc.y));
      }
    }
  }
  __syncwarp();
  cluster_barrier();
  // rows and groups: a thread per expert, each warp 32 of them
  for (int e0 = 32 * warp; e0 < 32 * PL; e0 += 32 * kMi8Warps) {
    // those of the experts before e0, counted anew by each warp
    int c0 = 0;
    for (int e = lane; e < e0; e += 32) {
      const int c = __popc(r.tmask[e]);
      c0 += c | (c + kMi8GroupRows - 1) / kMi8GroupRows << 16;
    }
    c0 = (int)__reduce_add_sync(0xffffffffu, (unsigned)c0);
    const int c = __popc(r.tmask[e0 + lane]), n = (c + kMi8GroupRows - 1) / kMi8GroupRows;
    int sum = c | n << 16;  // inclusive scan of both
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += a;
    }
    sum += c0;
    const int row = (sum & 0xFFFF) - c, grp = (sum >> 16) - n;
    r.start[e0 + lane] = (uint16_t)row;
    for (int i = 0; i < n; ++i) {
      r.group_expert[grp + i] = (uint16_t)(e0 + lane);
      r.group_row[grp + i] = (row + kMi8GroupRows * i) | min(kMi8GroupRows, c - kMi8GroupRows * i) << 16;
    }
    if (e0 == 32 * PL - 32 && lane == 31) r.groups = grp + n;
  }
  __syncthreads();
  for (int f = threadIdx.x; f < p.M * p.topk; f += 32 * kMi8Warps) {
    const int t = f / p.topk, e = r.id[f];
    const int at = r.start[e] + __popc(r.tmask[e] & ((1u << t) - 1u));
    r.row_token[at] = (uint16_t)t;
    r.row_weight[at] = __uint_as_float(r.w[f]);
  }
  fence_async_smem();  // the scratch becomes stages of bulk copies
  __syncthreads();
}

// Digits of four values: byte i of word d is digit d (0 the highest) of value i.
__device__ __forceinline__ void mi8_digits(const float (&x)[4], float S, uint32_t (&d)[3]) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int q = __float2int_rn(fminf(fmaxf(x[i] * S, -kMi8Top), kMi8Top));
    v[i] = ((uint32_t)q + 0x00808080u) ^ 0x00808080u;  // bytes 2, 1, 0: the signed digits
  }
  const uint32_t a = __byte_perm(v[0], v[1], 0x5140), b = __byte_perm(v[2], v[3], 0x5140);  // digits 2, 1 of two values
  d[2] = __byte_perm(a, b, 0x5410);
  d[1] = __byte_perm(a, b, 0x7632);
  d[0] = __byte_perm(__byte_perm(v[0], v[1], 0x0062), __byte_perm(v[2], v[3], 0x0062), 0x5410);
}

// silu(g) * u = g u a^2 / (1 + h^2), h = exp(-|g| / 2), a = 1 or, g < 0, h. A row of h has a scale of
// its own, so what counts is the product: exp(-|g|) is 0 or has lost bits from g = -87 down,
// where a large u still makes a normal number of it; its half is whole down to g = -174.
__device__ __forceinline__ float mi8_silu_mul(float g, float u) {
  const float h = expf(-0.5f * fabsf(g));
  const float a = g >= 0.f ? 1.f : h;
  return g * (a * __frcp_rn(fmaf(h, h, 1.f))) * (a * u);
}

__device__ __forceinline__ float4 ld_cluster_f4(const float* p, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(map_cluster(p, rank))
               : "memory");
  return v;
}

template <int PL, bool DOWN>
__global__ void __launch_bounds__(32 * kMi8Warps, 2)
mi8_kernel(const __grid_constant__ CUtensorMap tmap_w, Mi8Params p) {
  constexpr int C = kMi8Cluster[DOWN];
  extern __shared__ uint8_t smem_raw[];
  __shared__ Mi8Route<PL> r;
  __shared__ __align__(8) uint64_t bar_mem[3 * kMi8MaxStages + 5];
  // scale and its inverse: kernel 1 of each token, kernel 2 of each row of h
  __shared__ float2 s_scale[DOWN ? kMi8MaxRows : kMi8MaxM];
  __shared__ uint32_t tmem_slot_mem;
  __shared__ int abort_mem;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t stage_bytes = kI8ATile + (uint32_t)p.nb * kI8KB;
  float* ysum = reinterpret_cast<float*>(smem + p.stages * stage_bytes);  // kernel 2: [M][128]
  const uint32_t bars = smem_u32(bar_mem);
  auto bar_a = [&](int s) { return bars + 8u * s; };                        // weights landed
  auto bar_b = [&](int s) { return bars + 8u * (kMi8MaxStages + s); };      // digits written
  auto bar_empty = [&](int s) { return bars + 8u * (2 * kMi8MaxStages + s); };
  auto bar_tfull = [&](int a) { return bars + 8u * (3 * kMi8MaxStages + a); };
  auto bar_tempty = [&](int a) { return bars + 8u * (3 * kMi8MaxStages + 2 + a); };
  const uint32_t bar_done = bars + 8u * (3 * kMi8MaxStages + 4);  // issued MMAs have ended (on expiry)
  volatile int* abort_flag = &abort_mem;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar_a(s), 1);
      mbar_init(bar_b(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar_tfull(a), 1);
      mbar_init(bar_tempty(a), 4);
    }
    mbar_init(bar_done, 1);
    abort_mem = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot_mem)),
                 "r"((uint32_t)p.tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // Kernel 1 reads its inputs after the kernel before it; kernel 2 starts once every CTA of
  // kernel 1 has got past this wait, so the logits are complete for it already.
  for (int e = threadIdx.x; e < 32 * PL; e += blockDim.x) r.tmask[e] = 0u;
  if (!DOWN) {
    // this warp's tokens into L2 (a prefetch may precede the wait: it returns nothing, and L2
    // is where the kernel before this one writes)
    for (int t = (int)(blockIdx.x % C) + C * warp; t < p.M; t += C * kMi8Warps)
      for (int i = 32 * lane; i < p.E; i += 32 * 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.logits + (int64_t)t * p.E + i));
    for (int t = (int)(blockIdx.x % C) + C * warp; t < p.M; t += C * kMi8Warps)
      for (int i = 64 * lane; i < p.H; i += 64 * 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.X + (int64_t)t * p.H + i));
  }
  __syncwarp();
  cluster_barrier();  // the masks are clear in the whole cluster
  if (!DOWN) asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  mi8_route<PL, C, !DOWN>(p, r, s_scale, smem);  // (barriers within: the set-up above is visible after it)
  tc_fence_after();
  const uint32_t tmem = tmem_slot_mem;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // this CTA's units: (group, tile of weight rows)
  const int K = DOWN ? p.F : p.H;
  const int nk = (K + kI8KB - 1) / kI8KB;
  const int tiles = (p.F + 63) / 64;  // kernel 1
  const int first = DOWN ? (int)(blockIdx.x % (unsigned)p.split) : (int)blockIdx.x;
  const int col0 = DOWN ? (int)(blockIdx.x / (unsigned)p.split) * kI8Rows : 0;  // (past H: a spare CTA of the last cluster)
  int units = DOWN ? (col0 < p.H ? r.groups : 0) : r.groups * tiles;
  // Kernel 1 leaves CTAs out so that all finish in the same round: DRAM bounds it, and a last
  // round of a few CTAs would wait for their latency (3 us at 8 and at 32 tokens).
  const int grid = (int)gridDim.x, rounds = (units + grid - 1) / grid;
  const int step = DOWN ? p.split : (units + max(rounds, 1) - 1) / max(rounds, 1);
  if (!DOWN && first >= step) units = 0;
  auto group_of = [&](int u) { return DOWN ? u : u / tiles; };
  // scale of row j of a group that starts at row0
  auto row_scale = [&](int row0, int j) { return s_scale[DOWN ? row0 + j : r.row_token[row0 + j]]; };
  auto columns = [&](int u) { return (4 * (r.group_row[group_of(u)] >> 16) + 15) / 16 * 16; };

  const uint64_t limit = *const_cast<volatile unsigned long long*>(&g_wait_limit_ns);
  int issued = 0;  // by a role's one thread: stages copied (warp 0), consumed (warp 1)
  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      const int drop = g_test_drop_stage;  // test hook; -1 in normal use
      I8Ring at;
      bool ok = true;
      for (int u = first; u < units && ok; u += step) {
        const int e = r.group_expert[group_of(u)];
        for (int k = 0; k < nk; ++k, ++issued, at.next(p.stages)) {
          const int s = at.s;
          // (a barrier's phase before its first counts as complete)
          if (!(ok = mbar_wait_l(bar_empty(s), at.parity ^ 1, abort_flag, limit))) break;
          if (issued == drop) continue;  // test hook: this stage never arrives
          mbar_arrive_expect_tx(bar_a(s), kI8ATile);
          const uint32_t a_dst = sbase + s * stage_bytes;
          if (DOWN) {
            tma_load_2d(a_dst, &tmap_w, k * kI8KB, e * p.H + col0, bar_a(s));
          } else {
            tma_load_gate_up(a_dst, &tmap_w, k * kI8KB, u % tiles * 4, e, bar_a(s));
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      int done = 0;
      I8Ring at;
      bool ok = true;
      for (int u = first; u < units && ok; u += step, ++done) {
        const int a = done & 1;
        if (done >= 2 && !(ok = mbar_wait_l(bar_tempty(a), (done / 2 - 1) & 1, abort_flag, limit))) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(a * p.tstride);
        const uint32_t idesc = i8_idesc(kI8Rows, columns(u));
        for (int k = 0; k < nk; ++k, at.next(p.stages)) {
          if (!(ok = mbar_wait_l(bar_b(at.s), at.parity, abort_flag, limit) &&
                     mbar_wait_l(bar_a(at.s), at.parity, abort_flag, limit)))
            break;
          tc_fence_after();
          const uint32_t a0 = sbase + at.s * stage_bytes;
          const uint64_t ad = umma_desc_sw128(a0), bd = umma_desc_sw128(a0 + kI8ATile);
#pragma unroll
          for (int kk = 0; kk < kI8KB / 32; ++kk)  // 32 bytes of K on: 2 in the descriptors' units
            umma_i8(d, ad + 2 * kk, bd + 2 * kk, idesc, (k | kk) != 0);
          ++issued;
          umma_commit(bar_empty(at.s));
        }
        if (ok) umma_commit(bar_tfull(a));
      }
    }
  } else if (warp < 6) {
    // ---------------- epilogue ----------------
    const int q = warp & 3;
    if (DOWN)
      for (int t = 0; t < p.M; ++t) ysum[t * kI8Rows + 32 * q + lane] = 0.f;  // this thread's column
    int done = 0;
    for (int u = first; u < units; u += step, ++done) {
      const int a = done & 1;
      const int e = r.group_expert[group_of(u)], gr = r.group_row[group_of(u)];
      const int row0 = gr & 0xFFFF, rows = gr >> 16;
      const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * p.tstride);
      const int tile = DOWN ? 0 : u % tiles;
      bool up = lane >= 16;
      const int f = tile * 64 + 16 * q + (lane & 15);  // kernel 1
      const int n = col0 + 32 * q + lane;              // kernel 2
      float w = 0.f;
      if (DOWN) {
        if (n < p.H) w = p.sd[(int64_t)e * p.H + n];
      } else if (f < p.F) {
        w = p.sgu[(int64_t)e * 2 * p.F + (up ? p.F : 0) + f];
      }
      if (!__all_sync(0xffffffffu, mbar_wait_l(bar_tfull(a), (done / 2) & 1, abort_flag, limit))) break;
      tc_fence_after();
      const float inv = lane < rows ? row_scale(row0, lane).y : 0.f;  // (written before the digits)
      for (int j = 0; j < rows; j += 4) {
        int32_t v[16];
        tmem_ld16(d + 4 * j, v);
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float back = __shfl_sync(0xffffffffu, inv, min(j + i, rows - 1));
          y[i] = fmaf((float)v[4 * i], 65536.f, fmaf((float)v[4 * i + 1], 256.f, (float)v[4 * i + 2])) * back * w;
        }
        if (DOWN) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // (a masked expert weighs 0 and stays out, whatever it holds: 0 times a NaN would not)
            const float p_tj = j + i < rows ? r.row_weight[row0 + j + i] : 0.f;
            if (p_tj != 0.f) ysum[r.row_token[row0 + j + i] * kI8Rows + 32 * q + lane] += p_tj * y[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, up ? y[i] : y[i + 1], 16);
            const float hv = up ? mi8_silu_mul(got, y[i + 1]) : mi8_silu_mul(y[i], got);
            const int rj = j + i + (up ? 1 : 0);
            const bool in = rj < rows && f < p.F;
            uint32_t m = in ? __float_as_uint(hv) & 0x7FFFFFFFu : 0u;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (in) p.h[(int64_t)(row0 + rj) * p.F + f] = hv;
            if (rj < rows && (lane & 15) == 0) p.hmax[(int64_t)(row0 + rj) * p.hparts + tile * 4 + q] = m;
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_tempty(a));
    }
  } else {
    // ---------------- digits ----------------
    const int me = warp - 6;
    // first the rows' scales (the weights' stream is under way)
    if (DOWN) {
      asm volatile("griddepcontrol.wait;" ::: "memory");  // h is kernel 1's
      // 16 of this CTA's groups at a time, 8 threads a group
      for (int u = first + (threadIdx.x - 6 * 32) / 8 * step; u < units; u += 4 * kMi8DigitWarps * step) {
        const int row0 = r.group_row[u] & 0xFFFF, rows = r.group_row[u] >> 16;
        for (int j = threadIdx.x % 8; j < rows; j += 8) {
          const uint4* part = reinterpret_cast<const uint4*>(p.hmax + (int64_t)(row0 + j) * p.hparts);
          uint32_t m = 0;
#pragma unroll 12
          for (int i = 0; i < p.hparts / 4; ++i) {
            const uint4 h = __ldcg(part + i);
            m = max(max(m, max(h.x, h.y)), max(h.z, h.w));
          }
          s_scale[row0 + j] = mi8_scale<false>(m);
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kMi8DigitWarps) : "memory");
    }
    int turn = 0;  // whose stage it is
    I8Ring ring;
    bool ok = true;
    for (int u = first; u < units && ok; u += step) {
      const int gr = r.group_row[group_of(u)], row0 = gr & 0xFFFF, rows = gr >> 16;
      const float scale = lane < rows ? row_scale(row0, lane).x : 0.f;  // lane j: row j's
      for (int k = 0; k < nk; ++k, turn = (turn + 1) % kMi8DigitWarps, ring.next(p.stages)) {
        if (turn != me) continue;
        const int s = ring.s;
        // (parity tells passes apart as long as a warp is never two passes ahead of the
        // MMAs: with at least kMi8DigitWarps stages, its last stage came after them)
        if (!(ok = __all_sync(0xffffffffu, mbar_wait_l(bar_empty(s), ring.parity ^ 1, abort_flag, limit)))) break;
        uint8_t* b = smem + s * stage_bytes + kI8ATile;
        const int at = k * kI8KB + 4 * lane;
        for (int j0 = 0; j0 < rows; j0 += 4) {
          float x[4][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = row0 + min(j0 + j, rows - 1);
            if (DOWN) {
              const float4 t = at < K ? __ldcg(reinterpret_cast<const float4*>(p.h + (int64_t)row * p.F + at))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
              x[j][0] = t.x, x[j][1] = t.y, x[j][2] = t.z, x[j][3] = t.w;
            } else {
              const uint2 t = at < K ? __ldg(reinterpret_cast<const uint2*>(p.X + (int64_t)r.row_token[row] * p.H + at))
                                     : make_uint2(0u, 0u);
              x[j][0] = __uint_as_float(t.x << 16), x[j][1] = __uint_as_float(t.x & 0xFFFF0000u);
              x[j][2] = __uint_as_float(t.y << 16), x[j][3] = __uint_as_float(t.y & 0xFFFF0000u);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float S = __shfl_sync(0xffffffffu, scale, min(j0 + j, rows - 1));
            if (j0 + j < rows) {
              uint32_t dg[3];
              mi8_digits(x[j], S, dg);
#pragma unroll
              for (int c = 0; c < 3; ++c)
                *reinterpret_cast<uint32_t*>(b + sw128_offset(4 * (j0 + j) + c, lane >> 2) + 4 * (lane & 3)) = dg[c];
            }
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_b(s));
      }
    }
  }

  // ---- teardown; kernel 2 first sums over the cluster ----
  tc_fence_before();
  __syncthreads();
  // Where a wait has expired, copies and MMAs may be under way still (on the normal path the MMAs
  // have waited for the copies, and the epilogue for the MMAs): they end before anything is freed.
  if (*abort_flag) {
    if (warp == 0 && lane == 0) {
      const int drop = g_test_drop_stage;
      for (int i = max(0, issued - p.stages); i < issued; ++i)
        if (i != drop) mbar_wait_drain(bar_a(i % p.stages), (uint32_t)(i / p.stages) & 1u);
    }
    if (warp == 1 && lane == 0 && issued) {
      umma_commit(bar_done);
      mbar_wait_drain(bar_done, 0);
    }
    __syncwarp();
    __syncthreads();
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)p.tmem_cols)
                 : "memory");
  }
  if constexpr (DOWN) {
    // The CTAs of a column tile lie in one cluster; each finishes a share of the tile's sums,
    // adding its peers' in their order.
    __syncwarp();
    cluster_barrier();  // every CTA's sums are complete
    const uint32_t peer0 = (uint32_t)(blockIdx.x % C - first);
    for (int i = 4 * (first * (int)blockDim.x + (int)threadIdx.x); i < p.M * kI8Rows; i += 4 * p.split * (int)blockDim.x) {
      const int t = i / kI8Rows, c = col0 + i % kI8Rows;
      if (c >= p.H) continue;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int q = 0; q < p.split; ++q) {
        const float4 v = ld_cluster_f4(ysum + i, peer0 + q);
        y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
      }
      const int64_t at = (int64_t)t * p.H + c;  // (H % 16 == 0: four columns are in or out together)
      if (p.residual) {
        const float4 v = *reinterpret_cast<const float4*>(p.residual + at);
        y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
      }
      *reinterpret_cast<float4*>(p.Y + at) = y;
    }
    __syncwarp();
    cluster_barrier();  // no CTA leaves while its sums are read
  }
}

}  // namespace q4k
