// Matrix product in 8-bit integers with one scale per token and one per output channel,
// on 5th-generation tensor cores (tcgen05 + TMEM):
//
//   acc[m][n] = sum_k W[n][k] * X[m][k]                    int8 x int8, int32: exact
//   y[m][n]   = RN(RN(float(acc) * x_scale[m]) * w_scale[n])
//
// and, for SwiGLU, h[m][f] = silu(y[m][f]) * y[m][F + f] with F = N / 2, rounded to bf16.
// Because the sums are exact, the result does not depend on tiles, splits or their order.
//
// The weights are the MMA's A operand (128 weight rows = 128 TMEM lanes) and the tokens
// its B operand (NT <= 256 of them = NT TMEM columns): a few tokens then cost a narrow MMA
// instead of a mostly empty 128-row tile, and a thread of the epilogue owns one output
// channel, so a warp stores 32 neighbouring channels of a token at once, whatever N is.
//   warp 0     TMA producer: 128 bytes of K of the weight and token tiles per stage
//              (128-byte swizzle; rows and columns past the ends arrive as zeros).
//   warp 1     allocates TMEM; one lane issues tcgen05.mma kind::i8 (N=NT, K=32).
//   warps 2-9  epilogue: tcgen05.ld, scales, store; two warps per TMEM quadrant, taking the
//              token columns 16 at a time in turn.
// A CTA walks tiles with two accumulators, so that a tile's epilogue runs under the next
// one's MMAs.
// PAIR: a CTA pair computes 256 weight rows x NT tokens with cta_group::2 (each CTA its 128
// rows and half of the token tile, which both read): a lone CTA has to pull (128 + NT) x 128
// bytes per stage from L2, more than the ~64 bytes a cycle that an SM gets while its MMAs
// take 2 NT cycles; a pair (128 + NT / 2) x 128. The odd CTA's copies signal the even CTA's
// barriers, whose MMA lane issues for both.
// SPLIT: with too few tiles for the GPU the CTAs (or pairs) of a cluster split K: every CTA
// sends each other one of its share of the token columns through distributed shared
// memory, and sums and stores its own share.
// Measured, in graphs of a few calls: 17408 x 5120 at 4096 tokens 245 us (2.98 POPS at the 1.6 GHz
// that the power cap leaves, tensor pipe 80% busy; lone CTAs 279); 34816 x 5120 with SwiGLU at 512
// tokens 68 us (2.7 POPS), at one token 29.5 us (6.0 TB/s, 92% of the measured copy rate); 5120 x
// 17408 at eight tokens 18.1 us (split over six CTAs; unsplit 40), at 300 tokens 29.7 us. Called one
// after the other for longer, the power cap lowers the clock of the products that keep the
// tensor pipe busy: 286, 82 and 35 us at 4096, 512 and 300 tokens.
// SwiGLU tiles hold 64 gate and the matching 64 up rows, 16 of each per warp's 32 lanes, so
// that one shuffle brings a gate and its up value together.
// Every wait is bounded; on expiry the kernel latches Q4K_ERR_DEVICE_TIMEOUT, stops all
// roles, drains its own copies (bounded), frees TMEM and returns.
#pragma once
#include "common.cuh"
#include "gemm_tc.cuh"

namespace q4k {

constexpr int kI8Rows = 128;       // weight rows of a tile
constexpr int kI8KB = 128;         // bytes of K per stage
constexpr int kI8MaxNT = 256;      // tokens of a tile
constexpr int kI8MaxStages = 12;
constexpr int kI8EpiWarps = 8;
constexpr int kI8Threads = 32 * (2 + kI8EpiWarps);
constexpr uint32_t kI8ATile = kI8Rows * kI8KB;
// |acc| <= 128 * 128 * K < 2^31
constexpr int kI8MaxK = 131056;
constexpr int kI8MaxRows = 0x7fffffff - 1023;  // M and N at most: tiles past the end stay in 32 bits

struct I8GemmParams {
  const float* xs;
  const float* ws;
  void* Y;
  int M, N, K;
  int nt;        // tokens per tile (a multiple of 16)
  int n_tiles;   // tiles along the weight rows
  int m_tiles;
  int stages;
  int ksplit;    // CTAs (pairs) of a cluster that split K (SPLIT)
  int tstride;   // TMEM columns between the two accumulators (a multiple of 32)
  int tmem_cols; // columns to allocate: two accumulators (SPLIT: one), a power of two
  int tail;      // shared-memory offset of barriers and scales
  int boxed;     // SwiGLU: the weights' map is make_tmap_gate_up's
};

// The 64 gate and 64 up rows of a SwiGLU tile as one 5-D box: for each 16 rows of the
// gate (coordinate r16 of 16-row groups), those and the 16 matching up rows.
__device__ __forceinline__ void tma_load_gate_up(uint32_t dst, const CUtensorMap* map, int x, int r16, int e,
                                                 uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(0), "r"(r16), "r"(e), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void umma_i8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The pair's MMA (see umma2_f16kind).
__device__ __forceinline__ void umma2_i8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Completion of the MMAs issued so far, signalled on the barrier at this offset in the
// CTAs of the cluster that `mask` names.
__device__ __forceinline__ void umma2_commit(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}

// As tma_load_2d / tma_load_gate_up, for a CTA of a pair: `bar` (a cluster address) may be the
// peer's.
__device__ __forceinline__ void tma2_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
      "[%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma2_load_gate_up(uint32_t dst, const CUtensorMap* map, int x, int r16, int e,
                                                  uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
      "[%1, {%2, %3, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(0), "r"(r16), "r"(e), "r"(bar)
      : "memory");
}

// silu(g) * u = g u a^2 / (1 + h^2), h = exp(-|g| / 2), a = 1 or, g < 0, h: for a result that is
// rounded to bf16. The argument of ex2 is off by |g| 2^-24, ex2 by 2^-22 and, below the normal
// numbers, half a step of 2^-149, the reciprocal (of 1 to 2) by 2^-23; h enters twice: together
// below (|g| + 8) 2^-22 of the result, 2^-15 for |g| < 90 and 2^-14 wherever the result is a normal
// number. That is down to g = -181, u being large: by halves, the exponential does not leave
// fp32's range before, as long as ex2 keeps subnormal results (flushing them saved nothing:
// 512 x 34816 x 5120 67.5 us both ways). (With expf, tokens and 64-bit offsets one by
// one, the epilogue of 128 x 256 sums took 12 us, longer than the MMAs of 5120 in K.)
// V of them at once, step by step: their latencies overlap.
template <int V>
__device__ __forceinline__ void i8_silu_mul(const float (&g)[V], const float (&u)[V], float (&out)[V]) {
  float h[V], r[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    asm volatile("ex2.approx.f32 %0, %1;" : "=f"(h[i]) : "f"(fabsf(g[i]) * -0.72134752f));  // -log2(e) / 2
#pragma unroll
  for (int i = 0; i < V; ++i) asm volatile("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[i]) : "f"(fmaf(h[i], h[i], 1.f)));
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float a = g[i] >= 0.f ? 1.f : h[i];
    out[i] = g[i] * (a * r[i]) * (a * u[i]);
  }
}

// Instruction descriptor of kind::i8: int32 accumulators (2), signed A and B (1), both
// K-major.
__host__ __device__ __forceinline__ uint32_t i8_idesc(int m, int nt) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(nt >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, int32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ void st_release_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.release.cluster.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_acquire_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.acquire.cluster.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_s32(uint32_t addr, int32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// A place in a ring of stages, and the parity of its pass (the roles' single threads pay
// for every instruction, so no division by the runtime stage count).
struct I8Ring {
  int s = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      parity ^= 1;
    }
  }
};

template <bool BF16>
__device__ __forceinline__ void i8_store(uint8_t* at, float v) {
  if (BF16)
    *reinterpret_cast<__nv_bfloat16*>(at) = __float2bfloat16_rn(v);
  else
    *reinterpret_cast<float*>(at) = v;
}

// The output channel (row of W) that lane `lane` of TMEM quadrant q holds in a tile: its
// index within gate or up rows for SwiGLU (`up` set for the latter).
template <bool SWIGLU>
__device__ __forceinline__ int i8_row(int n_tile, int q, int lane, bool* up) {
  if (!SWIGLU) {
    *up = false;
    return n_tile * kI8Rows + 32 * q + lane;
  }
  *up = lane >= 16;
  return n_tile * (kI8Rows / 2) + 16 * q + (lane & 15);
}

template <bool SWIGLU, bool BF16, bool PAIR, bool SPLIT>
__global__ void __launch_bounds__(kI8Threads, 2)
i8_gemm_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x, I8GemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int P = PAIR ? 2 : 1;
  const uint32_t stage_bytes = kI8ATile + (uint32_t)(p.nt / P) * kI8KB;

  // barriers; full and tempty of a pair are the even CTA's
  const uint32_t bars = sbase + (uint32_t)p.tail;
  auto bar_full = [&](int s) { return bars + 8u * s; };
  auto bar_empty = [&](int s) { return bars + 8u * (kI8MaxStages + s); };
  auto bar_tfull = [&](int a) { return bars + 8u * (2 * kI8MaxStages + a); };
  auto bar_tempty = [&](int a) { return bars + 8u * (2 * kI8MaxStages + 2 + a); };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + p.tail + 8 * (2 * kI8MaxStages + 4));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + p.tail + 8 * (2 * kI8MaxStages + 4) + 4);
  const uint32_t bar_done = bars + 8u * (2 * kI8MaxStages + 5);    // issued MMAs have ended (on expiry)
  const uint32_t odd_issued = bars + 8u * (2 * kI8MaxStages + 6);  // stages that a pair's odd CTA has issued, plus 1
  float* s_xs = reinterpret_cast<float*>(smem + p.tail + 256);  // [epilogue warps][nt] token scales

  // place in the cluster: ranks P s + r: half r of the pair, share s of K
  const int csize = SPLIT ? P * p.ksplit : P;
  const int rank = (int)(blockIdx.x % (unsigned)csize);
  const int r = rank % P, ks = rank / P;
  const uint32_t leader = (uint32_t)(rank - r);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar_tfull(a), 1);
      mbar_init(bar_tempty(a), P * kI8EpiWarps);
    }
    mbar_init(bar_done, 1);
    *abort_flag = 0;
    if (PAIR) asm volatile("st.shared::cta.u32 [%0], %1;" ::"r"(odd_issued), "r"(0u) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    const uint32_t slot = smem_u32(const_cast<uint32_t*>(tmem_slot)), cols = (uint32_t)p.tmem_cols;
    if (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncwarp();
  if (PAIR)
    cluster_barrier();  // the peer's barriers and TMEM are ready too
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // everything above ran under the previous kernel; its results are read from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // SPLIT: one tile per cluster, this CTA's share of K; else the CTA's (pair's) tiles, all of K
  const int tiles = p.n_tiles * p.m_tiles;
  const int first = (int)(blockIdx.x / (unsigned)csize);
  const int step = SPLIT ? tiles : (int)(gridDim.x / (unsigned)P);
  const int nk_all = (p.K + kI8KB - 1) / kI8KB;
  const int k0 = SPLIT ? (int)((int64_t)nk_all * ks / p.ksplit) : 0;
  const int nk = SPLIT ? (int)((int64_t)nk_all * (ks + 1) / p.ksplit) - k0 : nk_all;  // >= 1
  const int half = p.N / 2;
  const uint64_t limit = *const_cast<volatile unsigned long long*>(&g_wait_limit_ns);
  // a tile's first token and this CTA's tile of weight rows
  auto tile_m0 = [&](int tile) { return tile % p.m_tiles * p.nt; };
  auto tile_n = [&](int tile) { return tile / p.m_tiles * P + r; };

  int issued = 0;  // by a role's one thread: stages copied (warp 0), consumed (warp 1)
  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      const int drop = g_test_drop_stage;  // test hook; -1 in normal use
      I8Ring at;
      bool ok = true;
      for (int tile = first; tile < tiles && ok; tile += step) {
        const int m0 = tile_m0(tile) + r * (p.nt / P), nti = tile_n(tile);
        for (int k = 0; k < nk; ++k, ++issued, at.next(p.stages)) {
          const int s = at.s;
          // (a barrier's phase before its first counts as complete)
          if (!(ok = mbar_wait_l(bar_empty(s), at.parity ^ 1, abort_flag, limit))) break;
          if (issued == drop) continue;  // test hook: this stage never arrives
          if (r == 0) mbar_arrive_expect_tx(bar_full(s), P * stage_bytes);
          const uint32_t a_dst = sbase + s * stage_bytes;
          const uint32_t bar = PAIR ? cluster_addr(bar_full(s), leader) : bar_full(s);
          const int x = (k0 + k) * kI8KB;
          auto load = [&](uint32_t dst, const CUtensorMap* map, int y) {
            if (PAIR)
              tma2_load_2d(dst, map, x, y, bar);
            else
              tma_load_2d(dst, map, x, y, bar);
          };
          if (SWIGLU && p.boxed) {
            if (PAIR)
              tma2_load_gate_up(a_dst, &tmap_w, x, nti * 4, 0, bar);
            else
              tma_load_gate_up(a_dst, &tmap_w, x, nti * 4, 0, bar);
          } else if (SWIGLU) {
            const int f0 = nti * (kI8Rows / 2);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              load(a_dst + (uint32_t)(32 * q) * kI8KB, &tmap_w, f0 + 16 * q);
              load(a_dst + (uint32_t)(32 * q + 16) * kI8KB, &tmap_w, half + f0 + 16 * q);
            }
          } else {
            load(a_dst, &tmap_w, nti * kI8Rows);
          }
          load(a_dst + kI8ATile, &tmap_x, m0);
        }
      }
      if (PAIR && r == 1) st_release_cluster_u32(cluster_addr(odd_issued, leader), (uint32_t)issued + 1u);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (of a pair: the even CTA's) ----------------
    if (lane == 0 && r == 0) {
      const uint32_t idesc = i8_idesc(P * kI8Rows, p.nt);
      const uint16_t both = (uint16_t)(3u << leader);
      int done = 0;
      I8Ring at;
      bool ok = true;
      for (int tile = first; tile < tiles && ok; tile += step, ++done) {
        const int a = done & 1;
        if (done >= 2) {
          ok = PAIR ? mbar_wait_cluster(bar_tempty(a), (done / 2 - 1) & 1, abort_flag)
                    : mbar_wait_l(bar_tempty(a), (done / 2 - 1) & 1, abort_flag, limit);
          if (!ok) break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(a * p.tstride);
        for (int k = 0; k < nk; ++k, at.next(p.stages)) {
          if (!(ok = mbar_wait_l(bar_full(at.s), at.parity, abort_flag, limit))) break;
          tc_fence_after();
          const uint32_t a0 = sbase + at.s * stage_bytes;
          const uint64_t ad = umma_desc_sw128(a0), bd = umma_desc_sw128(a0 + kI8ATile);
#pragma unroll
          for (int kk = 0; kk < kI8KB / 32; ++kk) {  // 32 bytes of K on: 2 in the descriptors' units
            if (PAIR)
              umma2_i8(d, ad + 2 * kk, bd + 2 * kk, idesc, (k | kk) != 0);
            else
              umma_i8(d, ad + 2 * kk, bd + 2 * kk, idesc, (k | kk) != 0);
          }
          ++issued;
          if (PAIR)
            umma2_commit(bar_empty(at.s), both);
          else
            umma_commit(bar_empty(at.s));
        }
        if (ok && PAIR) umma2_commit(bar_tfull(a), both);
        if (ok && !PAIR) umma_commit(bar_tfull(a));
      }
    }
  } else if (!SPLIT) {
    // ---------------- epilogue ----------------
    const int q = warp & 3, turn = (warp - 2) >> 2;
    int done = 0;
    const int rows = SWIGLU ? half : p.N;
    constexpr int kOut = BF16 ? 2 : 4;
    const int64_t pitch = (int64_t)rows * kOut;
    float* xs = s_xs + (warp - 2) * p.nt;  // a copy per warp: no barrier between warps, which may stop apart
    for (int tile = first; tile < tiles; tile += step, ++done) {
      const int a = done & 1;
      const int m0 = tile_m0(tile);
      const int mcount = min(p.nt, p.M - m0);
      for (int i = lane; i < p.nt; i += 32) xs[i] = i < mcount ? p.xs[m0 + i] : 0.f;
      bool up;
      const int n = i8_row<SWIGLU>(tile_n(tile), q, lane, &up);
      const float w = n < rows ? p.ws[up ? half + n : n] : 0.f;
      uint8_t* col = static_cast<uint8_t*>(p.Y) + (int64_t)n * kOut;  // the channel's outputs, a pitch apart
      __syncwarp();
      if (!__all_sync(0xffffffffu, mbar_wait_l(bar_tfull(a), (done / 2) & 1, abort_flag, limit))) break;
      tc_fence_after();
      const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * p.tstride);
      for (int c = 16 * turn; c < mcount; c += 16 * (kI8EpiWarps / 4)) {
        int32_t v[16];
        tmem_ld16(d + c, v);
        if (SWIGLU) {
          // lanes of the gate finish the even tokens, those of up the odd ones
          float g[8], u[8];
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(xs + c + i);
            const float y[4] = {(float)v[i] * x.x * w, (float)v[i + 1] * x.y * w, (float)v[i + 2] * x.z * w,
                                (float)v[i + 3] * x.w * w};
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              const float got = __shfl_xor_sync(0xffffffffu, up ? y[j] : y[j + 1], 16);
              g[(i + j) / 2] = up ? got : y[j];
              u[(i + j) / 2] = up ? y[j + 1] : got;
            }
          }
          float hv[8];
          i8_silu_mul(g, u, hv);
          if (n < rows) {
            const int left = mcount - c - (up ? 1 : 0);  // tokens from this lane's first on
            uint8_t* at = col + (m0 + c + (up ? 1 : 0)) * pitch;
#pragma unroll
            for (int i = 0; i < 8; ++i, at += 2 * pitch)
              if (2 * i < left) i8_store<BF16>(at, hv[i]);
          }
        } else if (n < rows) {
          uint8_t* at = col + (m0 + c) * pitch;
          float y[16];
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(xs + c + i);
            y[i] = (float)v[i] * x.x * w, y[i + 1] = (float)v[i + 1] * x.y * w;
            y[i + 2] = (float)v[i + 2] * x.z * w, y[i + 3] = (float)v[i + 3] * x.w * w;
          }
          if (c + 16 <= mcount) {
#pragma unroll
            for (int i = 0; i < 16; ++i, at += pitch) i8_store<BF16>(at, y[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i, at += pitch)
              if (c + i < mcount) i8_store<BF16>(at, y[i]);
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR)
          mbar_arrive_remote(bar_tempty(a), leader);
        else
          mbar_arrive(bar_tempty(a));
      }
    }
  }

  if constexpr (SPLIT) {
    // ---------------- reduction over the CTAs that share the tile's rows ----------------
    const int m0 = tile_m0(first), nti = tile_n(first);
    const int mcount = min(p.nt, p.M - m0);
    const int per = ((p.nt + p.ksplit - 1) / p.ksplit + 3) / 4 * 4;  // token columns that a CTA sums and stores
    // [ksplit][per][128]: the stages are free by then. A warp sends 32 neighbouring rows of a
    // column, 128 bytes in a row: peers' shared memory takes about a request every 3 cycles
    // whatever its size (16 bytes of a row at a time: 300 x 5120 x 17408 spent 10 us here)
    int32_t* part = reinterpret_cast<int32_t*>(smem);
    const int q = warp & 3, turn = (warp - 2) >> 2;
    bool ok = true;
    // the row that this thread sums, and its scales, asked for early
    constexpr int kCols = SWIGLU ? 64 : 128, kStep = 32 * kI8EpiWarps / kCols * 4;
    const int et = threadIdx.x - 64, n = nti * kCols + et % kCols;
    const bool in = et >= 0 && n < (SWIGLU ? half : p.N);
    const float w = in ? p.ws[n] : 0.f, wu = SWIGLU && in ? p.ws[half + n] : 0.f;
    if (warp >= 2) {
      for (int i = threadIdx.x - 64; i < mcount; i += 32 * kI8EpiWarps) s_xs[i] = p.xs[m0 + i];
      ok = __all_sync(0xffffffffu, mbar_wait_l(bar_tfull(0), 0, abort_flag, limit));
    }
    __syncwarp();
    cluster_barrier();  // no CTA's MMAs read its stages any more
    if (warp >= 2 && ok) {
      tc_fence_after();
      const uint32_t d = tmem + ((uint32_t)(q * 32) << 16);
      const uint32_t mine = sbase + (uint32_t)(ks * per * kI8Rows + 32 * q + lane) * 4u;
      int to = 16 * turn / per, left = 16 * turn % per;  // whose column comes next, and where in the share
      for (int c = 16 * turn; c < mcount; c += 16 * (kI8EpiWarps / 4)) {
        int32_t v[16];
        tmem_ld16(d + c, v);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          if (c + i < mcount) {
            const uint32_t at = cluster_addr(mine + (uint32_t)(left * kI8Rows) * 4u, (uint32_t)(P * to + r));
#pragma unroll
            for (int j = 0; j < 4; ++j) st_cluster_s32(at + (uint32_t)(j * kI8Rows) * 4u, v[i + j]);
          }
          if ((left += 4) >= per) left -= per, ++to;
        }
        for (left += 16 * (kI8EpiWarps / 4 - 1); left >= per; left -= per) ++to;
      }
      tc_fence_before();
    }
    __syncwarp();
    cluster_barrier();
    if (warp >= 2 && ok) {
      const int c0 = ks * per, c1 = min(per, mcount - c0);  // this CTA's columns of the tile
      auto sum = [&](int c, int row, float (&y)[4]) {
        int32_t t[4] = {0, 0, 0, 0};
        const int32_t* from = part + c * kI8Rows + row;
#pragma unroll 4
        for (int s = 0; s < p.ksplit; ++s, from += per * kI8Rows) {
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] += from[i * kI8Rows];
        }
        const float4 x = *reinterpret_cast<const float4*>(s_xs + c0 + c);  // (past mcount: no one's)
        y[0] = (float)t[0] * x.x, y[1] = (float)t[1] * x.y, y[2] = (float)t[2] * x.z, y[3] = (float)t[3] * x.w;
      };
      if (in) {
        constexpr int kOut = BF16 ? 2 : 4;
        const int64_t pitch = (int64_t)(SWIGLU ? half : p.N) * kOut;
        const int first_c = et / kCols * 4;
        uint8_t* at = static_cast<uint8_t*>(p.Y) + (m0 + c0 + first_c) * pitch + (int64_t)n * kOut;
        const int row = SWIGLU ? 32 * (et % 64 / 16) + et % 16 : et % 128;
        for (int c = first_c; c < c1; c += kStep, at += kStep * pitch) {
          float y[4], u[4] = {};
          sum(c, row, y);
          if (SWIGLU) sum(c, row + 16, u);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] *= w, u[i] *= wu;
          float out[4];
          if (SWIGLU) i8_silu_mul(y, u, out);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i < c1) i8_store<BF16>(at + i * pitch, SWIGLU ? out[i] : y[i]);
        }
      }
    }
  }

  // ---- teardown ----
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  // Where a wait has expired, this CTA's copies and MMAs may be under way still (on the normal
  // path the MMAs have waited for the copies, and the epilogue for the MMAs, of both CTAs of a
  // pair): they end before anything is freed. The even CTA sees to the pair's.
  if (*abort_flag && r == 0) {
    if (warp == 0 && lane == 0) {
      const int drop = g_test_drop_stage;
      auto drain = [&](int from, int to, bool odd_only) {
        for (int i = max(from, 0); i < to; ++i) {
          if (i == drop) continue;
          if (odd_only) mbar_arrive_expect_tx(bar_full(i % p.stages), stage_bytes);
          mbar_wait_drain(bar_full(i % p.stages), (uint32_t)(i / p.stages) & 1u);
        }
      };
      drain(issued - p.stages, issued, false);
      if (PAIR) {  // stages of which the odd CTA alone has issued its half
        const uint64_t t0 = global_timer_ns();
        uint32_t odd;
        // (it gives up a limit later than this one at most; waits look at the time every millisecond)
        while ((odd = ld_acquire_cluster_u32(odd_issued)) == 0u && global_timer_ns() - t0 < limit + 5000000u) {}
        drain(issued, (int)odd - 1, true);
      }
    }
    if (warp == 1 && lane == 0 && issued) {
      if (PAIR)
        umma2_commit(bar_done, (uint16_t)(1u << leader));
      else
        umma_commit(bar_done);
      mbar_wait_drain(bar_done, 0);
    }
    __syncwarp();
    __syncthreads();
  }
  if (PAIR) cluster_barrier();  // neither CTA leaves while the pair's MMAs, copies or arrivals may touch it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)p.tmem_cols) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)p.tmem_cols) : "memory");
  }
}

// ---- host side ----------------------------------------------------------------------

// int8 [rows][K], box 128 bytes of K x box_rows, 128-byte swizzle.
inline bool make_tmap_i8(CUtensorMap* m, const void* base, int64_t rows, int K, int box_rows) {
  auto enc = get_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)K};
  cuuint32_t box[2] = {(cuuint32_t)kI8KB, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// int8 gate and up rows [E][2][F][K], F % 16 == 0, viewed as [E][F / 16][2][16][K]: one box
// is 4 groups of 16 gate rows, each followed by the 16 matching up rows. (Sixteen-row boxes,
// eight of them per stage, kept the one producing thread busy for ~700 cycles a stage.)
inline bool make_tmap_gate_up(CUtensorMap* m, const void* base, int E, int F, int K) {
  auto enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t k = (cuuint64_t)K, f = (cuuint64_t)F;
  cuuint64_t dims[5] = {k, 16, 2, f / 16, (cuuint64_t)E};
  cuuint64_t strides[4] = {k, f * k, 16 * k, 2 * f * k};
  cuuint32_t box[5] = {(cuuint32_t)kI8KB, 16, 2, 4, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace q4k
