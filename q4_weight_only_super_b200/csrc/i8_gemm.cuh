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
//   warp 1     allocates TMEM; one lane issues tcgen05.mma kind::i8 (M=128, N=NT, K=32).
//   warps 2-5  epilogue: tcgen05.ld, scales, store.
// A CTA walks tiles with two accumulators, so that a tile's epilogue runs under the next
// one's MMAs. With too few tiles for the GPU a cluster of up to eight CTAs splits K
// (SPLIT): every CTA sends each peer that peer's share of the token columns through
// distributed shared memory, and sums and stores its own share.
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
constexpr int kI8Threads = 192;
constexpr uint32_t kI8ATile = kI8Rows * kI8KB;
// |acc| <= 128 * 128 * K < 2^31
constexpr int kI8MaxK = 131056;

struct I8GemmParams {
  const float* xs;
  const float* ws;
  void* Y;
  int M, N, K;
  int nt;        // tokens per tile (a multiple of 16)
  int n_tiles;   // tiles along the weight rows
  int m_tiles;
  int stages;
  int csplit;    // CTAs of a cluster that split K (SPLIT)
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

// Instruction descriptor of kind::i8: int32 accumulators (2), signed A and B (1), both
// K-major, M = 128, N = nt.
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

__device__ __forceinline__ void st_cluster_s32(uint32_t saddr, uint32_t rank, int32_t v) {
  asm volatile(
      "{\n .reg .b32 ra;\n mapa.shared::cluster.u32 ra, %0, %1;\n"
      " st.shared::cluster.b32 [ra], %2;\n}" ::"r"(saddr),
      "r"(rank), "r"(v)
      : "memory");
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
__device__ __forceinline__ void i8_store(void* Y, int64_t at, float v) {
  if (BF16)
    static_cast<__nv_bfloat16*>(Y)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(Y)[at] = v;
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

template <bool SWIGLU, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(kI8Threads)
i8_gemm_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x, I8GemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t stage_bytes = kI8ATile + (uint32_t)p.nt * kI8KB;

  const uint32_t bars = sbase + (uint32_t)p.tail;
  auto bar_full = [&](int s) { return bars + 8u * s; };
  auto bar_empty = [&](int s) { return bars + 8u * (kI8MaxStages + s); };
  auto bar_tfull = [&](int a) { return bars + 8u * (2 * kI8MaxStages + a); };
  auto bar_tempty = [&](int a) { return bars + 8u * (2 * kI8MaxStages + 2 + a); };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + p.tail + 8 * (2 * kI8MaxStages + 4));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + p.tail + 8 * (2 * kI8MaxStages + 4) + 4);
  float* s_xs = reinterpret_cast<float*>(smem + p.tail + 256);  // [4 warps][kI8MaxNT] token scales

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar_tfull(a), 1);
      mbar_init(bar_tempty(a), 4);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(const_cast<uint32_t*>(tmem_slot))), "r"((uint32_t)p.tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // everything above ran under the previous kernel; its results are read from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // SPLIT: one tile per cluster, this CTA's share of K; else this CTA's tiles, all of K
  const int tiles = p.n_tiles * p.m_tiles;
  const int rank = SPLIT ? (int)(blockIdx.x % (unsigned)p.csplit) : 0;
  const int first = SPLIT ? (int)(blockIdx.x / (unsigned)p.csplit) : (int)blockIdx.x;
  const int step = SPLIT ? tiles : (int)gridDim.x;
  const int nk_all = (p.K + kI8KB - 1) / kI8KB;
  const int k0 = SPLIT ? (int)((int64_t)nk_all * rank / p.csplit) : 0;
  const int nk = SPLIT ? (int)((int64_t)nk_all * (rank + 1) / p.csplit) - k0 : nk_all;  // >= 1
  const int half = p.N / 2;
  const uint64_t limit = *const_cast<volatile unsigned long long*>(&g_wait_limit_ns);

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      const int drop = g_test_drop_stage;  // test hook; -1 in normal use
      int it = 0;
      I8Ring at;
      bool ok = true;
      for (int tile = first; tile < tiles && ok; tile += step) {
        const int m0 = tile % p.m_tiles * p.nt, nti = tile / p.m_tiles;
        for (int k = 0; k < nk; ++k, ++it, at.next(p.stages)) {
          const int s = at.s;
          // (a barrier's phase before its first counts as complete)
          if (!(ok = mbar_wait_l(bar_empty(s), at.parity ^ 1, abort_flag, limit))) break;
          if (it == drop) continue;  // test hook: this stage never arrives
          mbar_arrive_expect_tx(bar_full(s), stage_bytes);
          const uint32_t a_dst = sbase + s * stage_bytes;
          const int x = (k0 + k) * kI8KB;
          if (SWIGLU && p.boxed) {
            tma_load_gate_up(a_dst, &tmap_w, x, nti * 4, 0, bar_full(s));
          } else if (SWIGLU) {
            const int f0 = nti * (kI8Rows / 2);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              tma_load_2d(a_dst + (uint32_t)(32 * q) * kI8KB, &tmap_w, x, f0 + 16 * q, bar_full(s));
              tma_load_2d(a_dst + (uint32_t)(32 * q + 16) * kI8KB, &tmap_w, x, half + f0 + 16 * q, bar_full(s));
            }
          } else {
            tma_load_2d(a_dst, &tmap_w, x, nti * kI8Rows, bar_full(s));
          }
          tma_load_2d(a_dst + kI8ATile, &tmap_x, x, m0, bar_full(s));
        }
      }
      // every issued stage lands before this CTA may exit (on the normal path the MMA
      // role has waited for all of them)
      if (*abort_flag)
        for (int i = max(0, it - p.stages); i < it; ++i)
          if (i != drop) mbar_wait_drain(bar_full(i % p.stages), (i / p.stages) & 1);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      const uint32_t idesc = i8_idesc(kI8Rows, p.nt);
      int done = 0;
      I8Ring at;
      bool ok = true;
      for (int tile = first; tile < tiles && ok; tile += step, ++done) {
        const int a = done & 1;
        if (done >= 2 && !(ok = mbar_wait_l(bar_tempty(a), (done / 2 - 1) & 1, abort_flag, limit))) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(a * p.tstride);
        for (int k = 0; k < nk; ++k, at.next(p.stages)) {
          if (!(ok = mbar_wait_l(bar_full(at.s), at.parity, abort_flag, limit))) break;
          tc_fence_after();
          const uint32_t a0 = sbase + at.s * stage_bytes;
          const uint64_t ad = umma_desc_sw128(a0), bd = umma_desc_sw128(a0 + kI8ATile);
#pragma unroll
          for (int kk = 0; kk < kI8KB / 32; ++kk)  // 32 bytes of K on: 2 in the descriptors' units
            umma_i8(d, ad + 2 * kk, bd + 2 * kk, idesc, (k | kk) != 0);
          umma_commit(bar_empty(at.s));
        }
        if (ok) umma_commit(bar_tfull(a));
      }
    }
  } else if (!SPLIT) {
    // ---------------- epilogue ----------------
    const int q = warp & 3;
    int done = 0;
    const int64_t ldy = SWIGLU ? half : p.N;
    const int rows = SWIGLU ? half : p.N;
    for (int tile = first; tile < tiles; tile += step, ++done) {
      const int a = done & 1;
      const int m0 = tile % p.m_tiles * p.nt, nti = tile / p.m_tiles;
      const int mcount = min(p.nt, p.M - m0);
      float* xs = s_xs + q * kI8MaxNT;  // a copy per warp: no barrier between warps, which may stop apart
      for (int i = lane; i < p.nt; i += 32) xs[i] = i < mcount ? p.xs[m0 + i] : 0.f;
      bool up;
      const int r = i8_row<SWIGLU>(nti, q, lane, &up);
      const float w = r < rows ? p.ws[up ? half + r : r] : 0.f;
      __syncwarp();
      if (!__all_sync(0xffffffffu, mbar_wait_l(bar_tfull(a), (done / 2) & 1, abort_flag, limit))) break;
      tc_fence_after();
      const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * p.tstride);
      for (int c = 0; c < mcount; c += 16) {
        int32_t v[16];
        tmem_ld16(d + c, v);
        if (SWIGLU) {
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float y0 = (float)v[i] * xs[c + i] * w, y1 = (float)v[i + 1] * xs[c + i + 1] * w;
            const float got = __shfl_xor_sync(0xffffffffu, up ? y0 : y1, 16);
            const float hv = up ? silu_mul(got, y1) : silu_mul(y0, got);
            const int m = c + i + (up ? 1 : 0);
            if (m < mcount && r < rows) i8_store<BF16>(p.Y, (int64_t)(m0 + m) * ldy + r, hv);
          }
        } else if (r < rows) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c + i < mcount) i8_store<BF16>(p.Y, (int64_t)(m0 + c + i) * ldy + r, (float)v[i] * xs[c + i] * w);
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_tempty(a));
    }
  }

  if constexpr (SPLIT) {
    // ---------------- reduction over the cluster ----------------
    const int tile = first;
    const int m0 = tile % p.m_tiles * p.nt, nti = tile / p.m_tiles;
    const int mcount = min(p.nt, p.M - m0);
    const int per = (p.nt + p.csplit - 1) / p.csplit;  // token columns that a CTA sums and stores
    int32_t* part = reinterpret_cast<int32_t*>(smem);  // [csplit][per][128]: the stages are free by then
    const int q = warp & 3;
    bool ok = true;
    if (warp >= 2) ok = __all_sync(0xffffffffu, mbar_wait_l(bar_tfull(0), 0, abort_flag, limit));
    __syncwarp();
    cluster_barrier();  // no CTA's MMAs read its stages any more
    if (warp >= 2 && ok) {
      tc_fence_after();
      const uint32_t d = tmem + ((uint32_t)(q * 32) << 16);
      for (int c = 0; c < mcount; c += 16) {
        int32_t v[16];
        tmem_ld16(d + c, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int col = c + i;
          if (col < mcount)
            st_cluster_s32(smem_u32(part + ((int64_t)rank * per + col % per) * kI8Rows + 32 * q + lane),
                           (uint32_t)(col / per), v[i]);
        }
      }
      tc_fence_before();
    }
    __syncwarp();
    cluster_barrier();
    if (warp >= 2 && ok) {
      const int et = threadIdx.x - 64;
      const int c1 = min(per, mcount - rank * per);
      auto sum = [&](int c, int row) {
        int32_t t = 0;
        for (int s = 0; s < p.csplit; ++s) t += part[(s * per + c) * kI8Rows + row];
        return (float)t;
      };
      if (SWIGLU) {
        const int f = nti * (kI8Rows / 2) + (et & 63);
        const int row = 32 * ((et & 63) >> 4) + (et & 15);
        if (f < half) {
          const float wg = p.ws[f], wu = p.ws[half + f];
          for (int c = et >> 6; c < c1; c += 2) {
            const int m = m0 + rank * per + c;
            const float xs = p.xs[m];
            i8_store<BF16>(p.Y, (int64_t)m * half + f, silu_mul(sum(c, row) * xs * wg, sum(c, row + 16) * xs * wu));
          }
        }
      } else {
        const int n = nti * kI8Rows + et;
        if (n < p.N) {
          const float w = p.ws[n];
          for (int c = 0; c < c1; ++c) {
            const int m = m0 + rank * per + c;
            i8_store<BF16>(p.Y, (int64_t)m * p.N + n, sum(c, et) * p.xs[m] * w);
          }
        }
      }
    }
  }

  // ---- teardown ----
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)p.tmem_cols)
                 : "memory");
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
