// Rows of bf16 to int8 codes with one fp32 scale per row (the activations of the int8
// product, one scale per token; or, at load time, its weights, one per output channel).
//
//   amax = max_k |x_k|,  scale = RN_fp32(amax / 127),  q_k = RNE(127 x_k / amax)
//
// The code is the exact quotient rounded to nearest, ties to even. A quotient rounded to 24
// bits decides that as well as the exact one: 127 x has 15 significant bits and amax 8, so a
// quotient that is not half an odd number is at least 2^-17 of one away, and half odd
// numbers below 128 are representable. (Ties are common: one value in a few hundred.)
// A row of zeros gets scale 0 and codes 0; a row that holds an infinity or a NaN gets scale
// NaN and codes 0, so that every product with it is NaN.
#pragma once
#include "common.cuh"

namespace q4k {

__device__ __forceinline__ float i8_bf16_at(const uint32_t (&w)[4], int i) {
  return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
}

// Codes of eight values, amax and rcp = RN(1 / amax) given, SCALED: the values times `two`
// first. The quotient by one residual step: t is within 2 ulp of it, 127 x - t amax is exact,
// and the corrected t rounds correctly; adding 1.5 * 2^23 rounds it to the integer that the
// sum's low byte holds.
template <bool SCALED>
__device__ __forceinline__ uint2 i8_codes(const uint4& a, float amax, float rcp, float two) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  uint32_t m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = 127.f * (SCALED ? i8_bf16_at(w, i) * two : i8_bf16_at(w, i));  // exact
    const float t = x * rcp;
    m[i] = __float_as_uint(fmaf(fmaf(-t, amax, x), rcp, t) + 12582912.f);
  }
  uint2 o;
  o.x = __byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410);
  o.y = __byte_perm(__byte_perm(m[4], m[5], 0x0040), __byte_perm(m[6], m[7], 0x0040), 0x5410);
  return o;
}

// TPR threads per row, 32 .. 1024 (several rows per CTA below 256). The row stays in
// registers between the maximum and the codes when it has at most TPR * 8 * V values; the
// rest of a longer one is read again. Bound by DRAM (3 bytes a value); what counts is few
// instructions per value: 4096 x 5120 takes 12.4 us (5.1 TB/s, 77% of the measured copy rate),
// with a code's remainder checked and mended by a branch 18.4 us, with all eight codes redone
// exactly where one is near a tie 14.3 us (ties are common enough to send most warps there).
template <int TPR, int V>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
i8_quantize_kernel(const uint16_t* __restrict__ X, int M, int K, int8_t* __restrict__ Q, float* __restrict__ scale) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kRows = kThreads / TPR;
  constexpr int kWarps = TPR / 32;  // warps of a row
  const int lane = threadIdx.x & 31;
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  const bool live = row < M;
  const int nv = K / 8;
  const uint16_t* x = X + (live ? row : 0) * K;
  uint4 v[V];
  uint32_t m = 0;
  auto take = [&](const uint4& a) {
    m = __vmaxu2(__vmaxu2(m, __vmaxu2(a.x & 0x7FFF7FFFu, a.y & 0x7FFF7FFFu)),
                 __vmaxu2(a.z & 0x7FFF7FFFu, a.w & 0x7FFF7FFFu));
  };
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int p = t + i * TPR;
    v[i] = live && p < nv ? ldg_stream_u4(x + 8 * (int64_t)p) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) take(v[i]);
  if (live)
    for (int p = t + V * TPR; p < nv; p += TPR) take(ldg_u4(x + 8 * (int64_t)p));
  uint32_t mb = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));  // bits of amax
  if constexpr (kWarps > 1) {
    __shared__ uint32_t part[kThreads / 32];
    const int warp = threadIdx.x >> 5;
    if (lane == 0) part[warp] = mb;
    __syncthreads();
    const int w0 = warp / kWarps * kWarps;
    mb = __reduce_max_sync(0xffffffffu, lane < kWarps ? part[w0 + lane] : 0u);
  }
  if (!live) return;
  const bool good = mb < 0x7F80u;
  float amax = bf16_bits_to_float(mb);
  if (t == 0) scale[row] = good ? amax / 127.f : __uint_as_float(0x7FC00000u);
  int8_t* q = Q + row * K;
  auto each = [&](auto&& codes) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int p = t + i * TPR;
      if (p < nv) *reinterpret_cast<uint2*>(q + 8 * (int64_t)p) = codes(v[i]);
    }
    for (int p = t + V * TPR; p < nv; p += TPR)
      *reinterpret_cast<uint2*>(q + 8 * (int64_t)p) = codes(ldg_u4(x + 8 * (int64_t)p));
  };
  if (!good || mb == 0) {
    each([](const uint4&) { return make_uint2(0u, 0u); });
  } else if (mb >= 0x7180u || mb < 0x2000u) {
    // 127 x would overflow, or 1 / amax not be normal: all times a power of two first
    const float two = mb >= 0x7180u ? 0x1p-64f : 0x1p64f;
    amax *= two;
    const float rcp = 1.f / amax;
    each([&](const uint4& a) { return i8_codes<true>(a, amax, rcp, two); });
  } else {
    const float rcp = 1.f / amax;
    each([&](const uint4& a) { return i8_codes<false>(a, amax, rcp, 1.f); });
  }
}

}  // namespace q4k
