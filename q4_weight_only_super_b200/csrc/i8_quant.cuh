// Rows of bf16 to int8 codes with one fp32 scale per row (the activations of the int8
// product, one scale per token; or, at load time, its weights, one per output channel).
//
//   amax = max_k |x_k|,  scale = RN_fp32(amax / 127),  q_k = RNE(127 x_k / amax)
//
// The code is the exact quotient rounded to nearest, ties to even: 127 x has 15
// significant bits, so the remainder 127 x - q amax of a candidate q is exact in fp32 and
// settles what a rounded reciprocal leaves open next to a tie. A row of zeros gets scale 0
// and codes 0; a row that holds an infinity or a NaN gets scale NaN and codes 0, so that
// every product with it is NaN.
#pragma once
#include "common.cuh"

namespace q4k {

constexpr int kI8QVec = 4;  // 8-value pieces of a row that a thread keeps in registers

// Code of x, given amax > 0 and inv = RN(127 / amax), all three scaled by the same power
// of two so that 127 x does not overflow.
__device__ __forceinline__ int i8_code(float x, float amax, float inv) {
  float q = rintf(x * inv);
  const float rem = fmaf(-q, amax, 127.f * x);  // exact
  const float twice = fabsf(rem) * 2.f;
  if (twice >= amax) {  // next to or on a tie: rare
    const float step = rem > 0.f ? 1.f : -1.f;
    if (twice > amax || ((int)q & 1)) q += step;
  }
  return (int)q;
}

// TPR threads per row, 32 .. 1024 (several rows per CTA at 32). The row stays in registers
// between the maximum and the codes when it has at most TPR * 8 * kI8QVec values; the rest
// of a longer one is read again.
template <int TPR>
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
  uint4 v[kI8QVec];
  uint32_t m = 0;
  auto take = [&](const uint4& a) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  };
#pragma unroll
  for (int i = 0; i < kI8QVec; ++i) {
    const int p = t + i * TPR;
    v[i] = live && p < nv ? ldg_stream_u4(x + 8 * (int64_t)p) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < kI8QVec; ++i) take(v[i]);
  if (live)
    for (int p = t + kI8QVec * TPR; p < nv; p += TPR) take(ldg_u4(x + 8 * (int64_t)p));
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
  // the same power of two on x and amax: 127 x stays in range and 127 / amax is normal
  const float two = mb >= 0x7180u ? 0x1p-64f : (mb < 0x2000u ? 0x1p64f : 1.f);
  amax *= two;
  const float inv = good && mb ? 127.f / amax : 0.f;
  int8_t* q = Q + row * K;
  auto put = [&](int p, const uint4& a) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    uint32_t o[2] = {0u, 0u};
    if (good && mb) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xv = bf16_bits_to_float(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu) * two;
        o[i >> 2] |= ((uint32_t)i8_code(xv, amax, inv) & 0xFFu) << (8 * (i & 3));
      }
    }
    *reinterpret_cast<uint2*>(q + 8 * (int64_t)p) = make_uint2(o[0], o[1]);
  };
#pragma unroll
  for (int i = 0; i < kI8QVec; ++i) {
    const int p = t + i * TPR;
    if (p < nv) put(p, v[i]);
  }
  for (int p = t + kI8QVec * TPR; p < nv; p += TPR) put(p, ldg_u4(x + 8 * (int64_t)p));
}

}  // namespace q4k
