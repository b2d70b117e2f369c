// int8_matmul_kernels.cuh -- out[m, n] = (sum_k a[m, k] w[n, k]) * w_scale[n] * a_scale[m]
// (+ bias[n]) for int8 a and w, sm_103a.
#pragma once

#include "fp8q_device.cuh"

namespace fp8q {

struct MmParams {
  const int8_t* a;
  const int8_t* w;
  const float* a_scale;
  const float* w_scale;
  const uint16_t* bias;  // bf16 or null
  void* out;             // [m, n] bf16 or fp32
  int64_t lda;
  int64_t m, n, k;
};

// The epilogue's value: the sum as fp32, each factor rounded once.
__device__ __forceinline__ float mm_value(float acc, float ws, float as, float bias) {
  return __fmaf_rn(__fmul_rn(acc, ws), as, bias);
}

// A store that keeps its place in the program.
template <bool F32>
__device__ __forceinline__ void mm_store(void* out, float v) {
  if (F32)
    asm volatile("st.global.f32 [%0], %1;" ::"l"(out), "f"(v) : "memory");
  else
    asm volatile("st.global.b16 [%0], %1;" ::"l"(out), "h"(uint16_t(pack_bf16x2(v, 0.0f)))
                 : "memory");
}

// Four int8 of a word as two fp16 pairs.
__device__ __forceinline__ void int8_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(0x64806480u));
  asm("sub.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(0x64806480u));
}

// 64 x 64 outputs per CTA of 256 threads, 4 x 4 per thread, products of four int8 by dp4a.
constexpr int kMmTile = 64, kMmThreads = 256, kMmStep = 64;

template <bool F32>
__global__ void __launch_bounds__(kMmThreads) int8_matmul_dp4a_kernel(MmParams p) {
  __shared__ int as[kMmStep / 4][kMmTile + 1], ws[kMmStep / 4][kMmTile + 1];
  allow_dependents();
  wait_for_producers();
  const int64_t n0 = int64_t(blockIdx.x) * kMmTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int lr = threadIdx.x >> 2, lk = (threadIdx.x & 3) * 16;
  for (int64_t m0 = int64_t(blockIdx.y) * kMmTile; m0 < p.m; m0 += int64_t(gridDim.y) * kMmTile) {
    int acc[4][4] = {};
    for (int64_t k0 = 0; k0 < p.k; k0 += kMmStep) {
      int4 av = make_int4(0, 0, 0, 0), wv = av;
      if (k0 + lk < p.k) {
        if (m0 + lr < p.m) av = *reinterpret_cast<const int4*>(p.a + (m0 + lr) * p.lda + k0 + lk);
        if (n0 + lr < p.n) wv = *reinterpret_cast<const int4*>(p.w + (n0 + lr) * p.k + k0 + lk);
      }
      __syncthreads();
      const int kk = lk / 4;
      as[kk][lr] = av.x, as[kk + 1][lr] = av.y, as[kk + 2][lr] = av.z, as[kk + 3][lr] = av.w;
      ws[kk][lr] = wv.x, ws[kk + 1][lr] = wv.y, ws[kk + 2][lr] = wv.z, ws[kk + 3][lr] = wv.w;
      __syncthreads();
#pragma unroll 4
      for (int q = 0; q < kMmStep / 4; ++q) {
        int a[4], w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = as[q][ty + 16 * i], w[i] = ws[q][tx + 16 * i];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(a[i], w[j], acc[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m < p.m && n < p.n)
          mm_store<F32>(static_cast<uint8_t*>(p.out) + (m * p.n + n) * (F32 ? 4 : 2),
                        mm_value(float(acc[i][j]), p.w_scale[n], p.a_scale[m],
                                 p.bias ? __uint_as_float(uint32_t(p.bias[n]) << 16) : 0.0f));
      }
  }
}

}  // namespace fp8q
