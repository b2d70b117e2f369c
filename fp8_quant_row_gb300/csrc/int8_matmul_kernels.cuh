// int8_matmul_kernels.cuh -- out[m, n] = (sum_k a[m, k] w[n, k]) * w_scale[n] * a_scale[m]
// (+ bias[n]) for int8 a and w, sm_103a: what its two kernels share (few tokens, and tiles on
// the 5th-generation tensor cores).
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

}  // namespace fp8q
