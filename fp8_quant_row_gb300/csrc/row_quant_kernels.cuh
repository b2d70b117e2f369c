// row_quant_kernels.cuh -- 8-bit rows with one fp32 scale each (sm_103a):
//   rms_norm_quant   [h = RN_bf16(x + residual)] -> p = h * w, scaled by 1/rms(h)
//   silu_mul_quant   p = RN_bf16(silu(gate)) * up
//
// Both form products p of two bf16 values, exact in fp32 (16 significant bits), take the row's
// largest magnitude P and emit codes of p * inv with inv = RN(QMAX * RN(1 / P)):
//   int8   RNE(p * inv), the product unrounded (one FMA against 1.5 * 2^23 rounds it to the
//          integer held in the low byte of the sum)
//   e4m3   E4M3(RN(p * inv))
// The norm's 1/rms is common to a row, cancels in p / P and only enters the row's scale, so
// the codes do not depend on the order of any sum.
// A row with a NaN or infinite product gets the scale NaN and codes 0; one whose products are
// all below 2^-100 in magnitude gets the scale 0 and codes 0.
#pragma once

#include "fp8q_device.cuh"

namespace fp8q {

constexpr int kRqThreads = 256;
constexpr float kRqTiny = 0x1p-100f;

// max(|a|, |b|, |c|), NaN if any is NaN.
__device__ __forceinline__ float absmax3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <bool INT8>
__device__ __forceinline__ constexpr float rq_qmax() {
  return INT8 ? 127.0f : 448.0f;
}

// RN(QMAX * RN(1 / top)), 0 for a row that has no codes (top tiny, infinite or NaN).
template <bool INT8>
__device__ __forceinline__ float rq_inverse(float top) {
  return top >= kRqTiny && top <= 3.402823466e38f ? __fmul_rn(rq_qmax<INT8>(), __frcp_rn(top))
                                                  : 0.0f;
}

// Four codes of p * inv in one word.
template <bool INT8>
__device__ __forceinline__ uint32_t rq_codes4(float p0, float p1, float p2, float p3, float inv) {
  if (INT8) {
    const uint32_t a = __float_as_uint(__fmaf_rn(p0, inv, 12582912.0f));
    const uint32_t b = __float_as_uint(__fmaf_rn(p1, inv, 12582912.0f));
    const uint32_t c = __float_as_uint(__fmaf_rn(p2, inv, 12582912.0f));
    const uint32_t d = __float_as_uint(__fmaf_rn(p3, inv, 12582912.0f));
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
  }
  return pack_e4m3x2(__fmul_rn(p0, inv), __fmul_rn(p1, inv)) |
         (pack_e4m3x2(__fmul_rn(p2, inv), __fmul_rn(p3, inv)) << 16);
}

// RN_bf16(RN_fp32(silu(g))) of two gates as fp32 values. silu(g) = g / (1 + 2^(-g log2 e)); the
// product in the exponent and the two approximate instructions leave a relative error of up to
// 2^-18 (at g = -87; 2^-22 near 0), and for each of the 65536 bf16 gates the result rounds to
// the same bf16 value as the exact one (the test goes over all of them).
// The flushing reciprocal gives 0 for g <= -87.5.
__device__ __forceinline__ float rq_sigmoid_denominator(float g) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(g, -1.4426950408889634f)));
  return __fadd_rn(1.0f, e);
}
__device__ __forceinline__ float rq_silu(float g) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(rq_sigmoid_denominator(g)));
  return __fmul_rn(g, r);
}
__device__ __forceinline__ uint32_t rq_silu2(uint32_t g) {
  return pack_bf16x2(rq_silu(bf_lo(g)), rq_silu(bf_hi(g)));
}

// Largest magnitude (NaN above infinity) and sum over the CTA, the same in every thread.
__device__ __forceinline__ void rq_block_reduce(float& top, float& sum, float* red, int warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t t = __reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) {
    red[warp] = __uint_as_float(t);
    red[32 + warp] = sum;
  }
  __syncthreads();
  t = __float_as_uint(lane < warps ? red[lane] : 0.0f);
  sum = lane < warps ? red[32 + lane] : 0.0f;
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, t));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
}

struct RmsParams {
  const uint16_t* x;
  const uint16_t* residual;
  const uint16_t* weight;
  uint16_t* h;
  uint8_t* q;
  float* scale;
  int64_t rows;
  int cols;
  float eps;
};

// One CTA per row: first pass sums h^2 and takes max|p| with h kept in shared memory, the
// second forms the codes.
template <bool INT8, bool RESID>
__global__ void __launch_bounds__(kRqThreads) rms_norm_quant_kernel(RmsParams p) {
  extern __shared__ uint4 rq_row[];  // [cols] bf16, then the reduction's 64 floats
  float* red = reinterpret_cast<float*>(rq_row + (p.cols >> 3));
  allow_dependents();
  wait_for_producers();
  const int chunks = p.cols >> 3;
  const uint4* wv = reinterpret_cast<const uint4*>(p.weight);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const uint4* xv = reinterpret_cast<const uint4*>(p.x + row * p.cols);
    float top = 0.0f, sum = 0.0f;
    for (int c = threadIdx.x; c < chunks; c += kRqThreads) {
      uint4 h = xv[c];
      const uint4 w = wv[c];
      uint32_t hw[4] = {h.x, h.y, h.z, h.w};
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
      if (RESID) {
        const uint4 r = reinterpret_cast<const uint4*>(p.residual + row * p.cols)[c];
        const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          hw[i] = pack_bf16x2(__fadd_rn(bf_lo(hw[i]), bf_lo(rw[i])),
                              __fadd_rn(bf_hi(hw[i]), bf_hi(rw[i])));
        h = make_uint4(hw[0], hw[1], hw[2], hw[3]);
        reinterpret_cast<uint4*>(p.h + row * p.cols)[c] = h;
      }
      rq_row[c] = h;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = bf_lo(hw[i]), b = bf_hi(hw[i]);
        top = absmax3(top, a * bf_lo(ww[i]), b * bf_hi(ww[i]));
        sum = fmaf(b, b, fmaf(a, a, sum));
      }
    }
    rq_block_reduce(top, sum, red, kRqThreads / 32);
    const float inv = rq_inverse<INT8>(top);
    uint2* qv = reinterpret_cast<uint2*>(p.q + row * p.cols);
    for (int c = threadIdx.x; c < chunks; c += kRqThreads) {
      const uint4 h = rq_row[c], w = wv[c];
      uint2 o = make_uint2(0u, 0u);
      if (inv != 0.0f) {
        o.x = rq_codes4<INT8>(bf_lo(h.x) * bf_lo(w.x), bf_hi(h.x) * bf_hi(w.x),
                              bf_lo(h.y) * bf_lo(w.y), bf_hi(h.y) * bf_hi(w.y), inv);
        o.y = rq_codes4<INT8>(bf_lo(h.z) * bf_lo(w.z), bf_hi(h.z) * bf_hi(w.z),
                              bf_lo(h.w) * bf_lo(w.w), bf_hi(h.w) * bf_hi(w.w), inv);
      }
      qv[c] = o;
    }
    if (threadIdx.x == 0) {
      const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, float(p.cols)), p.eps));
      float s = 0.0f;
      if (top >= kRqTiny) s = __fdiv_rn(__fmul_rn(top, rstd), rq_qmax<INT8>());
      // NaN also where the squares leave fp32 (|h| from about 2^60)
      if (!(top <= 3.402823466e38f) || !(sum <= 3.402823466e38f)) s = __uint_as_float(0x7FC00000u);
      p.scale[row] = s;
    }
    __syncthreads();
  }
}

struct SiluParams {
  const uint16_t* gate;
  const uint16_t* up;
  int64_t ld;
  uint8_t* q;
  float* scale;
  int64_t rows;
  int cols;
};

// One CTA per row: max|p| first, then the codes from a second reading of the row.
template <bool INT8>
__global__ void __launch_bounds__(kRqThreads) silu_mul_quant_kernel(SiluParams p) {
  __shared__ float red[64];
  allow_dependents();
  wait_for_producers();
  const int chunks = p.cols >> 3;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const uint4* gv = reinterpret_cast<const uint4*>(p.gate + row * p.ld);
    const uint4* uv = reinterpret_cast<const uint4*>(p.up + row * p.ld);
    float top = 0.0f, sum = 0.0f;
    for (int c = threadIdx.x; c < chunks; c += kRqThreads) {
      const uint4 g = gv[c], u = uv[c];
      const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t s = rq_silu2(gw[i]);
        top = absmax3(top, bf_lo(s) * bf_lo(uw[i]), bf_hi(s) * bf_hi(uw[i]));
      }
    }
    rq_block_reduce(top, sum, red, kRqThreads / 32);
    const float inv = rq_inverse<INT8>(top);
    uint2* qv = reinterpret_cast<uint2*>(p.q + row * p.cols);
    for (int c = threadIdx.x; c < chunks; c += kRqThreads) {
      uint32_t o[2] = {0u, 0u};
      if (inv != 0.0f) {
        const uint4 g = gv[c], u = uv[c];
        const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t s = rq_silu2(gw[2 * i]), t = rq_silu2(gw[2 * i + 1]);
          o[i] = rq_codes4<INT8>(bf_lo(s) * bf_lo(uw[2 * i]), bf_hi(s) * bf_hi(uw[2 * i]),
                                 bf_lo(t) * bf_lo(uw[2 * i + 1]), bf_hi(t) * bf_hi(uw[2 * i + 1]),
                                 inv);
        }
      }
      qv[c] = make_uint2(o[0], o[1]);
    }
    if (threadIdx.x == 0) {
      float s = top >= kRqTiny ? __fdiv_rn(top, rq_qmax<INT8>()) : 0.0f;
      if (!(top <= 3.402823466e38f)) s = __uint_as_float(0x7FC00000u);
      p.scale[row] = s;
    }
    __syncthreads();
  }
}

}  // namespace fp8q
