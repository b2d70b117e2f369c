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
// Bound: HBM. Measured on one GB300 (CUDA-graph replay, inputs larger than the L2 cache; share of
// the 6690 GB/s of a plain copy): norm with residual 16384 x 8192 143 us (98%), 4608 x 6144 32.5
// (91%); without residual 16384 x 8192 72 us (84%), 4608 x 6144 18.7 (68%: there its 16 warps an SM
// are at work on instructions, 64% of the issue slots, and wait for loads in 5% of their time); silu
// 4608 x 18432 65.7 us (97%), 4608 x 10240 37.8 (93%); one row of 6144 2.3 us, of 18432 3.0 us. What carried them: the products kept between the two passes as fp32 pairs (no
// second unpacking), all loads of a row issued at once, the next row's before the reduction.
//
// A row with a NaN or infinite product gets the scale NaN and codes 0; one whose products are
// all below 2^-100 in magnitude gets the scale 0 and codes 0.
#pragma once

#include "fp8q_device.cuh"

namespace fp8q {

constexpr int kRqRedBytes = 1024;  // two buffers of a CTA's partial results, of 96 floats each
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

// Four codes of p * inv in one word, the products given as pairs.
template <bool INT8>
__device__ __forceinline__ uint32_t rq_codes4(f2 p0, f2 p1, float inv) {
  const f2 inv2 = f2_make(inv, inv);
  if (INT8) {
    const f2 magic = f2_make(12582912.0f, 12582912.0f);
    const f2 a = fma2(p0, inv2, magic), b = fma2(p1, inv2, magic);
    return __byte_perm(__byte_perm(uint32_t(a.v), uint32_t(a.v >> 32), 0x0040),
                       __byte_perm(uint32_t(b.v), uint32_t(b.v >> 32), 0x0040), 0x5410);
  }
  const f2 a = mul2(p0, inv2), b = mul2(p1, inv2);
  return pack_e4m3x2(f2_lo(a), f2_hi(a)) | (pack_e4m3x2(f2_lo(b), f2_hi(b)) << 16);
}

// Products of two bf16 chunks of eight, and their largest magnitude.
__device__ __forceinline__ void rq_products8(f2 (&p)[4], uint4 a, uint4 b, float& top) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[i] = mul2(bf2_to_f2(x[i]), bf2_to_f2(y[i]));
    top = absmax3(top, f2_lo(p[i]), f2_hi(p[i]));
  }
}

template <bool INT8>
__device__ __forceinline__ uint2 rq_codes8(const f2 (&p)[4], float inv) {
  if (inv == 0.0f) return make_uint2(0u, 0u);  // (the products may be NaN or infinite)
  return make_uint2(rq_codes4<INT8>(p[0], p[1], inv), rq_codes4<INT8>(p[2], p[3], inv));
}

// Products kept in shared memory: 32 bytes a chunk.
__device__ __forceinline__ void rq_keep(uint4* lo, uint4* hi, const f2 (&p)[4]) {
  *lo = make_uint4(uint32_t(p[0].v), uint32_t(p[0].v >> 32), uint32_t(p[1].v),
                   uint32_t(p[1].v >> 32));
  *hi = make_uint4(uint32_t(p[2].v), uint32_t(p[2].v >> 32), uint32_t(p[3].v),
                   uint32_t(p[3].v >> 32));
}
__device__ __forceinline__ void rq_kept(f2 (&p)[4], uint4 lo, uint4 hi) {
  p[0] = f2_make(__uint_as_float(lo.x), __uint_as_float(lo.y));
  p[1] = f2_make(__uint_as_float(lo.z), __uint_as_float(lo.w));
  p[2] = f2_make(__uint_as_float(hi.x), __uint_as_float(hi.y));
  p[3] = f2_make(__uint_as_float(hi.z), __uint_as_float(hi.w));
}

// RN_bf16(RN_fp32(silu(g))) of two gates as fp32 values. silu(g) = g / (1 + 2^(-g log2 e)); the
// product in the exponent and the two approximate instructions leave a relative error of up to
// 2^-18 (at g = -87; 2^-22 near 0), and for each of the 65536 bf16 gates the result rounds to
// the same bf16 value as the exact one (the test goes over all of them).
// The flushing reciprocal gives 0 for g <= -87.5.
__device__ __forceinline__ uint32_t rq_silu2(uint32_t g) {
  const f2 v = bf2_to_f2(g);
  const f2 t = mul2(v, f2_make(-1.4426950408889634f, -1.4426950408889634f));
  float e0, e1, r0, r1;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(f2_lo(t)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(f2_hi(t)));
  const f2 d = add2(f2_make(e0, e1), f2_make(1.0f, 1.0f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(f2_lo(d)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(f2_hi(d)));
  const f2 s = mul2(v, f2_make(r0, r1));
  return pack_bf16x2(f2_lo(s), f2_hi(s));
}
__device__ __forceinline__ uint4 rq_silu8(uint4 g) {
  return make_uint4(rq_silu2(g.x), rq_silu2(g.y), rq_silu2(g.z), rq_silu2(g.w));
}

// A sum kept as an unevaluated pair: the additions' rounding errors (TwoSum) gather in lo, so that
// the sum, rounded to fp32 at the end, does not depend on the order, that is on how many rows a
// call has (but for sums within about 2^-44 of a rounding border).
struct RowSum {
  float hi = 0.0f, lo = 0.0f;
  __device__ __forceinline__ void add(float h, float l) {
    float s, e;
    two_sum(hi, h, s, e);
    hi = s;
    lo = __fadd_rn(lo, __fadd_rn(l, e));
  }
  __device__ __forceinline__ void add_lanes() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      add(__shfl_xor_sync(0xffffffffu, hi, o), __shfl_xor_sync(0xffffffffu, lo, o));
  }
};

// Largest magnitude (NaN above infinity) and, where `sum` is given, sum over the threads of a row: a
// warp, or the whole CTA through `red` (kRqRed floats), with one barrier after it before `red` is
// used again.
constexpr int kRqRed = 96;
__device__ __forceinline__ void rq_reduce(float& top, RowSum* sum, float* red, int warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t t = __reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7FFFFFFFu);
  if (sum) sum->add_lanes();
  if (warps > 1) {
    if (lane == 0) {
      red[warp] = __uint_as_float(t);
      if (sum) red[32 + warp] = sum->hi, red[64 + warp] = sum->lo;
    }
    __syncthreads();
    t = __reduce_max_sync(0xffffffffu, __float_as_uint(lane < warps ? red[lane] : 0.0f));
    if (sum) {
      sum->hi = lane < warps ? red[32 + lane] : 0.0f;
      sum->lo = lane < warps ? red[64 + lane] : 0.0f;
      sum->add_lanes();
    }
  }
  top = __uint_as_float(t);
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

template <bool INT8>
__device__ __forceinline__ void rms_store_scale(const RmsParams& p, int64_t row, float top,
                                                float sum) {
  const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, float(p.cols)), p.eps));
  float s = 0.0f;
  if (top >= kRqTiny) s = __fdiv_rn(__fmul_rn(top, rstd), rq_qmax<INT8>());
  // NaN also where the squares leave fp32 (|h| from about 2^60)
  if (!(top <= 3.402823466e38f) || !(sum <= 3.402823466e38f)) s = __uint_as_float(0x7FC00000u);
  p.scale[row] = s;
}

__device__ __forceinline__ uint4 add_bf16x8(uint4 a, uint4 b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f2 v = add2(bf2_to_f2(x[i]), bf2_to_f2(y[i]));
    r[i] = pack_bf16x2(f2_lo(v), f2_hi(v));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ float sum_squares8(uint4 h) {
  const uint32_t x[4] = {h.x, h.y, h.z, h.w};
  f2 sum = f2_make(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f2 v = bf2_to_f2(x[i]);
    sum = fma2(v, v, sum);
  }
  return __fadd_rn(f2_lo(sum), f2_hi(sum));
}

// A row lives in the registers of its threads: `per_row` threads (a warp, several rows a CTA; or
// the whole CTA), CPT chunks of eight values each. With MANY rows a thread keeps its weights and
// goes from row to row, one grid apart, with the next row's loads issued before the current
// row's reduction (at 6144 columns two CTAs of 256 threads an SM keep 49 KB in flight with the
// residual, 25 KB without it). With few rows a CTA has one.
template <bool INT8, bool RESID, int CPT, bool MANY>
__global__ void __launch_bounds__(MANY ? 256 : 1024, MANY ? 2 : 1)
    rms_norm_quant_kernel(RmsParams p, int per_row) {
  __shared__ float red[2][kRqRed];
  allow_dependents();
  const int t = threadIdx.x % per_row, chunks = p.cols >> 3, warps = per_row >> 5;
  const int rows_cta = blockDim.x / per_row;
  wait_for_producers();
  uint4 w[CPT], x[CPT], r[RESID ? CPT : 1];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    w[i] = make_uint4(0, 0, 0, 0);
    if (t + i * per_row < chunks)
      w[i] = reinterpret_cast<const uint4*>(p.weight)[t + i * per_row];
  }
  auto load = [&](int64_t row) {
    const uint4* xv = reinterpret_cast<const uint4*>(p.x) + row * chunks;
    const uint4* rv = reinterpret_cast<const uint4*>(p.residual) + row * chunks;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      x[i] = make_uint4(0, 0, 0, 0);
      if (t + i * per_row < chunks) x[i] = ld_stream(xv + t + i * per_row);
    }
    if (RESID) {
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        r[RESID ? i : 0] = make_uint4(0, 0, 0, 0);
        if (t + i * per_row < chunks) r[RESID ? i : 0] = ld_stream(rv + t + i * per_row);
      }
    }
  };
  int64_t row = int64_t(blockIdx.x) * rows_cta + threadIdx.x / per_row;
  const int64_t stride = int64_t(gridDim.x) * rows_cta;
  if (row < p.rows) load(row);
  for (int flip = 0; row < p.rows; row += stride, flip ^= 1) {
    const int64_t base = row * chunks;
    float top = 0.0f;
    RowSum sum;
    f2 prod[CPT][4];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      if (RESID) {
        x[i] = add_bf16x8(x[i], r[RESID ? i : 0]);
        if (t + i * per_row < chunks)
          reinterpret_cast<uint4*>(p.h)[base + t + i * per_row] = x[i];
      }
      sum.add(sum_squares8(x[i]), 0.0f);
      rq_products8(prod[i], x[i], w[i], top);
    }
    if (MANY && row + stride < p.rows) load(row + stride);
    rq_reduce(top, &sum, red[flip], warps);
    const float inv = rq_inverse<INT8>(top);
    uint2* qv = reinterpret_cast<uint2*>(p.q) + base;
#pragma unroll
    for (int i = 0; i < CPT; ++i)
      if (t + i * per_row < chunks) qv[t + i * per_row] = rq_codes8<INT8>(prod[i], inv);
    if (t == 0) rms_store_scale<INT8>(p, row, top, __fadd_rn(sum.hi, sum.lo));
    if (!MANY) break;
  }
}

// Wide rows: the inputs, then the products in their place, in shared memory, where each thread
// keeps what it alone uses; the CTAs of an SM overlap one another's loads and work.
template <bool INT8, bool RESID, int THREADS>
__global__ void __launch_bounds__(THREADS) rms_norm_quant_wide_kernel(RmsParams p) {
  extern __shared__ uint4 rq_smem[];
  float* red = reinterpret_cast<float*>(rq_smem);  // two buffers
  const int chunks = p.cols >> 3;
  uint4 *lo = rq_smem + kRqRedBytes / 16, *hi = lo + chunks;
  allow_dependents();
  const uint4* wv = reinterpret_cast<const uint4*>(p.weight);
  wait_for_producers();
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, flip ^= kRqRed) {
    const int64_t base = row * chunks;
    const uint4* xv = reinterpret_cast<const uint4*>(p.x) + base;
    const uint4* rv = reinterpret_cast<const uint4*>(p.residual) + base;
    for (int c = threadIdx.x; c < chunks; c += THREADS) {
      cp_async16(lo + c, xv + c);
      if (RESID) cp_async16(hi + c, rv + c);
    }
    cp_async_commit();
    cp_async_wait<0>();
    float top = 0.0f;
    RowSum sum;
#pragma unroll 2
    for (int c = threadIdx.x; c < chunks; c += THREADS) {
      uint4 h = lo[c];
      if (RESID) {
        h = add_bf16x8(h, hi[c]);
        reinterpret_cast<uint4*>(p.h)[base + c] = h;
      }
      sum.add(sum_squares8(h), 0.0f);
      f2 prod[4];
      rq_products8(prod, h, wv[c], top);
      rq_keep(lo + c, hi + c, prod);
    }
    rq_reduce(top, &sum, red + flip, THREADS / 32);
    const float inv = rq_inverse<INT8>(top);
    uint2* qv = reinterpret_cast<uint2*>(p.q) + base;
#pragma unroll 2
    for (int c = threadIdx.x; c < chunks; c += THREADS) {
      f2 prod[4];
      rq_kept(prod, lo[c], hi[c]);
      qv[c] = rq_codes8<INT8>(prod, inv);
    }
    if (threadIdx.x == 0) rms_store_scale<INT8>(p, row, top, __fadd_rn(sum.hi, sum.lo));
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

template <bool INT8>
__device__ __forceinline__ void silu_store_scale(const SiluParams& p, int64_t row, float top) {
  float s = top >= kRqTiny ? __fdiv_rn(top, rq_qmax<INT8>()) : 0.0f;
  if (!(top <= 3.402823466e38f)) s = __uint_as_float(0x7FC00000u);
  p.scale[row] = s;
}

// As rms_norm_quant_kernel: a row in the registers of its threads (three CTAs an SM: 23.0 us at
// 4608 x 6144 against 25.0 with two; the norm, with its weights and residual, is faster with two).
template <bool INT8, int CPT, bool MANY>
__global__ void __launch_bounds__(MANY ? 256 : 1024, MANY ? 3 : 1)
    silu_mul_quant_kernel(SiluParams p, int per_row) {
  __shared__ float red[2][kRqRed];
  allow_dependents();
  const int t = threadIdx.x % per_row, chunks = p.cols >> 3, warps = per_row >> 5;
  const int rows_cta = blockDim.x / per_row;
  wait_for_producers();
  uint4 g[CPT], u[CPT];
  auto load = [&](int64_t row) {
    const uint4* gv = reinterpret_cast<const uint4*>(p.gate + row * p.ld);
    const uint4* uv = reinterpret_cast<const uint4*>(p.up + row * p.ld);
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      g[i] = u[i] = make_uint4(0, 0, 0, 0);
      if (t + i * per_row < chunks) {
        g[i] = ld_stream(gv + t + i * per_row);
        u[i] = ld_stream(uv + t + i * per_row);
      }
    }
  };
  int64_t row = int64_t(blockIdx.x) * rows_cta + threadIdx.x / per_row;
  const int64_t stride = int64_t(gridDim.x) * rows_cta;
  if (row < p.rows) load(row);
  for (int flip = 0; row < p.rows; row += stride, flip ^= 1) {
    float top = 0.0f;
    f2 prod[CPT][4];
#pragma unroll
    for (int i = 0; i < CPT; ++i) rq_products8(prod[i], rq_silu8(g[i]), u[i], top);
    if (MANY && row + stride < p.rows) load(row + stride);
    rq_reduce(top, nullptr, red[flip], warps);
    const float inv = rq_inverse<INT8>(top);
    uint2* qv = reinterpret_cast<uint2*>(p.q) + row * chunks;
#pragma unroll
    for (int i = 0; i < CPT; ++i)
      if (t + i * per_row < chunks) qv[t + i * per_row] = rq_codes8<INT8>(prod[i], inv);
    if (t == 0) silu_store_scale<INT8>(p, row, top);
    if (!MANY) break;
  }
}

// Wide rows in shared memory (KEEP: gate and up, then the products in their place, each thread's
// own); rows that do not fit are read twice.
template <bool INT8, bool KEEP, int THREADS>
__global__ void __launch_bounds__(THREADS) silu_mul_quant_wide_kernel(SiluParams p) {
  extern __shared__ uint4 rq_smem[];
  float* red = reinterpret_cast<float*>(rq_smem);  // two buffers
  const int chunks = p.cols >> 3;
  uint4 *lo = rq_smem + kRqRedBytes / 16, *hi = lo + chunks;
  allow_dependents();
  wait_for_producers();
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, flip ^= kRqRed) {
    const uint4* gv = reinterpret_cast<const uint4*>(p.gate + row * p.ld);
    const uint4* uv = reinterpret_cast<const uint4*>(p.up + row * p.ld);
    if (KEEP) {
      for (int c = threadIdx.x; c < chunks; c += THREADS) {
        cp_async16(lo + c, gv + c);
        cp_async16(hi + c, uv + c);
      }
      cp_async_commit();
      cp_async_wait<0>();
    }
    float top = 0.0f;
#pragma unroll 2
    for (int c = threadIdx.x; c < chunks; c += THREADS) {
      f2 prod[4];
      rq_products8(prod, rq_silu8(KEEP ? lo[c] : gv[c]), KEEP ? hi[c] : uv[c], top);
      if (KEEP) rq_keep(lo + c, hi + c, prod);
    }
    rq_reduce(top, nullptr, red + flip, THREADS / 32);
    const float inv = rq_inverse<INT8>(top);
    uint2* qv = reinterpret_cast<uint2*>(p.q) + row * chunks;
#pragma unroll 2
    for (int c = threadIdx.x; c < chunks; c += THREADS) {
      f2 prod[4];
      float again = 0.0f;
      if (KEEP) rq_kept(prod, lo[c], hi[c]);
      else rq_products8(prod, rq_silu8(gv[c]), uv[c], again);
      qv[c] = rq_codes8<INT8>(prod, inv);
    }
    if (threadIdx.x == 0) silu_store_scale<INT8>(p, row, top);
  }
}

}  // namespace fp8q
