// cache_kernels.cuh -- heads of q, k and v on their way into attention (sm_103a):
//   qk_norm_rope   per-head RMSNorm and rotation of q and k
//   cache_write    the same pass, with k and v going to the pages of a cache
//   cache_read     sequences of a paged cache back as bf16 rows
//
// Norm and rotation: n = x w / sqrt(mean(x^2) + eps) over a head's values, then each rotated pair
// (a, b) -> (a c - b s, b c + a s) for its angle; all in fp32, one rounding at the end (bf16, or
// the codes of 8-bit rows). Angles are kept as turns in 64-bit fixed point: a pair's step is
// inv_freq 2^64 / (2 pi), a position times its step modulo 2^64 is the turn's fraction, exact
// integer arithmetic at any position; only the step is rounded (2^-53 relative, the double's own).
//
// A head's row lies in D / 16 lanes, two chunks of eight values each, one from either half of the
// row: the pairs of both rotations of a whole head, (i, i + D/2) and (2i, 2i + 1), then lie in one
// lane, and the row's sum and maximum take log2(D / 16) shuffles.
//
// 8-bit rows: P = max|x|, inv = RN(QMAX RN(1 / P)), codes RNE(x inv) (int8) or E4M3(RN(x inv)),
// scale P / QMAX; rows with a NaN or an infinity get the scale NaN and codes 0, rows below 2^-100
// scale and codes 0 (as row_quant_kernels.cuh).
#pragma once

#include "fp8q_device.cuh"
#include "row_quant_kernels.cuh"

namespace fp8q {

constexpr int kCacheInt8 = 0, kCacheE4m3 = 1, kCacheBf16 = 2;
constexpr unsigned kDevErrBadIndex = 2u;  // a slot, page or length outside the cache

struct CacheView {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int64_t k_stride, v_stride;  // bytes between pages
  int64_t ks_stride, vs_stride;  // values between pages
  int64_t pages;
  uint64_t page_magic;  // ceil(2^64 / page_size): slots to pages by a multiplication
  int page_size, heads;
};

// x / page_size for 0 <= x < 2^48, by x * ceil(2^64 / d): the excess x (M d - 2^64) is below
// 2^48 * 2^10 < 2^64 / d.
__device__ __forceinline__ int64_t page_of(int64_t x, uint64_t magic) {
  return int64_t(__umul64hi(uint64_t(x), magic));
}

constexpr int kRopeNone = 0, kRopeHalves = 1, kRopePairs = 2, kRopePart = 3;
constexpr int kMaxPairs = 128;

struct RopeView {
  const double* inv_freq;
  const int32_t* axis;    // null: all 0
  const void* positions;  // [axes, tokens], int32 or int64
  int64_t stride;         // between axes
  int axes, pairs;
  bool wide;  // int64 positions
};

struct HeadsParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_ld, k_ld, v_ld;
  uint16_t* q_out;
  uint16_t* k_out;
  int64_t q_out_ld, k_out_ld;
  const uint16_t* q_weight;  // null: no norm
  const uint16_t* k_weight;
  const int64_t* slots;
  CacheView cache;
  RopeView rope;
  int64_t tokens;
  int q_heads, kv_heads, parts;
  float eps;
};

// cos and sin of 2 pi t 2^-32: t to the nearest quarter turn by integers, then the Taylor series on
// [-pi/4, pi/4] (the first terms left out are below 2^-28 and 2^-29).
__device__ __forceinline__ void turn_cos_sin(uint32_t t, float& c, float& s) {
  const int q = int(t + 0x20000000u) >> 30;
  const float x = __fmul_rn(float(int(t - (uint32_t(q) << 30))), 1.4629180792671596e-9f);  // 2 pi 2^-32
  const float z = x * x;
  const float sp = x + x * z * (-1.6666667163e-1f + z * (8.3333337680e-3f + z * (-1.9841270114e-4f +
                   z * 2.7557319224e-6f)));
  const float cp = 1.0f + z * (-0.5f + z * (4.1666667908e-2f + z * (-1.3888889225e-3f +
                   z * (2.4801587642e-5f - z * 2.7557319224e-7f))));
  const float a = (q & 1) ? sp : cp, b = (q & 1) ? cp : sp;
  c = (q + 1) & 2 ? -a : a;
  s = q & 2 ? -b : b;
}

// The rotation's steps (turns per position, 64-bit fixed point) and axes, in shared memory.
struct RopeTable {
  uint64_t step[kMaxPairs];
  int axis[kMaxPairs];
};

__device__ __forceinline__ void rope_table(RopeTable& t, const RopeView& r) {
  for (int i = threadIdx.x; i < r.pairs; i += blockDim.x) {
    double turns = r.inv_freq[i] * 0.15915494309189535;  // 1 / (2 pi)
    turns -= rint(turns);
    t.step[i] = uint64_t(__double2ll_rn(turns * 18446744073709551616.0));
    t.axis[i] = r.axis ? min(max(r.axis[i], 0), r.axes - 1) : 0;
  }
  __syncthreads();
}

__device__ __forceinline__ int64_t rope_position(const RopeView& r, int axis, int64_t token) {
  const int64_t at = axis * r.stride + token;
  return r.wide ? static_cast<const int64_t*>(r.positions)[at]
                : static_cast<const int32_t*>(r.positions)[at];
}

__device__ __forceinline__ void rope_angle(const RopeView& r, const RopeTable& t, int pair,
                                           int64_t token, float& c, float& s) {
  c = 1.0f;
  s = 0.0f;
  if (pair < r.pairs) {
    const uint64_t turn = uint64_t(rope_position(r, t.axis[pair], token)) * t.step[pair];
    turn_cos_sin(uint32_t(turn >> 32), c, s);
  }
}

// Eight bf16 values of a 16-byte chunk as fp32.
__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = bf_lo(u[i]), x[2 * i + 1] = bf_hi(u[i]);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

template <bool INT8>
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
  const f2 p[4] = {f2_make(x[0], x[1]), f2_make(x[2], x[3]), f2_make(x[4], x[5]),
                   f2_make(x[6], x[7])};
  return rq_codes8<INT8>(p, inv);
}

// One row of the cache: bf16, or codes and scale. (a, b: the lane's two chunks of the row; u: the
// lane's place in it; all lanes of the warp take part, `live` ones store.)
template <int D, int TYPE>
__device__ __forceinline__ void store_row(const float (&a)[8], const float (&b)[8], int u, bool live,
                                          uint8_t* row, float* scale) {
  constexpr int LPH = D / 16;
  if (TYPE == kCacheBf16) {
    if (live) {
      reinterpret_cast<uint4*>(row)[u] = pack8(a);
      reinterpret_cast<uint4*>(row)[LPH + u] = pack8(b);
    }
    return;
  }
  constexpr bool INT8 = TYPE == kCacheInt8;
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = absmax3(top, a[j], b[j]);
#pragma unroll
  for (int o = 1; o < LPH; o <<= 1) top = absmax3(top, __shfl_xor_sync(0xffffffffu, top, o), 0.0f);
  const float inv = rq_inverse<INT8>(top);
  if (live) {
    reinterpret_cast<uint2*>(row)[u] = codes8<INT8>(a, inv);
    reinterpret_cast<uint2*>(row)[LPH + u] = codes8<INT8>(b, inv);
    if (u == 0) {
      float s = top >= kRqTiny ? __fdiv_rn(top, rq_qmax<INT8>()) : 0.0f;
      if (!(top <= 3.402823466e38f)) s = __uint_as_float(0x7FC00000u);
      *scale = s;
    }
  }
}

// A unit is a token's share of head steps: steps of 32 / (D / 16) heads, q's first, then k's and
// v's, `parts` warps taking them in turn. CACHE: k and v go to the cache (else k to k_out).
constexpr int kHeadsThreads = 256;

template <int D, int ROPE, bool CACHE, int TYPE>
__global__ void __launch_bounds__(kHeadsThreads) heads_kernel(const __grid_constant__ HeadsParams P) {
  constexpr int LPH = D / 16, HPW = 32 / LPH;
  __shared__ RopeTable table;
  const int lane = threadIdx.x & 31, g = lane / LPH, u = lane % LPH;
  wait_for_producers();
  allow_dependents();
  if (ROPE != kRopeNone) rope_table(table, P.rope);
  const int q_steps = (P.q_heads + HPW - 1) / HPW, kv_steps = (P.kv_heads + HPW - 1) / HPW;
  const int steps = q_steps + (CACHE ? 2 : 1) * kv_steps;
  const int64_t units = P.tokens * P.parts;
  const int64_t stride = int64_t(gridDim.x) * (kHeadsThreads / 32);
  for (int64_t unit = int64_t(blockIdx.x) * (kHeadsThreads / 32) + (threadIdx.x >> 5); unit < units;
       unit += stride) {
    const int64_t token = unit / P.parts;
    const int part = int(unit - token * P.parts);
    // where this token's k and v go
    int64_t page = 0;
    int at = 0;
    bool store = true;
    if (CACHE) {
      const int64_t slot = P.slots[token];
      store = slot >= 0 && slot < P.cache.pages * P.cache.page_size;
      if (store) {
        page = page_of(slot, P.cache.page_magic);
        at = int(slot - page * P.cache.page_size);
      } else if (slot >= 0 && lane == 0) {
        report_device_error(kDevErrBadIndex);
      }
    }
    // cos and sin of the lane's pairs: slot 0 chunk a, slot 1 chunk b
    constexpr int NC = ROPE == kRopePart ? 16 : 8;
    float cs[NC], sn[NC];
    if (ROPE == kRopeHalves) {
#pragma unroll
      for (int j = 0; j < 8; ++j) rope_angle(P.rope, table, u * 8 + j, token, cs[j], sn[j]);
    } else if (ROPE == kRopePairs) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        rope_angle(P.rope, table, (j < 4 ? 0 : D / 4 - 4) + u * 4 + j, token, cs[j], sn[j]);
    } else if (ROPE == kRopePart) {
      // the chunk pairs with another, `half` chunks away; the second of a pair has -s
      const int half = P.rope.pairs / 8;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int chunk = u + (j < 8 ? 0 : LPH);
        const int first = chunk < half ? chunk : chunk - half;
        rope_angle(P.rope, table, chunk < 2 * half ? first * 8 + (j & 7) : kMaxPairs, token, cs[j],
                   sn[j]);
        if (chunk < half) sn[j] = -sn[j];
      }
    }
    for (int step = part; step < steps; step += P.parts) {
      const int kind = step < q_steps ? 0 : step < q_steps + kv_steps ? 1 : 2;
      const int h = (step - (kind == 0 ? 0 : kind == 1 ? q_steps : q_steps + kv_steps)) * HPW + g;
      const bool live = h < (kind == 0 ? P.q_heads : P.kv_heads);
      const uint16_t* src = kind == 0   ? P.q + token * P.q_ld
                            : kind == 1 ? P.k + token * P.k_ld
                                        : P.v + token * P.v_ld;
      uint4 wa = make_uint4(0, 0, 0, 0), wb = wa;
      if (live) {
        const uint4* row = reinterpret_cast<const uint4*>(src + int64_t(h) * D);
        wa = ld_stream(row + u);
        wb = ld_stream(row + LPH + u);
      }
      float a[8], b[8];
      unpack8(wa, a);
      unpack8(wb, b);
      const uint16_t* weight = kind == 0 ? P.q_weight : P.k_weight;
      if (kind < 2 && weight) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __fmaf_rn(a[j], a[j], __fmaf_rn(b[j], b[j], sum));
#pragma unroll
        for (int o = 1; o < LPH; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float r = __frsqrt_rn(__fmaf_rn(sum, 1.0f / D, P.eps));
        float w[8];
        unpack8(*reinterpret_cast<const uint4*>(weight + u * 8), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = a[j] * r * w[j];
        unpack8(*reinterpret_cast<const uint4*>(weight + D / 2 + u * 8), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = b[j] * r * w[j];
      }
      if (kind < 2) {
        if (ROPE == kRopeHalves) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = a[j], y = b[j];
            a[j] = x * cs[j] - y * sn[j];
            b[j] = y * cs[j] + x * sn[j];
          }
        } else if (ROPE == kRopePairs) {
          // (pairs that are not rotated stay: an infinity beside a zero sine would not)
          const bool all = P.rope.pairs == D / 2;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = a[2 * j], y = a[2 * j + 1];
            if (all || u * 4 + j < P.rope.pairs) {
              a[2 * j] = x * cs[j] - y * sn[j];
              a[2 * j + 1] = y * cs[j] + x * sn[j];
            }
            const float z = b[2 * j], w = b[2 * j + 1];
            if (all || D / 4 + u * 4 + j < P.rope.pairs) {
              b[2 * j] = z * cs[4 + j] - w * sn[4 + j];
              b[2 * j + 1] = w * cs[4 + j] + z * sn[4 + j];
            }
          }
        } else if (ROPE == kRopePart) {
          const int half = P.rope.pairs / 8;
          const int ya = u < half ? u + half : u < 2 * half ? u - half : u;
          const int xb = u + LPH;
          const int yb = xb < half ? xb + half : xb < 2 * half ? xb - half : xb;
          float oa[8], ob[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float pa0 = __shfl_sync(0xffffffffu, a[j], ya % LPH, LPH);
            const float pa1 = __shfl_sync(0xffffffffu, b[j], ya % LPH, LPH);
            const float pb0 = __shfl_sync(0xffffffffu, a[j], yb % LPH, LPH);
            const float pb1 = __shfl_sync(0xffffffffu, b[j], yb % LPH, LPH);
            oa[j] = a[j] * cs[j] + (ya < LPH ? pa0 : pa1) * sn[j];
            ob[j] = b[j] * cs[8 + j] + (yb < LPH ? pb0 : pb1) * sn[8 + j];
          }
          // a chunk that is not rotated stays as it is (an infinity beside a zero sine would not)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (u < 2 * half) a[j] = oa[j];
            if (xb < 2 * half) b[j] = ob[j];
          }
        }
      }
      if (kind == 0 || !CACHE) {
        uint16_t* dst = kind == 0 ? P.q_out + token * P.q_out_ld : P.k_out + token * P.k_out_ld;
        if (live) {
          uint4* row = reinterpret_cast<uint4*>(dst + int64_t(h) * D);
          row[u] = pack8(a);
          row[LPH + u] = pack8(b);
        }
      } else if (CACHE) {
        constexpr int E = TYPE == kCacheBf16 ? 2 : 1;
        const int64_t row = int64_t(h) * P.cache.page_size + at;
        uint8_t* dst = (kind == 1 ? P.cache.k + page * P.cache.k_stride
                                  : P.cache.v + page * P.cache.v_stride) + row * (D * E);
        float* scale = kind == 1 ? P.cache.k_scale + page * P.cache.ks_stride + row
                                 : P.cache.v_scale + page * P.cache.vs_stride + row;
        store_row<D, TYPE>(a, b, u, live && store, dst, scale);
      }
    }
  }
}

// ------------------------------------------------------------------------------------------
// cache_read
// ------------------------------------------------------------------------------------------

struct ReadParams {
  CacheView cache;
  const int32_t* table;
  int64_t table_ld;
  const int64_t* offsets;  // [batch + 1]
  uint16_t* k;
  uint16_t* v;
  int64_t rows;
  int batch, width;
};

constexpr int kReadThreads = 256, kReadRows = 16;

// Eight 8-bit codes as bf16(code * scale).
template <int TYPE>
__device__ __forceinline__ uint4 dequant8(uint2 w, float s) {
  float x[8];
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (TYPE == kCacheInt8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[4 * i + j] = float(int8_t(u[i] >> (8 * j)));
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(u[i] >> (16 * j))));
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\t"
            "cvt.f32.f16 %1, hi;\n\t}"
            : "=f"(x[4 * i + 2 * j]), "=f"(x[4 * i + 2 * j + 1])
            : "r"(h));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] *= s;
  return pack8(x);
}

// A CTA takes 16 output rows, that is tokens: their places are looked up once, then each lane copies
// eight values of one head's row, tokens first (a page holds a head's tokens side by side).
template <int D, int TYPE>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const __grid_constant__ ReadParams P) {
  constexpr int E = TYPE == kCacheBf16 ? 2 : 1, LPR = D / 8;
  __shared__ int64_t page_s[kReadRows];
  __shared__ int at_s[kReadRows];
  wait_for_producers();
  allow_dependents();
  const int64_t row0 = int64_t(blockIdx.x) * kReadRows;
  if (threadIdx.x < kReadRows) {
    const int64_t row = row0 + threadIdx.x;
    int64_t page = -1;
    int at = 0;
    if (row < P.rows && row >= P.offsets[0] && row < P.offsets[P.batch]) {
      int lo = 0, hi = P.batch;  // the last sequence that starts at or before the row
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (P.offsets[mid] <= row) lo = mid; else hi = mid;
      }
      const int64_t t = row - P.offsets[lo], n = page_of(t, P.cache.page_magic);
      at = int(t - n * P.cache.page_size);
      page = n < P.width ? P.table[lo * P.table_ld + n] : -1;
      if (page < 0 || page >= P.cache.pages) {
        page = -2;
        report_device_error(kDevErrBadIndex);
      }
    }
    page_s[threadIdx.x] = page;
    at_s[threadIdx.x] = at;
  }
  __syncthreads();
  const int H = P.cache.heads;
  const int work = 2 * H * kReadRows * LPR;
  for (int i = threadIdx.x; i < work; i += kReadThreads) {
    const int u = i % LPR, r = (i / LPR) % kReadRows, hk = i / (LPR * kReadRows);
    const int h = hk >> 1;
    const bool is_v = hk & 1;
    const int64_t page = page_s[r];
    if (page == -1) continue;  // not a row of any sequence
    uint4 out = make_uint4(0, 0, 0, 0);
    if (page >= 0) {
      const int64_t at = int64_t(h) * P.cache.page_size + at_s[r];
      const uint8_t* src = (is_v ? P.cache.v + page * P.cache.v_stride
                                 : P.cache.k + page * P.cache.k_stride) + (at * D + u * 8) * E;
      if (TYPE == kCacheBf16) {
        out = ld_stream(reinterpret_cast<const uint4*>(src));
      } else {
        const float s = is_v ? P.cache.v_scale[page * P.cache.vs_stride + at]
                             : P.cache.k_scale[page * P.cache.ks_stride + at];
        out = dequant8<TYPE>(__ldcs(reinterpret_cast<const uint2*>(src)), s);
      }
    }
    uint16_t* dst = (is_v ? P.v : P.k) + ((row0 + r) * H + h) * D + u * 8;
    st_stream(reinterpret_cast<uint4*>(dst), out);
  }
}

}  // namespace fp8q
