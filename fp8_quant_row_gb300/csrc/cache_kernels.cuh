// cache_kernels.cuh -- heads of q, k and v on their way into attention (sm_103a):
//   qk_norm_rope   per-head RMSNorm and rotation of q and k
//   cache_write    the same pass, with k and v going to the pages of a cache
//   cache_read     sequences of a paged cache back as bf16 rows
//
// Norm and rotation: n = x w / sqrt(mean(x^2) + eps) over a head's values, then each rotated pair
// (a, b) -> (a c - b s, b c + a s) for its angle; all in fp32, one rounding at the end (bf16, or
// the codes of 8-bit rows). Angles are kept as turns in 64-bit fixed point: a pair's step is
// inv_freq 2^64 / (2 pi), a position times its step modulo 2^64 is the turn's fraction, exact
// integer arithmetic at any position; only the step is rounded (2^-52 of itself, 1 / (2 pi) and the
// product, and 2^-65 turns).
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
constexpr unsigned kDevErrBadIndex = 2u;  // a slot or page outside the cache

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

// x / page_size for 0 <= x < 2^48, by the high word of x M, M = ceil(2^64 / d): exact where
// x (M d - 2^64) < 2^64, and M d - 2^64 < d <= 2^10.
__device__ __forceinline__ int64_t page_of(int64_t x, uint64_t magic) {
  return int64_t(__umul64hi(uint64_t(x), magic));
}

constexpr int kRopeNone = 0, kRopeHalves = 1, kRopePairs = 2;
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
  int q_heads, kv_heads;
  int group_tokens, parts;  // tokens a CTA takes at a time (1, 2, 4, 8), CTAs that share a token
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

__device__ __forceinline__ uint64_t rope_step(double inv_freq) {
  double turns = inv_freq * 0.15915494309189535;  // 1 / (2 pi)
  turns -= rint(turns);
  return uint64_t(__double2ll_rn(turns * 18446744073709551616.0));
}

__device__ __forceinline__ int64_t rope_position(const RopeView& r, int axis, int64_t token) {
  const int64_t at = axis * r.stride + token;
  return r.wide ? static_cast<const int64_t*>(r.positions)[at]
                : static_cast<const int32_t*>(r.positions)[at];
}

// A copy of 16 bytes to shared memory, zeros where `in` is false.
__device__ __forceinline__ void cp_async_if(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ uint4 lds_words(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

// Eight bf16 values of a 16-byte chunk as fp32 pairs.
__device__ __forceinline__ void unpack8(uint4 w, f2 (&x)[4]) {
  x[0] = bf2_to_f2(w.x), x[1] = bf2_to_f2(w.y), x[2] = bf2_to_f2(w.z), x[3] = bf2_to_f2(w.w);
}
__device__ __forceinline__ uint4 pack8(const f2 (&x)[4]) {
  return make_uint4(pack_bf16x2(f2_lo(x[0]), f2_hi(x[0])), pack_bf16x2(f2_lo(x[1]), f2_hi(x[1])),
                    pack_bf16x2(f2_lo(x[2]), f2_hi(x[2])), pack_bf16x2(f2_lo(x[3]), f2_hi(x[3])));
}
__device__ __forceinline__ f2 neg2(f2 a) { return f2{a.v ^ 0x8000000080000000ull}; }

// One row of the cache: bf16, or codes and scale. (a, b: the lane's chunks ca and cb of the row; all
// lanes of the warp take part, `live` ones store; one lane a row is the `first`.)
template <int D, int TYPE>
__device__ __forceinline__ void store_row(const f2 (&a)[4], const f2 (&b)[4], int ca, int cb,
                                          bool first, bool live, uint8_t* row, float* scale) {
  if (TYPE == kCacheBf16) {
    if (live) {
      reinterpret_cast<uint4*>(row)[ca] = pack8(a);
      reinterpret_cast<uint4*>(row)[cb] = pack8(b);
    }
    return;
  }
  constexpr bool INT8 = TYPE == kCacheInt8;
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    top = absmax3(absmax3(top, f2_lo(a[j]), f2_hi(a[j])), f2_lo(b[j]), f2_hi(b[j]));
#pragma unroll
  for (int o = 1; o < D / 16; o <<= 1)
    top = absmax3(top, __shfl_xor_sync(0xffffffffu, top, o), 0.0f);
  const float inv = rq_inverse<INT8>(top);
  if (live) {
    reinterpret_cast<uint2*>(row)[ca] = rq_codes8<INT8>(a, inv);
    reinterpret_cast<uint2*>(row)[cb] = rq_codes8<INT8>(b, inv);
    if (first) {
      float s = top >= kRqTiny ? __fdiv_rn(top, rq_qmax<INT8>()) : 0.0f;
      if (!(top <= 3.402823466e38f)) s = __uint_as_float(0x7FC00000u);
      *scale = s;
    }
  }
}

// A CTA takes groups of T tokens, 8 / T warps a token. A group's angles are formed once, a thread one
// or two, into one of two buffers while the group before it is worked on (its positions are asked for
// before that), with one barrier a group. Each warp takes steps of 32 / (D / 16)
// heads, q's first, then k's and v's. A step's rows come through a ring of the warp's own (cp.async,
// each lane the pieces that it reads), three steps ahead of the current one and on into the next group.
// `parts` CTAs share a token's steps where there are few tokens. CACHE: k and v go to the cache (else
// k to k_out).
// A lane's chunks: with rotated halves a pair of chunks `half` apart (of the first 2 half of a row; of
// the others one from either half of them), so that the pairs (i, i + pairs) lie in one lane for a part
// of a head too; else one from either half of the row.
// Bound: the issue of instructions before HBM, so two CTAs an SM with registers for all: at three a
// third more instructions went into forming addresses again (8192 tokens of 48 + 8 heads into E4M3:
// 53.4 us, 49.2 with two). Measured: these 45.3 us (82% of the copy's 6754.5 GB/s), q and k of 4352
// tokens of 24 + 24 heads over three axes 18.7 (85%; 55% of the issue slots), one token 2.7 to 3.0.

// 1 / sqrt(x): the approximate instruction (2^-22) and one Newton step, within an ulp.
__device__ __forceinline__ float heads_rsqrt(float x) {
  float y;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return __fmaf_rn(0.5f * y, __fmaf_rn(-x * y, y, 1.0f), y);
}

template <int N>
struct Kind {
  static constexpr int value = N;
};
constexpr int kHeadsThreads = 256, kHeadsWarps = 8, kHeadsTokens = 8, kHeadsStages = 4, kHeadsAngles = 2;

template <int D, int ROPE, bool CACHE, int TYPE>
__global__ void __launch_bounds__(kHeadsThreads, 2) heads_kernel(const __grid_constant__ HeadsParams P) {
  constexpr int LPH = D / 16, HPW = 32 / LPH, PAIRS = D / 2;
  __shared__ RopeTable table;
  __shared__ __align__(16) float cos_s[2][ROPE ? kHeadsAngles * kHeadsThreads : 1];
  __shared__ __align__(16) float sin_s[2][ROPE ? kHeadsAngles * kHeadsThreads : 1];
  __shared__ uint4 ring_s[kHeadsWarps][kHeadsStages][2][32];
  __shared__ float4 weight_s[2][D / 4];  // q's, k's: values 0-3 of each chunk, then values 4-7
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane / LPH, u = lane % LPH;
  const int T = P.group_tokens, warps = kHeadsWarps / T;  // of a token, in this CTA
  const int mine = warp / warps;                          // this warp's token in the group
  wait_for_producers();
  allow_dependents();
  const int pairs = ROPE ? P.rope.pairs : 0;
  const int half = ROPE == kRopeHalves ? pairs / 8 : LPH;
  const int ca = u < half ? u : u + half, cb = u < half ? u + half : u + LPH;
  const int q_steps = (P.q_heads + HPW - 1) / HPW, kv_steps = (P.kv_heads + HPW - 1) / HPW;
  const int steps = q_steps + (CACHE ? 2 : 1) * kv_steps;
  const int64_t groups = (P.tokens + T - 1) / T;
  const int step0 = (blockIdx.x % P.parts) * warps + (warp - mine * warps), stride = P.parts * warps;
  const int grid = gridDim.x / P.parts;
  // The next step to copy: its head's row, at strides of `ahead` heads within q, k and v.
  const int ahead = stride * HPW;
  int64_t f_group = blockIdx.x / P.parts;
  int f_step = step0, f_end = 0, f_h = 0, f_heads = 0, fs = 0;
  const uint16_t *f_src = nullptr, *f_row = nullptr;  // the head's row; some row of the token
  bool f_more = false;
  const uint32_t ring = smem_addr(&ring_s[warp][0][0][lane]);
  auto f_start = [&]() {
    const int64_t token = f_group * T + mine;
    f_more = f_step < steps && token < P.tokens;
    if (!f_more) return;
    const int kind = f_step < q_steps ? 0 : f_step < q_steps + kv_steps ? 1 : 2;
    const int begin = kind == 0 ? 0 : kind == 1 ? q_steps : q_steps + kv_steps;
    f_end = kind == 0 ? q_steps : begin + kv_steps;
    f_heads = kind == 0 ? P.q_heads : P.kv_heads;
    f_h = (f_step - begin) * HPW + g;
    f_row = kind == 0 ? P.q + token * P.q_ld : kind == 1 ? P.k + token * P.k_ld : P.v + token * P.v_ld;
    f_src = f_row + int64_t(f_h) * D;
  };
  auto fetch = [&]() {
    if (f_more) {
      const bool in = f_h < f_heads;
      const uint4* row = reinterpret_cast<const uint4*>(in ? f_src : f_row);
      cp_async_if(ring + fs, row + ca, in);
      cp_async_if(ring + fs + 512, row + cb, in);
      f_step += stride;
      f_h += ahead;
      f_src += ahead * D;
      if (f_step >= f_end) {
        if (f_step >= steps) f_step = step0, f_group += grid;
        f_start();
      }
    }
    cp_async_commit();
    fs = fs == (kHeadsStages - 1) * 1024 ? 0 : fs + 1024;
  };
  f_start();
#pragma unroll 1
  for (int i = 0; i < kHeadsStages - 1; ++i) fetch();

  // the weights and the rotation's table, all their loads under way at once
  static_assert(PAIRS <= kHeadsThreads && 2 * D <= 2 * kHeadsThreads, "an entry or two a thread");
  uint32_t wv[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = threadIdx.x + j * kHeadsThreads;
    const uint16_t* w = i >= D ? P.k_weight : P.q_weight;
    if (i < 2 * D && w) wv[j] = w[i % D];
  }
  if constexpr (ROPE != kRopeNone) {
    if (threadIdx.x < pairs) {
      const int axis = P.rope.axis ? P.rope.axis[threadIdx.x] : 0;
      table.step[threadIdx.x] = rope_step(P.rope.inv_freq[threadIdx.x]);
      table.axis[threadIdx.x] = min(max(axis, 0), P.rope.axes - 1);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = threadIdx.x + j * kHeadsThreads, x = i % D;
    if (i < 2 * D)
      reinterpret_cast<float*>(weight_s[i / D])[(x & 4) * (D / 8) + (x >> 3) * 4 + (x & 3)] =
          __uint_as_float(wv[j] << 16);
  }
  __syncthreads();
  // The thread's angles of the group to come, and this warp's slot there.
  int64_t position[kHeadsAngles] = {}, slot_next = 0;
  auto ask = [&](int64_t group) {
    if (group >= groups) return;
    if constexpr (ROPE != kRopeNone) {
#pragma unroll
      for (int j = 0; j < kHeadsAngles; ++j) {
        const int i = threadIdx.x + j * kHeadsThreads, t = i / PAIRS, pair = i % PAIRS;
        if (t < T && pair < pairs && group * T + t < P.tokens)
          position[j] = rope_position(P.rope, table.axis[pair], group * T + t);
      }
    }
    if (CACHE && group * T + mine < P.tokens) slot_next = P.slots[group * T + mine];
  };
  auto form = [&](int buffer) {
    if constexpr (ROPE != kRopeNone) {
#pragma unroll
      for (int j = 0; j < kHeadsAngles; ++j) {
        const int i = threadIdx.x + j * kHeadsThreads, t = i / PAIRS, pair = i % PAIRS;
        if (t < T && pair < pairs)
          turn_cos_sin(uint32_t((uint64_t(position[j]) * table.step[pair]) >> 32), cos_s[buffer][i],
                       sin_s[buffer][i]);
      }
    }
  };
  int stage = 0;
  auto work = [&](int64_t token, int64_t slot, int buffer) {
    if (token >= P.tokens) return;
    // cos and sin of the lane's pairs, two to a word pair
    f2 cs[ROPE ? 4 : 1], sn[ROPE ? 4 : 1];
    if constexpr (ROPE != kRopeNone) {
      const int p0 = mine * PAIRS + u * (ROPE == kRopeHalves ? 8 : 4);
      const int p1 = p0 + (ROPE == kRopeHalves ? 4 : D / 4);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float4 c = *reinterpret_cast<const float4*>(&cos_s[buffer][x ? p1 : p0]);
        const float4 s = *reinterpret_cast<const float4*>(&sin_s[buffer][x ? p1 : p0]);
        cs[2 * x] = f2_make(c.x, c.y), cs[2 * x + 1] = f2_make(c.z, c.w);
        sn[2 * x] = f2_make(s.x, s.y), sn[2 * x + 1] = f2_make(s.z, s.w);
      }
    }
    // where this token's k and v go
    int64_t page = 0;
    int at = 0;
    bool store = true;
    if (CACHE) {
      store = slot >= 0 && slot < P.cache.pages * P.cache.page_size;
      if (store) {
        page = page_of(slot, P.cache.page_magic);
        at = int(slot - page * P.cache.page_size);
      } else if (slot >= 0 && lane == 0) {
        report_device_error(kDevErrBadIndex);
      }
    }
    int step = step0;
    // The steps of q, k or v: heads from `h` on.
    auto run = [&](auto what, int begin, int end, int heads) {
      constexpr int KIND = decltype(what)::value;
      constexpr bool TO_CACHE = CACHE && KIND > 0;
      constexpr int E = TYPE == kCacheBf16 ? 2 : 1;
      int h = (step - begin) * HPW + g;
      uint16_t* dst = nullptr;
      uint8_t* to = nullptr;
      float* scale = nullptr;
      if constexpr (TO_CACHE) {
        const int64_t row = int64_t(h) * P.cache.page_size + at;
        to = (KIND == 1 ? P.cache.k + page * P.cache.k_stride : P.cache.v + page * P.cache.v_stride) +
             row * (D * E);
        scale = KIND == 1 ? P.cache.k_scale + page * P.cache.ks_stride + row
                          : P.cache.v_scale + page * P.cache.vs_stride + row;
      } else {
        dst = (KIND == 0 ? P.q_out + token * P.q_out_ld : P.k_out + token * P.k_out_ld) + int64_t(h) * D;
      }
      const uint4* weight = reinterpret_cast<const uint4*>(KIND == 0 ? P.q_weight : P.k_weight);
      for (; step < end; step += stride) {
        fetch();
        cp_async_wait<kHeadsStages - 1>();
        f2 a[4], b[4];
        unpack8(lds_words(ring + stage), a);
        unpack8(lds_words(ring + stage + 512), b);
        stage = stage == (kHeadsStages - 1) * 1024 ? 0 : stage + 1024;
        if (KIND < 2 && weight) {
          f2 s0 = mul2(a[0], a[0]), s1 = mul2(b[0], b[0]);
#pragma unroll
          for (int j = 1; j < 4; ++j) s0 = fma2(a[j], a[j], s0), s1 = fma2(b[j], b[j], s1);
          s0 = add2(s0, s1);
          float sum = f2_lo(s0) + f2_hi(s0);
#pragma unroll
          for (int o = 1; o < LPH; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          const float r = heads_rsqrt(__fmaf_rn(sum, 1.0f / D, P.eps));
          const f2 rr = f2_make(r, r);
          const float4* w = weight_s[KIND & 1];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float4 p = w[x * (D / 8) + ca], q = w[x * (D / 8) + cb];
            a[2 * x] = mul2(mul2(a[2 * x], rr), f2_make(p.x, p.y));
            a[2 * x + 1] = mul2(mul2(a[2 * x + 1], rr), f2_make(p.z, p.w));
            b[2 * x] = mul2(mul2(b[2 * x], rr), f2_make(q.x, q.y));
            b[2 * x + 1] = mul2(mul2(b[2 * x + 1], rr), f2_make(q.z, q.w));
          }
        }
        if constexpr (KIND < 2 && ROPE == kRopeHalves) {
          auto turn = [&]() {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const f2 x = a[j], y = b[j];
              a[j] = fma2(y, neg2(sn[j]), mul2(x, cs[j]));
              b[j] = fma2(x, sn[j], mul2(y, cs[j]));
            }
          };
          if (half == LPH) turn();  // (no lane apart)
          else if (u < half) turn();
        } else if constexpr (KIND < 2 && ROPE == kRopePairs) {
          auto turn = [&](f2 v, int j) {
            const float c = (j & 1) ? f2_hi(cs[j / 2]) : f2_lo(cs[j / 2]);
            const float s = (j & 1) ? f2_hi(sn[j / 2]) : f2_lo(sn[j / 2]);
            const float x = f2_lo(v), y = f2_hi(v);
            return f2_make(x * c - y * s, y * c + x * s);
          };
          if (pairs == PAIRS) {
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] = turn(a[j], j), b[j] = turn(b[j], 4 + j);
          } else {  // pairs that are not rotated stay: an infinity beside a zero sine would not
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (u * 4 + j < pairs) a[j] = turn(a[j], j);
              if (D / 4 + u * 4 + j < pairs) b[j] = turn(b[j], 4 + j);
            }
          }
        }
        const bool live = h < heads;
        if constexpr (TO_CACHE) {
          store_row<D, TYPE>(a, b, ca, cb, u == 0, live && store, to, scale);
          to += int64_t(ahead) * P.cache.page_size * (D * E);
          scale += ahead * P.cache.page_size;
        } else {
          if (live) {
            uint4* row = reinterpret_cast<uint4*>(dst);
            row[ca] = pack8(a);
            row[cb] = pack8(b);
          }
          dst += ahead * D;
        }
        h += ahead;
      }
    };
    run(Kind<0>(), 0, q_steps, P.q_heads);
    run(Kind<1>(), q_steps, q_steps + kv_steps, P.kv_heads);
    if constexpr (CACHE) run(Kind<2>(), q_steps + kv_steps, steps, P.kv_heads);
  };
  int buffer = 0;
  ask(blockIdx.x / P.parts);
  form(0);
  for (int64_t group = blockIdx.x / P.parts; group < groups; group += grid, buffer ^= 1) {
    const int64_t token = group * T + mine, slot = slot_next;
    if (ROPE != kRopeNone) __syncthreads();
    ask(group + grid);
    work(token, slot, buffer);
    form(buffer ^ 1);
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
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// A CTA takes 16 output rows, that is tokens: their places are looked up once, then each lane copies
// 16 bytes of one head's row at a time, tokens first (a page holds a head's tokens side by side), four
// of them under way at once. Measured: 16 sequences of 100 to 16384 tokens of 8 heads, bf16 160 us (100% of
// the copy's rate), E4M3 135.6 (89%), int8 146 (83%: conversions); 32 rows a CTA the same for these and
// 4.2 for 3.0 us where there are few, 64 rows 142 and 154.
constexpr int kReadAhead = 4;

template <int D, int TYPE>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const __grid_constant__ ReadParams P) {
  constexpr bool QUANT = TYPE != kCacheBf16;
  constexpr int E = QUANT ? 1 : 2, LPR = D * E / 16;  // lanes a row
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
  for (int i0 = threadIdx.x; i0 < work; i0 += kReadThreads * kReadAhead) {
    uint4 x[kReadAhead];
    float s[kReadAhead];
    uint16_t* dst[kReadAhead];
#pragma unroll
    for (int j = 0; j < kReadAhead; ++j) {
      const int i = i0 + j * kReadThreads;
      const int u = i % LPR, r = (i / LPR) % kReadRows, hk = i / (LPR * kReadRows);
      const int h = hk >> 1;
      const bool is_v = hk & 1;
      const int64_t page = i < work ? page_s[r] : -1;
      x[j] = make_uint4(0, 0, 0, 0);
      s[j] = 0.0f;
      // (-1: not a row of any sequence)
      dst[j] = page == -1 ? nullptr : (is_v ? P.v : P.k) + ((row0 + r) * H + h) * D + u * (16 / E);
      if (page >= 0) {
        const int64_t at = int64_t(h) * P.cache.page_size + at_s[r];
        const uint8_t* src = (is_v ? P.cache.v + page * P.cache.v_stride
                                   : P.cache.k + page * P.cache.k_stride) + at * (D * E) + u * 16;
        x[j] = ld_stream(reinterpret_cast<const uint4*>(src));
        if (QUANT)
          s[j] = is_v ? P.cache.v_scale[page * P.cache.vs_stride + at]
                      : P.cache.k_scale[page * P.cache.ks_stride + at];
      }
    }
#pragma unroll
    for (int j = 0; j < kReadAhead; ++j) {
      if (!dst[j]) continue;
      uint4* to = reinterpret_cast<uint4*>(dst[j]);
      if (QUANT) {
        st_stream(to, dequant8<TYPE>(make_uint2(x[j].x, x[j].y), s[j]));
        st_stream(to + 1, dequant8<TYPE>(make_uint2(x[j].z, x[j].w), s[j]));
      } else {
        st_stream(to, x[j]);
      }
    }
  }
}

}  // namespace fp8q
