// paged_attention_kernels.cuh -- attention of one new token per sequence over a paged cache (sm_103a).
//
//   s_t = scale q . k_t,  o = sum_t exp(s_t) v_t / sum_t exp(s_t),  t in [max(0, len - window), len)
//
// Each k and v row is read once; with G query heads a key/value head that is 4 G flops a value, so HBM
// bounds it up to about a hundred heads. What matters is that loads never pause and that the
// instructions a byte stay few.
//
// A warp takes tiles of 16 tokens of one key/value head, its own running maximum, sum and
// accumulators, through a ring of its own: every lane copies (cp.async) exactly the 16-byte pieces
// that it will read, so that the ring needs no barrier and no swizzle. The products run on mma.sync
// m16n8k16 with the tokens as rows of S^T = K Q^T and the head's values as rows of O^T = V^T P^T: the
// eight columns are query heads, so a group of up to eight costs one product. (tcgen05 takes both
// operands or one from shared memory in its own layout, and needs 8-bit codes converted there; at
// these sizes the tensor rate does not bound.) The order of a head's values within S's sum is free,
// as is that of its values among O's rows, so both follow the 16-byte pieces.
//
// int8 and E4M3 codes are exact in fp16. q (bf16) goes to fp16 times a power of two for each head,
// exact down to 2^-24 of its head's largest value. A token's key scale multiplies its logit; its
// value scale its weight, which is rounded to fp16 (2^-12 relative, against the output's 2^-9).
// Over a bf16 cache the weights go as two bf16 (16 bits of them).
//
// Weights are taken relative to a running maximum that is only raised when a logit exceeds it by
// 2^6 (a vote, no shuffles in most tiles); with value scales, a second factor keeps the fp16 weights
// below 2^15.
#pragma once

#include "cache_kernels.cuh"
#include "int8_matmul_few_kernels.cuh"
#include "int8_matmul_kernels.cuh"

namespace fp8q {

struct AttnParams {
  const uint16_t* q;  // [batch, q_heads, D], row stride q_ld
  int64_t q_ld;
  CacheView cache;
  const int32_t* table;
  int64_t table_ld;
  const int32_t* lengths;
  uint16_t* out;  // [batch, q_heads, D]
  float* lse;     // [batch, q_heads] or null
  float* part_o;  // partial sums of pieces: [2 grid][heads of a block][D]
  float* part_ml;  // [2 grid][heads of a block][2]: maximum (log2 units), sum
  int batch, width, window;  // width: pages a sequence may have
  int q_heads, group, blocks;  // heads a key/value head; blocks of 8 NT of them
  int grid;  // CTAs of the attention kernel
  float scale_log2;
  uint32_t tile_magic;  // ceil(2^32 / (page_size / 16))
  int page_tiles;
};

constexpr float kAttnNone = -1e30f;  // the maximum before any token

template <int TYPE, int D, int NT>
struct AttnLayout {
  static constexpr int E = TYPE == kCacheBf16 ? 2 : 1;
  static constexpr int kWarps = D * E >= 512 ? 4 : 8;
  static constexpr int KP = D * E / 64;   // 16-byte pieces of a key row a lane (four lanes a row)
  static constexpr int VB = D * E >= 128 ? 16 : 8;  // bytes of a value piece (eight lanes a row)
  static constexpr int VP = D * E / (8 * VB);
  static constexpr int kHalf = 16 * D * E;  // a tile's keys
  static constexpr int kScales = TYPE == kCacheBf16 ? 0 : 128;
  static constexpr int kStage = 2 * kHalf + kScales;
  static constexpr int kMergePass = 4;  // blocks of 16 values merged at a time
  static constexpr int kMerge = kWarps * kMergePass * 128 * 4;
  static constexpr int kStats = kWarps * 8 * NT * 2 * 4;
  static constexpr int kRoom = (232448 - kMerge - kStats) / (kWarps * kStage);
  static constexpr int kStages = kRoom < 6 ? kRoom : 6;
  static constexpr int kBytes = kWarps * kStages * kStage + kMerge + kStats;
  static constexpr int MT = D / 16;
};

// A sequence's tiles: [first, first + n), its tokens [lo, hi).
struct AttnSpan {
  int lo, hi, first, n;
};
__device__ __forceinline__ AttnSpan attn_span(const AttnParams& P, int b) {
  AttnSpan s;
  s.hi = min(max(P.lengths[b], 0), P.width * P.cache.page_size);
  s.lo = P.window > 0 ? max(s.hi - P.window, 0) : 0;
  s.first = s.lo >> 4;
  s.n = ((s.hi + 15) >> 4) - s.first;
  return s;
}

// tile / page_tiles: by the ceiling's product where tile * page_tiles < 2^32 (the host's limits).
__device__ __forceinline__ int attn_page(const AttnParams& P, int tile) {
  return P.page_tiles == 1 ? tile : int(__umulhi(uint32_t(tile), P.tile_magic));
}

// The work's split, found by each warp from the lengths: all tiles in one order (sequence, block of
// heads, tile), an equal share of them for each CTA; or, where the segments (a sequence's tiles for one
// block of heads) are short, whole segments for each CTA or each warp.

// The sequence that holds tile `at` of a block of heads, and the tiles before it.
struct AttnPlace {
  int b;
  int64_t before;
};

// Totals over the sequences; with `want` >= 0 also the sequence that holds that tile.
__device__ __forceinline__ int64_t attn_scan(const AttnParams& P, int& most, int64_t& mine,
                                             int64_t& incl) {
  const int lane = threadIdx.x & 31;
  const int per = (P.batch + 31) >> 5, b0 = min(lane * per, P.batch), b1 = min(b0 + per, P.batch);
  mine = 0;
  most = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = attn_span(P, b).n;
    mine += n;
    most = max(most, n);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  return __shfl_sync(0xffffffffu, incl, 31);
}

__device__ __forceinline__ AttnPlace attn_find(const AttnParams& P, int64_t mine, int64_t incl,
                                               int64_t want) {
  const int per = (P.batch + 31) >> 5;
  const unsigned has = __ballot_sync(0xffffffffu, want < incl);
  AttnPlace r;
  if (has == 0) {  // past the last
    r.b = P.batch;
    r.before = __shfl_sync(0xffffffffu, incl, 31);
    return r;
  }
  const int owner = __ffs(has) - 1;
  int64_t before = __shfl_sync(0xffffffffu, incl - mine, owner);
  int b = owner * per;
  for (;; ++b) {  // (ends within the owner's sequences: their sum passes `want`)
    const int n = attn_span(P, b).n;
    if (want < before + n) break;
    before += n;
  }
  r.b = b;
  r.before = before;
  return r;
}

// How the tiles are shared out (never by tile where no sequence has more than W: the host launches
// no join then). kByTile: CTA c takes tiles [c, c + 1) * quota of all; kBySegment: CTA
// c the segments c, c + grid, ...; kByWarp: each warp its own segments.
constexpr int kByTile = 0, kBySegment = 1, kByWarp = 2;
struct AttnSplit {
  int mode;
  int64_t quota;
};
template <int W>
__device__ __forceinline__ AttnSplit attn_split(const AttnParams& P, int64_t tiles, int most) {
  const int64_t heads = int64_t(P.cache.heads) * P.blocks;
  const int64_t all = tiles * heads, segments = heads * P.batch;
  AttnSplit s;
  s.mode = kByTile;
  s.quota = max((all + P.grid - 1) / P.grid, int64_t(1));
  // rounds of a tile a warp: shared by tiles, whole segments a CTA, whole segments a warp
  const int64_t by_tile = (s.quota + W - 1) / W + 2 * (1 + s.quota * segments / max(all, int64_t(1)));
  const int64_t per_cta = (segments + P.grid - 1) / P.grid;
  const int64_t by_segment = per_cta * ((most + W - 1) / W + 2) - 1;
  const int64_t by_warp = (segments + int64_t(P.grid) * W - 1) / (int64_t(P.grid) * W) * (most + 1);
  if (by_segment <= by_tile || most <= W) s.mode = kBySegment;
  if (by_warp <= by_segment && (by_warp <= by_tile || most <= W)) s.mode = kByWarp;
  return s;
}

// ------------------------------------------------------------------------------------------

template <int BYTES>
__device__ __forceinline__ void cp_async_if(uint32_t dst, const void* src, bool in) {
  static_assert(BYTES == 4 || BYTES == 8 || BYTES == 16, "a copy of 4, 8 or 16 bytes");
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(in ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES),
                 "r"(in ? BYTES : 0)
                 : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <int TYPE>
__device__ __forceinline__ void attn_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (TYPE == kCacheBf16) mma_bf16(d, a[0], a[1], a[2], a[3], b0, b1);
  else mma_f16(d, a[0], a[1], a[2], a[3], b0, b1);
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Four codes as two fp16 pairs.
template <int TYPE>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (TYPE == kCacheInt8) {
    int8_to_f16(w, lo, hi);
  } else {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// First value (of two) of rows r and r + 8 in block j of O^T, for row r of the lanes.
template <int TYPE, int D>
__device__ __forceinline__ int attn_value_of(int j, int r) {
  constexpr int E = TYPE == kCacheBf16 ? 2 : 1;
  constexpr int VB = D * E >= 128 ? 16 : 8, per = VB / E / 2;  // blocks a piece
  return ((j / per) * 8 + r) * (VB / E) + (j % per) * 2;
}

template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(AttnLayout<TYPE, D, NT>::kWarps * 32, 1)
    paged_attention_kernel(const __grid_constant__ AttnParams P) {
  using L = AttnLayout<TYPE, D, NT>;
  constexpr bool QUANT = TYPE != kCacheBf16;
  constexpr int W = L::kWarps, S = L::kStages, E = L::E, KP = L::KP, VP = L::VP, MT = L::MT;
  constexpr int KS = QUANT ? 4 : 2;  // matrix steps (16 values of a key row) a piece
  extern __shared__ __align__(128) uint8_t attn_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  uint8_t* ring = attn_smem + warp * (S * L::kStage);
  float* merge = reinterpret_cast<float*>(attn_smem + W * S * L::kStage);
  float* stats = reinterpret_cast<float*>(attn_smem + W * S * L::kStage + L::kMerge);
  allow_dependents();
  wait_for_producers();

  int most;
  int64_t mine, incl;
  const int64_t tiles = attn_scan(P, most, mine, incl);
  const int heads = P.cache.heads * P.blocks;
  const AttnSplit split = attn_split<W>(P, tiles, most);
  const bool by_warp = split.mode == kByWarp, by_tile = split.mode == kByTile;
  const int64_t segments = int64_t(heads) * P.batch;
  const int64_t unit = by_warp ? int64_t(blockIdx.x) * W + warp : blockIdx.x;
  const int64_t units = by_warp ? int64_t(P.grid) * W : P.grid;
  const int step = by_warp ? 1 : W;

  // The first segment (its number) and tile of this unit.
  int64_t seg0 = unit, left0 = INT64_MAX;  // left0: tiles of this CTA's share
  int pos0 = 0;
  if (by_tile) {
    const int64_t t0 = min(split.quota * unit, tiles * heads), t1 = min(t0 + split.quota, tiles * heads);
    if (t0 >= t1) return;
    const AttnPlace at = attn_find(P, mine, incl, t0 / heads);
    const int64_t local = t0 - at.before * heads;
    const int n = attn_span(P, at.b).n;
    seg0 = int64_t(at.b) * heads + local / n;
    pos0 = int(local % n);
    left0 = t1 - t0;
  }
  const int64_t seg_step = by_tile ? 1 : units;

  // ---- the fetching side: the next tile to copy
  int64_t f_seg = seg0, f_left = left0;
  int f_n = 0, f_first = 0, f_lo = 0, f_hi = 0, f_h = 0, f_b = 0;
  int f_pos = pos0 + (by_warp ? 0 : warp);
  int f_used = pos0;  // (by tiles: where this segment's part of the share begins)
  auto f_load = [&]() {
    f_b = int(f_seg / heads);
    f_h = int(f_seg - int64_t(f_b) * heads) / P.blocks;
    const AttnSpan s = attn_span(P, f_b);
    f_n = s.n;
    f_first = s.first;
    f_lo = s.lo;
    f_hi = s.hi;
  };
  bool f_more = f_seg < segments;
  if (f_more) f_load();
  // Moves on to a segment that has the tile f_pos.
  auto f_settle = [&]() {
    while (f_more) {
      const int end = int(min(int64_t(f_n), f_used + f_left));  // of this segment's part
      if (f_pos < end) return;
      const int over = by_tile ? f_pos - end : warp;  // the tiles go round the warps
      if (by_tile) f_left -= end - f_used;
      f_used = 0;
      f_seg += seg_step;
      f_more = f_seg < segments && f_left > 0;
      if (!f_more) return;
      f_pos = by_warp ? 0 : over;
      f_load();
    }
  };
  int f_page = -1;
  auto f_lookup = [&]() {
    if (f_more) {
      f_page = P.table[f_b * P.table_ld + attn_page(P, f_first + f_pos)];
    }
  };
  uint32_t bad = 0;  // which of the tiles under way have no page, the newest in bit 0
  int fs = 0;
  auto fetch = [&]() {
    bad <<= 1;
    if (f_more) {
      const int tile = f_first + f_pos;
      const int in_page = tile - attn_page(P, tile) * P.page_tiles;
      const bool fine = f_page >= 0 && f_page < P.cache.pages;
      if (!fine) {
        bad |= 1;
        if (lane == 0) report_device_error(kDevErrBadIndex);
      }
      const int64_t page = fine ? f_page : 0;
      const int lo = fine ? f_lo - tile * 16 : 16, hi = fine ? f_hi - tile * 16 : 0;
      const int64_t row = int64_t(f_h) * P.cache.page_size + in_page * 16;
      const uint32_t dst = smem_addr(ring + fs * L::kStage);
      const uint8_t* k = P.cache.k + page * P.cache.k_stride + row * (D * E);
      const uint8_t* v = P.cache.v + page * P.cache.v_stride + row * (D * E);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = r + 8 * i;
        const bool in = t >= lo && t < hi;
#pragma unroll
        for (int p = 0; p < KP; ++p)
          cp_async_if<16>(dst + ((i * KP + p) * 32 + lane) * 16, k + t * (D * E) + p * 64 + c * 16, in);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 2 * c + (i & 1) + 8 * (i >> 1);
        const bool in = t >= lo && t < hi;
#pragma unroll
        for (int p = 0; p < VP; ++p)
          cp_async_if<L::VB>(dst + L::kHalf + ((i * VP + p) * 32 + lane) * L::VB,
                             v + t * (D * E) + (p * 8 + r) * L::VB, in);
      }
      if (QUANT) {
        const int t = r + 8 * (c & 1);
        const float* s = c < 2 ? P.cache.k_scale + page * P.cache.ks_stride
                               : P.cache.v_scale + page * P.cache.vs_stride;
        cp_async_if<4>(dst + 2 * L::kHalf + (c * 8 + r) * 4, s + row + t, t >= lo && t < hi);
      }
      f_pos += step;
      f_settle();
      f_lookup();
    }
    cp_async_commit();
    fs = fs + 1 == S ? 0 : fs + 1;
  };
  f_settle();
  f_lookup();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch();

  // ---- the computing side
  int cs = 0;
  int turn = 0;  // (by tiles: the warp that takes the segment's first tile)
  int64_t left = left0;
  for (int64_t seg = seg0; seg < segments && left > 0; seg += seg_step) {
    const int b = int(seg / heads), hb = int(seg - int64_t(b) * heads);
    const int h = hb / P.blocks, block = hb - h * P.blocks;
    const AttnSpan span = attn_span(P, b);
    const int begin = seg == seg0 ? pos0 : 0;
    const int end = int(min(int64_t(span.n), begin + left));
    if (by_tile && span.n == 0) continue;
    const int count = end - begin;
    left -= by_tile ? count : 0;
    const int head0 = h * P.group + block * 8 * NT;          // first query head of the block
    const int live = min(8 * NT, P.group - block * 8 * NT);  // query heads in it

    // q as the columns of S^T: the values that face this lane's part of a key row
    uint32_t qf[NT][KP * KS][2];
    float fac[NT][2];  // logits in log2 units, for the lane's two heads
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = j * 8 + r;
      const uint4* row = reinterpret_cast<const uint4*>(P.q + b * P.q_ld + int64_t(head0 + n) * D);
      uint4 x[KP * KS / 2];
#pragma unroll
      for (int p = 0; p < KP; ++p)
#pragma unroll
        for (int i = 0; i < KS / 2; ++i)
          x[p * (KS / 2) + i] = n < live ? row[(p * 4 + c) * (KS / 2) + i] : make_uint4(0, 0, 0, 0);
      if (!QUANT) {
#pragma unroll
        for (int i = 0; i < KP * KS / 2; ++i) {
          qf[j][2 * i][0] = x[i].x, qf[j][2 * i][1] = x[i].y;
          qf[j][2 * i + 1][0] = x[i].z, qf[j][2 * i + 1][1] = x[i].w;
        }
        fac[j][0] = fac[j][1] = P.scale_log2;
      } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < KP * KS / 2; ++i)
          m = max_u16x2(max_u16x2(m, x[i].x & 0x7FFF7FFFu),
                        max_u16x2(x[i].y & 0x7FFF7FFFu,
                                  max_u16x2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu)));
        uint32_t e = max(m & 0xFFFFu, m >> 16) >> 7;  // exponent of the head's largest value
        e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
        e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
        e = min(max(e, 10u), 244u);  // (smaller ones count as zero in effect, larger ones overflow)
        const float up = __uint_as_float((254u - e + 8u) << 23);  // 2^(127 + 8 - e): below 2^9
#pragma unroll
        for (int i = 0; i < KP * KS / 2; ++i) {
          const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int w = 0; w < 4; ++w)
            qf[j][2 * i + w / 2][w & 1] = pack_f16x2(bf_lo(u[w]) * up, bf_hi(u[w]) * up);
        }
        const float down = P.scale_log2 * __uint_as_float((e - 8u) << 23);  // 2^(e - 8 - 127)
        fac[j][0] = __shfl_sync(0xffffffffu, down, 8 * c);
        fac[j][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
      }
    }

    float o[NT][MT][4];
    float m[NT][2], l[NT][2], kf[NT][2];  // maximum, this lane's sum, weights' factor
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[j][i][x] = 0.0f;
#pragma unroll
      for (int x = 0; x < 2; ++x) m[j][x] = kAttnNone, l[j][x] = 0.0f, kf[j][x] = 0x1p100f;
    }

    const int start = by_warp ? begin : begin + ((warp - turn) & (W - 1));
    for (int pos = start; pos < end; pos += step) {
      __syncwarp();  // (the stage that fetch() overwrites has been read by all lanes)
      fetch();
      cp_async_wait<S - 1>();
      __syncwarp();
      const uint8_t* stage = ring + cs * L::kStage;
      cs = cs + 1 == S ? 0 : cs + 1;
      if ((bad >> (S - 1)) & 1) continue;

      // S^T
      float s[NT][2][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[j][0][x] = s[j][1][x] = 0.0f;
#pragma unroll
      for (int p = 0; p < KP; ++p) {
        const uint4* at = reinterpret_cast<const uint4*>(stage) + p * 32 + lane;
        const uint4 x4 = at[0], y4 = at[KP * 32];
        const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w}, y[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
        for (int w = 0; w < KS; ++w) {
          uint32_t a[4];
          if (QUANT) {
            codes_to_f16<TYPE>(x[w], a[0], a[2]);
            codes_to_f16<TYPE>(y[w], a[1], a[3]);
          } else {
            a[0] = x[(2 * w) & 3], a[2] = x[(2 * w + 1) & 3];
            a[1] = y[(2 * w) & 3], a[3] = y[(2 * w + 1) & 3];
          }
#pragma unroll
          for (int j = 0; j < NT; ++j)
            attn_mma<TYPE>(s[j][w & 1], a, qf[j][p * KS + w][0], qf[j][p * KS + w][1]);
        }
      }

      // weights
      float ks[2] = {1.0f, 1.0f}, vs[2] = {1.0f, 1.0f};
      if (QUANT) {
        const float* sc = reinterpret_cast<const float*>(stage + 2 * L::kHalf) + r;
        ks[0] = sc[0], ks[1] = sc[8], vs[0] = sc[16], vs[1] = sc[24];
      }
      const int tok0 = (span.first + pos) * 16;
      const bool edge = tok0 < span.lo || tok0 + 16 > span.hi;
      float t[NT][4], w[NT][4];
      bool over = false;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          t[j][x] = (s[j][0][x] + s[j][1][x]) * fac[j][x & 1];
          if (QUANT) t[j][x] *= ks[x >> 1];
        }
      }
      if (edge) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int tok = tok0 + r + 8 * (x >> 1);
            if (tok < span.lo || tok >= span.hi) t[j][x] = -INFINITY;
          }
      }
      float p[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          p[j][x] = ex2(t[j][x] - m[j][x & 1]);
          w[j][x] = QUANT ? p[j][x] * kf[j][x & 1] * vs[x >> 1] : p[j][x];
          over |= p[j][x] > 64.0f;
          if (QUANT) over |= w[j][x] > 32768.0f;
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float top = fmaxf(t[j][x], t[j][x + 2]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float m1 = fmaxf(m[j][x], top), f = ex2(m[j][x] - m1);
            m[j][x] = m1;
            l[j][x] *= f;
            float gain = f;
            p[j][x] = ex2(t[j][x] - m1);
            p[j][x + 2] = ex2(t[j][x + 2] - m1);
            if (QUANT) {
              float wt = fmaxf(p[j][x] * vs[0], p[j][x + 2] * vs[1]);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) wt = fmaxf(wt, __shfl_xor_sync(0xffffffffu, wt, d));
              // a power of two that takes the tile's largest weight to 2^8 .. 2^9, no larger than
              // what keeps the sums so far from growing
              const int e = min(max(int(__float_as_uint(wt) >> 23) & 255, 27), 227);
              float k1 = __uint_as_float(uint32_t(254 + 8 - e) << 23);
              k1 = fminf(k1, __fdividef(kf[j][x], f));
              gain = __fdividef(k1, kf[j][x]) * f;
              kf[j][x] = k1;
              w[j][x] = p[j][x] * k1 * vs[0];
              w[j][x + 2] = p[j][x + 2] * k1 * vs[1];
            } else {
              w[j][x] = p[j][x];
              w[j][x + 2] = p[j][x + 2];
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) o[j][i][x] *= gain, o[j][i][x + 2] *= gain;
          }
      }
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        l[j][0] += p[j][0] + p[j][2];
        l[j][1] += p[j][1] + p[j][3];
        if (QUANT) {
          ph[j][0] = transpose8x8(pack_f16x2(w[j][0], w[j][1]));
          ph[j][1] = transpose8x8(pack_f16x2(w[j][2], w[j][3]));
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t hi = pack_bf16x2(w[j][2 * i], w[j][2 * i + 1]);
            ph[j][i] = transpose8x8(hi);
            pl[j][i] = transpose8x8(pack_bf16x2(w[j][2 * i] - bf_lo(hi), w[j][2 * i + 1] - bf_hi(hi)));
          }
        }
      }

      // O^T
#pragma unroll
      for (int pc = 0; pc < VP; ++pc) {
        uint32_t x[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* at = stage + L::kHalf + ((i * VP + pc) * 32 + lane) * L::VB;
          if (L::VB == 16) {
            const uint4 y = *reinterpret_cast<const uint4*>(at);
            x[i][0] = y.x, x[i][1] = y.y, x[i][2] = y.z, x[i][3] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2*>(at);
            x[i][0] = y.x, x[i][1] = y.y;
          }
        }
#pragma unroll
        for (int wd = 0; wd < L::VB / 4; ++wd) {
#pragma unroll
          for (int half = 0; half < (QUANT ? 2 : 1); ++half) {
            uint32_t a[4];
            if (QUANT) {
              const uint32_t sel = half ? 0x7362u : 0x5140u;
              codes_to_f16<TYPE>(__byte_perm(x[0][wd], x[1][wd], sel), a[0], a[1]);
              codes_to_f16<TYPE>(__byte_perm(x[2][wd], x[3][wd], sel), a[2], a[3]);
            } else {
              a[0] = __byte_perm(x[0][wd], x[1][wd], 0x5410), a[1] = __byte_perm(x[0][wd], x[1][wd], 0x7632);
              a[2] = __byte_perm(x[2][wd], x[3][wd], 0x5410), a[3] = __byte_perm(x[2][wd], x[3][wd], 0x7632);
            }
            const int i = pc * (L::VB / E / 2) + wd * (QUANT ? 2 : 1) + half;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              attn_mma<TYPE>(o[j][i], a, ph[j][0], ph[j][1]);
              if (!QUANT) attn_mma<TYPE>(o[j][i], a, pl[j][0], pl[j][1]);
            }
          }
        }
      }
    }

    // ---- this warp's sums
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[j][x] += __shfl_xor_sync(0xffffffffu, l[j][x], d);
        if (QUANT) {
          const float inv = 1.0f / kf[j][x];
#pragma unroll
          for (int i = 0; i < MT; ++i) o[j][i][x] *= inv, o[j][i][x + 2] *= inv;
        }
      }
    if (by_warp) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int n = j * 8 + 2 * c + x;
          if (n >= live) continue;
          const int64_t row = int64_t(b) * P.q_heads + head0 + n;
          const float inv = l[j][x] == 0.0f ? 0.0f : 1.0f / l[j][x];
#pragma unroll
          for (int i = 0; i < MT; ++i)
            *reinterpret_cast<uint32_t*>(P.out + row * D + attn_value_of<TYPE, D>(i, r)) =
                pack_bf16x2(o[j][i][x] * inv, o[j][i][x + 2] * inv);
          if (P.lse && r == 0)
            P.lse[row] = l[j][x] == 0.0f ? -INFINITY : (m[j][x] + log2f(l[j][x])) * 0.6931471805599453f;
        }
      continue;
    }
    // ---- the CTA's sums: its warps' joined, 64 values of the head at a time
    if (r == 0) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float* at = stats + (warp * 8 * NT + j * 8 + 2 * c + x) * 2;
          at[0] = m[j][x];
          at[1] = l[j][x];
        }
    }
    const bool whole = begin == 0 && end == span.n;
    const int slot = 2 * blockIdx.x + (seg == seg0 ? 0 : 1);
    constexpr int BP = L::kMergePass;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i0 = 0; i0 < MT; i0 += BP) {
#pragma unroll
        for (int i = 0; i < BP; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            merge[((warp * BP + i) * 4 + x) * 32 + lane] = o[j][i0 + i][x];
        __syncthreads();
        for (int e = threadIdx.x; e < BP * 64; e += W * 32) {
          const int ln = e & 31, x = (e >> 5) & 1, i = e >> 6;
          const int n = j * 8 + 2 * (ln & 3) + x;
          if (n < live) {
            float top = kAttnNone;
#pragma unroll
            for (int v = 0; v < W; ++v) top = fmaxf(top, stats[(v * 8 * NT + n) * 2]);
            float sum = 0.0f, a0 = 0.0f, a1 = 0.0f;
#pragma unroll
            for (int v = 0; v < W; ++v) {
              const float f = ex2(stats[(v * 8 * NT + n) * 2] - top);
              sum += f * stats[(v * 8 * NT + n) * 2 + 1];
              a0 += f * merge[((v * BP + i) * 4 + x) * 32 + ln];
              a1 += f * merge[((v * BP + i) * 4 + x + 2) * 32 + ln];
            }
            const int d = attn_value_of<TYPE, D>(i0 + i, ln >> 2);
            const bool first = i0 == 0 && i == 0 && (ln >> 2) == 0;
            if (whole) {
              const int64_t row = int64_t(b) * P.q_heads + head0 + n;
              const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
              *reinterpret_cast<uint32_t*>(P.out + row * D + d) = pack_bf16x2(a0 * inv, a1 * inv);
              if (P.lse && first)
                P.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
            } else {
              const int64_t row = int64_t(slot) * (8 * NT) + n;
              *reinterpret_cast<float2*>(P.part_o + row * D + d) = make_float2(a0, a1);
              if (first) P.part_ml[2 * row] = top, P.part_ml[2 * row + 1] = sum;
            }
          }
        }
        __syncthreads();
      }
    if (by_tile) turn = (turn + count) & (W - 1);
  }
  cp_async_wait<0>();
}

// Joins the pieces of segments that several CTAs shared: a CTA for each segment and query head.
template <int D, int W, int NT>
__global__ void __launch_bounds__(D / 2) attn_join_kernel(const __grid_constant__ AttnParams P) {
  wait_for_producers();
  allow_dependents();
  int most;
  int64_t mine, incl;
  const int64_t tiles = attn_scan(P, most, mine, incl);
  const AttnSplit split = attn_split<W>(P, tiles, most);
  if (split.mode != kByTile) return;
  const int heads = P.cache.heads * P.blocks;
  const int b = blockIdx.x / heads, hb = blockIdx.x - b * heads;
  const int h = hb / P.blocks, block = hb - h * P.blocks, n = blockIdx.y;
  if (n >= min(8 * NT, P.group - block * 8 * NT)) return;
  // tiles before sequence b
  const int per = (P.batch + 31) >> 5, owner = b / per;
  int64_t before = __shfl_sync(0xffffffffu, incl - mine, owner);
  for (int i = owner * per; i < b; ++i) before += attn_span(P, i).n;
  const int count = attn_span(P, b).n;
  const int64_t row = int64_t(b) * P.q_heads + h * P.group + block * 8 * NT + n;
  if (count == 0) {  // no token: no CTA has it
    *reinterpret_cast<uint32_t*>(P.out + row * D + 2 * threadIdx.x) = 0u;
    if (P.lse && threadIdx.x == 0) P.lse[row] = -INFINITY;
    return;
  }
  const int64_t s0 = before * heads + int64_t(hb) * count, s1 = s0 + count;
  const int64_t c0 = s0 / split.quota, c1 = (s1 - 1) / split.quota;
  if (c0 == c1) return;  // whole
  auto slot = [&](int64_t cta) {  // 0 where the piece is its CTA's first
    const bool first = cta > c0 || s0 == c0 * split.quota;
    return (2 * cta + (first ? 0 : 1)) * (8 * NT) + n;
  };
  float top = kAttnNone;
  for (int64_t i = c0; i <= c1; ++i) top = fmaxf(top, P.part_ml[2 * slot(i)]);
  float sum = 0.0f, a0 = 0.0f, a1 = 0.0f;
  for (int64_t i = c0; i <= c1; ++i) {
    const int64_t at = slot(i);
    const float f = ex2(P.part_ml[2 * at] - top);
    const float2 v = *reinterpret_cast<const float2*>(P.part_o + at * D + 2 * threadIdx.x);
    sum += f * P.part_ml[2 * at + 1];
    a0 += f * v.x;
    a1 += f * v.y;
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  *reinterpret_cast<uint32_t*>(P.out + row * D + 2 * threadIdx.x) = pack_bf16x2(a0 * inv, a1 * inv);
  if (P.lse && threadIdx.x == 0)
    P.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace fp8q
