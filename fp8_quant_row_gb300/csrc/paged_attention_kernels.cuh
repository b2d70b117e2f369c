// paged_attention_kernels.cuh -- attention of one new token per sequence over a paged cache (sm_103a).
//
//   s_t = scale q . k_t,  o = sum_t exp(s_t) v_t / sum_t exp(s_t),  t in [max(0, len - window), len)
//
// Each k and v row is read once; with G query heads a key/value head that is 4 G flops a value, so HBM
// bounds it up to about a hundred heads. What matters is that loads never pause and that the
// instructions a byte stay few.
//
// A warp takes tiles of 16 tokens of one key/value head, its own running maximum, sum and
// accumulators, through a ring of its own: one lane asks for a tile's keys and values by TMA (boxes of
// 128 bytes x 16 tokens, 128-byte swizzle), the scales by bulk copies. (Copies of 16 bytes a lane,
// cp.async, kept to 4.5 TB/s: 66.6 us for 32 sequences of 4000 in E4M3, 8 heads, 53 with bulk copies.)
// The products run on mma.sync
// m16n8k16 with the tokens as rows of S^T = K Q^T and the head's values as rows of O^T = V^T P^T: the
// eight columns are query heads, so a group of up to eight costs one product. (tcgen05 takes both
// operands or one from shared memory in its own layout, and needs 8-bit codes converted there; at
// these sizes the tensor rate does not bound.) The order of a head's values within S's sum is free,
// as is that of its values among O's rows, so both follow the 16-byte pieces.
//
// int8 and E4M3 codes are exact in fp16. q (bf16) goes to fp16 times a power of two for each head,
// exact down to 2^-24 of its head's largest value. A token's key scale multiplies its logit; its
// value scale its weight, which is rounded to fp16 (2^-11 relative, against the output's 2^-8).
// Over a bf16 cache the weights go as two bf16 (16 bits of them).
//
// Weights are taken relative to a running maximum that is only raised when a logit exceeds it by
// 2^6 (a vote, no shuffles in most tiles); with value scales, a second factor keeps the fp16 weights
// below 2^15; over a bf16 cache weights times 2^-24 do the same for the sums.
//
// Measured (of 6754.5 GB/s, the copy's): bf16 64 x 4000 tokens under 16 heads 306 us (101%), 32
// sequences of 500 to 4096 under 24 heads 139.6 (96%), E4M3 32 x 16000 under 32 heads over 8 167 (96%), 64 of
// 3 to 8192 99.8 (82%), int8 1 x 131072 under 64 over 8 54.4 (75%), 33 of 1 to 2000 21.9 (47%), one of 57
// 5.0. About 12 us are fixed: lengths, page table and first tiles one after another, the CTA's sums, the
// join. With 64 x 4000 under 128 heads over 8 (114.5 us, 70%) two warps a scheduler wait for their
// instructions' results; twelve warps an SM, 168 registers, change it by 2% either way.
#pragma once

#include "cache_kernels.cuh"
#include "int8_matmul_few_kernels.cuh"
#include "int8_matmul_kernels.cuh"

#include <cuda.h>

namespace fp8q {

// x / d for x * d < 2^64.
struct FastDiv {
  uint64_t magic;  // ceil(2^64 / d); 0 for d = 1
};
__device__ __forceinline__ int64_t fast_div(int64_t x, FastDiv d) {
  return d.magic ? int64_t(__umul64hi(uint64_t(x), d.magic)) : x;
}

struct AttnParams {
  const uint16_t* q;  // [batch, q_heads, D], row stride q_ld
  int64_t q_ld;
  CacheView cache;
  const int32_t* table;
  int64_t table_ld;
  const int32_t* lengths;
  uint16_t* out;  // [batch, q_heads, D]
  float* lse;     // [batch, q_heads] or null
  // Pieces of segments: their outputs (AttnLayout::kPiece values; divided by their sums, so that
  // they are no larger than the values they come from) and for each head the maximum
  // (log2 units) and the sum; a slot for each warp's first piece, then two for each CTA.
  float* part_o;
  float2* part_ml;
  int batch, width, window;  // width: pages a sequence may have
  int q_heads, group, blocks;  // heads a key/value head; blocks of 8 NT of them
  int grid, ctas;       // CTAs that are resident at once; all: as many, or twice as many
  int segments, heads;  // heads: blocks of heads a sequence
  int warp_rounds;      // segments a warp, if each warp takes whole ones
  FastDiv by_warps, by_heads, by_blocks;  // by grid * warps, by heads, by blocks
  float scale_log2;
  uint32_t tile_magic;  // ceil(2^32 / (page_size / 16))
  int page_tiles;
};

// The maximum before any token: no logit lies below it but -infinity (an infinite maximum would make
// NaN of the difference with itself).
constexpr float kAttnNone = -3.402823466e38f;

// Warps of a CTA and CTAs an SM: sixteen warps where their registers (accumulators D / 4 NT, queries
// as many) leave room for that, else eight to twelve. (Two blocks of heads of 64: 12 warps 46.7 us, eight
// 56.5, at 32 x 8000 tokens of 64 over 4 heads; 39 since the copies are asked for from uniform registers.)
constexpr int attn_warps(int type, int d, int nt) {
  return (type == kCacheBf16 ? 2 : 1) * d >= 512 || (d == 64 && nt == 2) ? 4 : 8;
}
constexpr int attn_ctas(int type, int d, int nt) {
  return d == 64 && nt == 2 ? 3 : (type == kCacheBf16 ? 2 : 1) * d <= 128 && nt == 1 ? 2 : 1;
}

template <int TYPE, int D, int NT>
struct AttnLayout {
  static constexpr int E = TYPE == kCacheBf16 ? 2 : 1;
  static constexpr int kWarps = attn_warps(TYPE, D, NT), kCtas = attn_ctas(TYPE, D, NT);
  static constexpr int KP = D * E / 64;   // 16-byte pieces of a key row a lane (four lanes a row)
  static constexpr int VB = D * E >= 128 ? 16 : 8;  // bytes of a value piece (eight lanes a row)
  static constexpr int VP = D * E / (8 * VB);
  static constexpr int kLine = D * E >= 128 ? D * E : 128;  // bytes of a map's row: a token, or two
  static constexpr int kLines = 16 * D * E / kLine;         // of a tile
  static constexpr int kBoxes = kLine / 128;                // columns of 128 bytes, swizzled
  static constexpr int kHalf = 16 * D * E;                  // a tile's keys
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kScales = TYPE == kCacheBf16 ? 0 : 128;  // a stage's key and value scales
  static constexpr int MT = D / 16;
  static constexpr int kItems = NT * MT * 2;       // pairs of values a lane holds of a piece
  static constexpr int kPiece = kItems * 64;       // values of a piece: 8 NT heads
  static constexpr int kStats = kWarps * 2 * (8 * NT * 20 + 8);  // of the CTA's pieces
  static constexpr int kMost = 233472 / kCtas - 1024 - (233472 / kCtas) % 128;  // a CTA's share of an SM's
  static constexpr int kRoom = (kMost - kStats) / (kWarps * (kStage + kScales + 8));
  static constexpr int kStages = kRoom < 6 ? kRoom : 6;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kBytes = kWarps * (kRing + kStages * (kScales + 8)) + kStats;
  static_assert(kRing >= kPiece * 4, "a warp's ring holds its last piece");
};

// A sequence's tiles: [first, first + n), its tokens [lo, hi).
struct AttnSpan {
  int lo, hi, first, n;
};
// Where tiles are shared out, a segment counts as so many more: its queries, page lookups and
// accumulators cost a warp about that (33 sequences of 1 .. 2000 tokens, 8 heads: 22.2 us, 23.5 with 3).
constexpr int kAttnExtra = 8;
__device__ __forceinline__ int attn_weight(const AttnSpan& s) { return s.n ? s.n + kAttnExtra : 0; }

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

// The work's split, found by each warp from the lengths (the loops are kept rolled: code that runs
// once costs the time to fetch it). A segment is a sequence's tiles for one block of heads.

// Weighted tiles of a block of heads: over all sequences, those of this lane's sequences and those up
// to them; the longest's tiles.
struct AttnScan {
  int total, mine, incl, most;
};
__device__ __forceinline__ AttnScan attn_scan(const AttnParams& P) {
  const int lane = threadIdx.x & 31;
  const int per = (P.batch + 31) >> 5, b1 = min(lane * per + per, P.batch);
  AttnScan s = {0, 0, 0, 0};
#pragma unroll 1
  for (int b = lane * per; b < b1; ++b) {
    const AttnSpan x = attn_span(P, b);
    s.mine += attn_weight(x);
    s.most = max(s.most, x.n);
  }
  s.most = __reduce_max_sync(0xffffffffu, s.most);
  s.incl = s.mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, s.incl, o);
    if (lane >= o) s.incl += v;
  }
  s.total = __shfl_sync(0xffffffffu, s.incl, 31);
  return s;
}

// The sequence that holds the weighted tile `want` (below the total) of a block of heads, and those
// before it.
struct AttnPlace {
  int b, before;
};
__device__ __forceinline__ AttnPlace attn_find(const AttnParams& P, const AttnScan& s, int want) {
  const int owner = __ffs(__ballot_sync(0xffffffffu, want < s.incl)) - 1;
  AttnPlace r;
  r.before = __shfl_sync(0xffffffffu, s.incl - s.mine, owner);
  r.b = owner * ((P.batch + 31) >> 5);
#pragma unroll 1
  for (;; ++r.b) {  // (ends within the owner's sequences: their sum passes `want`)
    const int n = attn_weight(attn_span(P, r.b));
    if (want < r.before + n) return r;
    r.before += n;
  }
}

// How the tiles are shared out.
//   kByTile     each warp the same number of weighted tiles, of all in one order (sequence, block of
//               heads, tile): pieces of segments are joined by the CTA, and by the join kernel across CTAs
//   kBySegment  a CTA for each segment, its warps the same number of tiles
//   kByWarp     each warp whole segments
// Costs in tiles of a warp (about 0.5 us). Never by tile where no sequence has more tiles than a CTA
// has warps: the host launches no join then.
// SMs do not draw on the memory alike: with equal shares of long sequences the slowest quarter of them
// takes 15% longer than the rest. So the host launches twice the resident CTAs where there may be
// much work, and if there is (kMuchWork tiles a warp), the first half takes kFirstShare of it and the
// second, launched as the first ones end, the rest in small shares (64 x 4000 tokens, 16 heads of bf16:
// 310 us, 328 with equal shares; 32 x 16000, E4M3 168 and 178; shares of 0.86 and 0.94 171 and 176).
// Not with less, where the pieces cost more than the balance gives (20 sequences of 1000 to 8000, int8,
// 20 tiles a warp: 46.6 us, 43.3 with equal shares), nor for few segments, whose last would fall into
// hundreds of pieces (1 x 131072: 79 us, 55 with equal shares), nor for two blocks of 8-bit heads (no gain).
constexpr int kByTile = 0, kBySegment = 1, kByWarp = 2;
constexpr int kCostJoin = 8, kCostMerge = 2, kMuchWork = 40;
constexpr float kFirstShare = 0.9f;
struct AttnSplit {
  int mode, quota, rest;  // quota: by tile, of a warp of the first CTAs; rest: of the others
};
template <int W>
__device__ __forceinline__ AttnSplit attn_split(const AttnParams& P, const AttnScan& scan) {
  AttnSplit s;
  s.quota = max(int(fast_div(int64_t(scan.total) * P.heads + (P.grid * W - 1), P.by_warps)), 1);
  s.rest = 0;
  const int by_tile = scan.most <= W ? INT32_MAX : s.quota + kCostJoin;
  const int by_segment =
      P.segments <= P.grid ? (scan.most + W - 1) / W + kCostMerge : INT32_MAX;
  const int by_warp = (P.warp_rounds == 1 ? 0 : s.quota) + scan.most;
  s.mode = by_segment <= by_tile ? kBySegment : kByTile;
  if (by_warp < min(by_tile, by_segment)) s.mode = kByWarp;
  if (s.mode == kByTile && P.ctas > P.grid && s.quota >= kMuchWork) {
    const int first = __float2int_ru(__fmul_rn(float(s.quota), kFirstShare));
    s.rest = s.quota - first;  // (the quota was rounded up: together they reach the end)
    s.quota = first;
  }
  return s;
}

// By tile: a CTA's first weighted tile, and its warps' quota.
template <int W>
__host__ __device__ __forceinline__ int64_t attn_begin(const AttnParams& P, const AttnSplit& s, int cta) {
  const int over = max(cta - P.grid, 0);
  return (int64_t(cta - over) * s.quota + int64_t(over) * s.rest) * W;
}
// The CTA that has a weighted tile. (These two run on the host as well, where their sizes are tested.)
template <int W>
__host__ __device__ __forceinline__ int attn_cta(const AttnParams& P, const AttnSplit& s, int64_t t) {
  const int64_t border = int64_t(P.grid) * s.quota * W;
  // (a quota is below 2^31, a CTA's tiles are not below 2^32: only small numbers are divided in 32 bits)
  const int64_t size = int64_t(t < border ? s.quota : s.rest) * W, at = t < border ? t : t - border;
  const int n = (at | size) <= int64_t(UINT32_MAX) ? int(uint32_t(at) / uint32_t(size)) : int(at / size);
  return t < border ? n : n + P.grid;
}

// A segment: sequence, key/value head, block of that head's queries.
struct AttnSegment {
  int b, h, block;
};
__device__ __forceinline__ AttnSegment attn_segment(const AttnParams& P, int seg) {
  AttnSegment s;
  s.b = int(fast_div(seg, P.by_heads));
  const int rest = seg - s.b * P.heads;
  s.h = int(fast_div(rest, P.by_blocks));
  s.block = rest - s.h * P.blocks;
  return s;
}

// ------------------------------------------------------------------------------------------

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

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
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

// Values of a head in one row of the lanes: runs of `kRun` side by side, blocks j of O^T holding two
// each (in rows r and r + 8).
template <int TYPE, int D>
struct AttnValues {
  static constexpr int E = TYPE == kCacheBf16 ? 2 : 1;
  static constexpr int kRun = (D * E >= 128 ? 16 : 8) / E;
  // the first value of block j's two in row r of the lanes
  static __device__ __forceinline__ int of(int j, int r) {
    return ((j / (kRun / 2)) * 8 + r) * kRun + (j % (kRun / 2)) * 2;
  }
};

__device__ __forceinline__ float attn_lse(float top, float sum) {
  return sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

// 1 / sum, any finite number for a sum of 0. (No branch: loads are asked for ahead across it.)
__device__ __forceinline__ float attn_inverse(float sum) {
  return __fdividef(1.0f, fmaxf(sum, 0x1p-100f));
}

// Two values of a head's row of the output.
template <int TYPE, int D>
__device__ __forceinline__ void attn_store(const AttnParams& P, int64_t row, int block, int r, float2 o,
                                           float2 ml) {
  *reinterpret_cast<uint32_t*>(P.out + row * D + AttnValues<TYPE, D>::of(block, r)) = pack_bf16x2(o.x, o.y);
  if (P.lse && r == 0 && block == 0) P.lse[row] = attn_lse(ml.x, ml.y);
}

template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(AttnLayout<TYPE, D, NT>::kWarps * 32, AttnLayout<TYPE, D, NT>::kCtas)
    paged_attention_kernel(const __grid_constant__ AttnParams P,
                           const __grid_constant__ CUtensorMap map_k,
                           const __grid_constant__ CUtensorMap map_v) {
  using L = AttnLayout<TYPE, D, NT>;
  constexpr bool QUANT = TYPE != kCacheBf16;
  constexpr int W = L::kWarps, S = L::kStages, E = L::E, KP = L::KP, VP = L::VP, MT = L::MT;
  constexpr int KS = QUANT ? 4 : 2;  // matrix steps (16 values of a key row) a piece
  // A bf16 cache's weights (up to 2^6) go into the products times 2^-24, so that a warp's sums of 2^18
  // tokens' values up to bf16's largest stay within fp32 (8-bit caches have the factor kf for that); weights
  // below 2^-102 of the largest lose bits for it, below 2^-109 all.
  constexpr float kDown = 0x1p-24f;
  extern __shared__ __align__(1024) uint8_t attn_smem[];
  // (The warp's number from one lane: what follows from it, addresses and the walk over segments, then
  // stays in uniform registers, where the copies want it. With an elected lane asking for them, 64 x 4000
  // tokens of E4M3 under 128 heads over 8: 137 -> 119 us, 64 sequences of 3 to 8192 under 32: 106.5 ->
  // 103.7; registers 240 -> 217 with two blocks, 160 -> 130 over bf16.)
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  uint8_t* ring = attn_smem + warp * L::kRing;
  uint8_t* scales = attn_smem + W * L::kRing + warp * S * L::kScales;
  uint64_t* full = reinterpret_cast<uint64_t*>(attn_smem + W * (L::kRing + S * L::kScales)) + warp * S;
  float2* stats = reinterpret_cast<float2*>(attn_smem + W * (L::kRing + S * (L::kScales + 8)));  // [warp][first, last][head]
  float2* total = stats + 2 * W * 8 * NT;                            // of a piece's segment
  float* factor = reinterpret_cast<float*>(total + 2 * W * 8 * NT);  // of a piece in its segment
  int2* open = reinterpret_cast<int2*>(factor + 2 * W * 8 * NT);     // [warp][first, last]
  if (lane == 0) {
    if (warp == 0) {  // the copies' descriptions, ahead of their first use
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_v)) : "memory");
    }
    for (int i = 0; i < S; ++i) mbar_init(full + i, 1);
    fence_mbar_init();
  }
  __syncwarp();
  wait_for_producers();
  allow_dependents();  // (not before: the join reads the lengths while this kernel runs)

  const AttnScan scan = attn_scan(P);
  const AttnSplit split = attn_split<W>(P, scan);
  const bool by_warp = split.mode == kByWarp;
  const int unit = blockIdx.x * W + warp, units = P.grid * W;
  // the second half, where there is nothing for it
  if (int(blockIdx.x) >= P.grid &&
      (split.rest == 0 || attn_begin<W>(P, split, blockIdx.x) >= int64_t(scan.total) * P.heads))
    return;

  // This warp's share: from weighted tile `at0` of segment s0 on, `share` of them (by warp: segment
  // after segment). `extra` ones stand before a segment's tiles.
  const int extra = split.mode == kByTile ? kAttnExtra : 0;
  AttnSegment s0 = {0, 0, 0};
  int at0 = 0, share = 0;
  if (split.mode == kByTile) {
    const int quota = int(blockIdx.x) < P.grid ? split.quota : split.rest;
    const int64_t t0 = attn_begin<W>(P, split, blockIdx.x) + int64_t(quota) * warp;
    const int64_t all = int64_t(scan.total) * P.heads;
    if (t0 < all) {
      share = int(min(int64_t(quota), all - t0));
      const AttnPlace at = attn_find(P, scan, int(fast_div(t0, P.by_heads)));
      const uint32_t local = uint32_t(t0 - int64_t(at.before) * P.heads);
      const uint32_t n = attn_weight(attn_span(P, at.b)), hb = local / n;
      s0 = attn_segment(P, int(hb));
      s0.b = at.b;
      at0 = int(local - hb * n);
    }
  } else {
    const int seg = by_warp ? unit : blockIdx.x;
    if (seg < P.segments) {
      s0 = attn_segment(P, seg);
      share = INT32_MAX;
      if (!by_warp) {
        const int n = attn_span(P, s0.b).n, q = (n + W - 1) / W;
        at0 = min(q * warp, n);
        share = min(q, n - at0);
      }
    }
  }
  // The segment after s: false if there is none.
  auto next_segment = [&](AttnSegment& s) {
    if (by_warp) {
      const int seg = (s.b * P.heads + s.h * P.blocks + s.block);
      if (seg >= P.segments - units) return false;
      s = attn_segment(P, seg + units);
    } else if (++s.block == P.blocks) {
      s.block = 0;
      if (++s.h == P.cache.heads) s.h = 0, ++s.b;
    }
    return s.b < P.batch;
  };

  // ---- the fetching side: the next tile to copy
  AttnSegment fg = s0;
  AttnSpan f = {0, 0, 0, 0};
  int f_at = at0, f_left = share, f_pos = 0, f_end = 0, f_row = 0;  // f_row: tiles into the page
  // Pages of the piece from f_page0 on, one a lane, and the 32 after them: their loads are under way
  // long before they are needed.
  int f_page0 = 0, f_pages = 0, f_pages_next = 0;
  bool f_more = share > 0, f_new = true, f_fine = true;
  int f_page = 0, f_line = 0;  // the tile's first line in the page's map
  const float *f_ks = nullptr, *f_vs = nullptr;
  // The piece that begins at f_at, or the next that has a tile.
  auto f_settle = [&]() {
#pragma unroll 1
    for (; f_more; f_at = 0) {
      f = attn_span(P, fg.b);
      const int part = min((f.n ? f.n + extra : 0) - f_at, f_left);
      if (!by_warp) f_left -= part;
      f_pos = max(f_at - extra, 0);
      f_end = f_at + part - extra;
      if (f_pos < f_end) {
        const int32_t* table = P.table + fg.b * P.table_ld;
        const int last = attn_page(P, f.first + f_end - 1);
        f_page0 = attn_page(P, f.first + f_pos);
        f_row = f.first + f_pos - f_page0 * P.page_tiles;
        f_pages = table[min(f_page0 + lane, last)];
        if (f_page0 + 32 <= last) f_pages_next = table[min(f_page0 + 32 + lane, last)];
        f_new = true;
        break;
      }
      f_more = f_left > 0 && next_segment(fg);
    }
  };
  uint32_t bad = 0;  // which of the tiles under way have no page, the newest in bit 0
  int fs = 0;
  auto fetch = [&]() {
    bad <<= 1;
    if (f_more) {
      if (f_new) {
        const int nth = attn_page(P, f.first + f_pos);
        if (nth == f_page0 + 32) {
          f_page0 = nth;
          f_pages = f_pages_next;
          const int last = attn_page(P, f.first + f_end - 1);
          if (nth + 32 <= last)
            f_pages_next = P.table[fg.b * P.table_ld + min(nth + 32 + lane, last)];
        }
        f_page = __shfl_sync(0xffffffffu, f_pages, nth - f_page0);
        f_fine = f_page >= 0 && f_page < P.cache.pages;
        if (!f_fine && lane == 0) report_device_error(kDevErrBadIndex);
        f_new = false;
        const int row = fg.h * P.cache.page_size + f_row * 16;  // in the page
        f_line = row * (D * E) / L::kLine;
        if (QUANT) {
          f_ks = P.cache.k_scale + f_page * P.cache.ks_stride + row;
          f_vs = P.cache.v_scale + f_page * P.cache.vs_stride + row;
        }
      }
      bad |= f_fine ? 0 : 1;
      if (elect_lane()) {
        uint64_t* bar = full + fs;
        if (f_fine) {
          const uint32_t dst = smem_addr(ring) + fs * L::kStage;
          mbar_arrive_expect_tx(bar, L::kStage + L::kScales);
#pragma unroll
          for (int p = 0; p < L::kBoxes; ++p)
            tma_load_3d(dst + p * 2048, &map_k, p * 128, f_line, f_page, bar);
#pragma unroll
          for (int p = 0; p < L::kBoxes; ++p)
            tma_load_3d(dst + L::kHalf + p * 2048, &map_v, p * 128, f_line, f_page, bar);
          if (QUANT) {
            uint8_t* to = scales + fs * L::kScales;
            bulk_load(to, f_ks, 64, bar);
            bulk_load(to + 64, f_vs, 64, bar);
          }
        } else {
          mbar_arrive(bar);
        }
      }
      f_line += L::kLines;
      if (QUANT) f_ks += 16, f_vs += 16;
      f_new = ++f_row == P.page_tiles;
      if (f_new) f_row = 0;
      if (++f_pos == f_end) {
        f_more = f_left > 0 && next_segment(fg);
        f_at = 0;
        f_settle();
      }
    }
    fs = fs + 1 == S ? 0 : fs + 1;
  };
  f_settle();

  // ---- the computing side. Before the first tile the ring is filled.
  int warm = S - 1, left = share;
  // Where this lane's pieces lie in a tile: its key row's chunks c and c + 4 (of 16 bytes, of a column
  // of 128), its value rows' chunk r, under the swizzle (a chunk's number XOR its line's).
  constexpr bool PAIRED = D * E == 64;  // two tokens a line
  const int k_at = PAIRED ? (r >> 1) * 128 + ((((r & 1) * 4 + c) ^ (r >> 1)) << 4)
                          : r * 128 + ((c ^ r) << 4);
  const int v_at = PAIRED ? c * 128 + (((r >> 1) ^ c) << 4) + (r & 1) * 8
                          : 2 * c * 128 + ((r ^ (2 * c)) << 4);
  int cs = 0;
  uint32_t phase = 0;
  bool failed = false;
  int2 open_first = {-1, 0}, open_last = {-1, 0};  // pieces: segment, whether it starts (1), ends (2)
  AttnSegment sg = s0;
  bool more = share > 0;
  for (int at = at0; more; at = 0, more = !failed && left > 0 && next_segment(sg)) {
    const AttnSpan span = attn_span(P, sg.b);
    const int part = min((span.n ? span.n + extra : 0) - at, left);
    const int begin = max(at - extra, 0), end = at + part - extra;
    if (!by_warp) {
      left -= part;
      if (begin >= end) continue;
    }
    const int head0 = sg.h * P.group + sg.block * 8 * NT;       // first query head of the block
    const int live = min(8 * NT, P.group - sg.block * 8 * NT);  // query heads in it
    const int64_t row0 = int64_t(sg.b) * P.q_heads + head0;

    // q as the columns of S^T: the values that face this lane's part of a key row. (As they lie in
    // memory until the first tile; asked for before the ring's first tiles.)
    uint32_t qf[NT][KP * KS][2];
    float fac[NT][2];  // logits in log2 units, for the lane's two heads
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = j * 8 + r;
      const uint4* row =
          reinterpret_cast<const uint4*>(P.q + sg.b * P.q_ld + int64_t(head0 + n) * D) + c * (KS / 2);
#pragma unroll
      for (int i = 0; i < KP * KS / 2; ++i) {
        const uint4 x = n < live ? row[(i / (KS / 2)) * 4 * (KS / 2) + i % (KS / 2)]
                                 : make_uint4(0, 0, 0, 0);
        qf[j][2 * i][0] = x.x, qf[j][2 * i][1] = x.y;
        qf[j][2 * i + 1][0] = x.z, qf[j][2 * i + 1][1] = x.w;
      }
      fac[j][0] = fac[j][1] = P.scale_log2;
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

#pragma unroll 1
    for (int pos = begin - warm; pos < end; ++pos) {
      __syncwarp();  // (the stage that fetch() overwrites has been read by all lanes)
      fetch();
      if (pos < begin) continue;
      if (QUANT && pos == begin) {  // q to fp16
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < KP * KS; ++i)
            m = max_u16x2(m, max_u16x2(qf[j][i][0] & 0x7FFF7FFFu, qf[j][i][1] & 0x7FFF7FFFu));
          uint32_t e = max(m & 0xFFFFu, m >> 16) >> 7;  // exponent of the head's largest value
          e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
          e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
          e = min(max(e, 10u), 254u);
          const float up = __uint_as_float((254u - e + 8u) << 23);  // 2^(127 + 8 - e): below 2^9
#pragma unroll
          for (int i = 0; i < KP * KS; ++i)
#pragma unroll
            for (int w = 0; w < 2; ++w)
              qf[j][i][w] = pack_f16x2(bf_lo(qf[j][i][w]) * up, bf_hi(qf[j][i][w]) * up);
          const float down = P.scale_log2 * __uint_as_float((e - 8u) << 23);  // 2^(e - 8 - 127)
          fac[j][0] = __shfl_sync(0xffffffffu, down, 8 * c);
          fac[j][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
        }
      }
      if (!__all_sync(0xffffffffu, mbar_wait(full + cs, phase))) {  // (a defect: nothing more is asked for)
        if (lane == 0) report_device_error(kDevErrWaitTimeout);
        failed = true;
        break;
      }
      const uint8_t* st = ring + cs * L::kStage;
      const float* sc = reinterpret_cast<const float*>(scales + cs * L::kScales) + r;
      if (++cs == S) cs = 0, phase ^= 1;
      if ((bad >> (S - 1)) & 1) continue;

      // S^T
      float s[NT][2][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[j][0][x] = s[j][1][x] = 0.0f;
#pragma unroll
      for (int p = 0; p < KP; ++p) {
        // rows r and r + 8, in the column p / 2
        const int at = (p >> 1) * 2048 + (k_at ^ ((p & 1) * 64));
        const uint4 x4 = *reinterpret_cast<const uint4*>(st + at);
        const uint4 y4 = *reinterpret_cast<const uint4*>(st + (PAIRED ? 512 + (at ^ 64) : 1024 + at));
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
          // (the head's factor with the key's scale first: a far query's sum times its factor may leave
          // fp32 where the logit does not)
          t[j][x] = (s[j][0][x] + s[j][1][x]) * (QUANT ? fac[j][x & 1] * ks[x >> 1] : fac[j][x & 1]);
        }
      }
      if (edge) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int tok = tok0 + r + 8 * (x >> 1);
            if (tok < span.lo || tok >= span.hi) t[j][x] = -INFINITY, vs[x >> 1] = 0.0f;
          }
      }
      float p[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          p[j][x] = ex2(t[j][x] - m[j][x & 1]);
          w[j][x] = QUANT ? p[j][x] * kf[j][x & 1] * vs[x >> 1] : p[j][x] * kDown;
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
              // a power of two that takes the tile's largest weight to 2^8 .. 2^9 (from 2^108, for rows
              // of zeros, down to 2^-119 at the end of fp32), no larger than what keeps the sums so far
              // from growing
              const int e = min(max(int(__float_as_uint(wt) >> 23) & 255, 27), 254);
              float k1 = __uint_as_float(uint32_t(254 + 8 - e) << 23);
              k1 = fminf(k1, __fdividef(kf[j][x], f));
              // (the factors may be more than 2^128 apart where all before counts for nothing)
              gain = f == 0.0f ? 0.0f : __fdividef(k1, kf[j][x]) * f;
              kf[j][x] = k1;
              w[j][x] = p[j][x] * k1 * vs[0];
              w[j][x + 2] = p[j][x + 2] * k1 * vs[1];
            } else {
              w[j][x] = p[j][x] * kDown;
              w[j][x + 2] = p[j][x + 2] * kDown;
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
          // tokens 2c + (i & 1) + 8 (i / 2)
          if (PAIRED) {
            const uint2 y = *reinterpret_cast<const uint2*>(
                st + L::kHalf + (i >> 1) * 512 + (v_at ^ (((i ^ (i >> 1)) & 1) * 64)));
            x[i][0] = y.x, x[i][1] = y.y;
          } else {
            const uint4 y = *reinterpret_cast<const uint4*>(
                st + L::kHalf + pc * 2048 + (i >> 1) * 1024 + ((i & 1) ? (v_at ^ 16) + 128 : v_at));
            x[i][0] = y.x, x[i][1] = y.y, x[i][2] = y.z, x[i][3] = y.w;
          }
        }
        if (edge && TYPE != kCacheInt8) {  // (a weight of 0 does not hide a NaN)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = tok0 + 2 * c + (i & 1) + 8 * (i >> 1);
            if (tok < span.lo || tok >= span.hi) {
#pragma unroll
              for (int w4 = 0; w4 < L::VB / 4; ++w4) x[i][w4] = 0u;
            }
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

    warm = 0;
    if (failed) break;

    // ---- this warp's sums
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[j][x] += __shfl_xor_sync(0xffffffffu, l[j][x], d);
      }
    const bool whole = begin == 0 && end == span.n;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float f = __fdividef(1.0f, QUANT ? kf[j][x] : kDown);
        f = l[j][x] == 0.0f ? 0.0f : __fdividef(f, l[j][x]);
#pragma unroll
        for (int i = 0; i < MT; ++i) o[j][i][x] *= f, o[j][i][x + 2] *= f;
      }
    if (whole) {  // a whole segment
      using V = AttnValues<TYPE, D>;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int n = j * 8 + 2 * c + x;
          if (n >= live) continue;
          uint16_t* to = P.out + (row0 + n) * D + r * V::kRun;
#pragma unroll
          for (int i = 0; i < MT; i += 4) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = pack_bf16x2(o[j][i + q][x], o[j][i + q][x + 2]);
            *reinterpret_cast<uint4*>(to + V::of(i, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (P.lse && r == 0) P.lse[row0 + n] = attn_lse(m[j][x], l[j][x]);
        }
      continue;
    }
    // A piece: the warp's last one stays in its ring, an earlier one (there can be one, its first)
    // waits in the workspace.
    const bool last = left <= 0;
    float2* to = (last ? reinterpret_cast<float2*>(ring)
                       : reinterpret_cast<float2*>(P.part_o + int64_t(unit) * L::kPiece)) + lane;
    __syncwarp();  // (all lanes have read the ring)
    const int2 what = make_int2(sg.b * P.heads + sg.h * P.blocks + sg.block,
                                (begin == 0 ? 1 : 0) | (end == span.n ? 2 : 0));
    if (last) open_last = what; else open_first = what;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (r == 0)
          stats[(warp * 2 + last) * (8 * NT) + j * 8 + 2 * c + x] = make_float2(m[j][x], l[j][x]);
#pragma unroll
        for (int i = 0; i < MT; ++i)
          to[((j * MT + i) * 2 + x) * 32] = make_float2(o[j][i][x], o[j][i][x + 2]);
      }
  }
  if (failed) {  // the copies under way have landed before the shared memory can go
    for (int i = 0; i < S; ++i) mbar_wait(full + i, phase ^ (i < cs ? 1 : 0));
  }
  if (by_warp) return;

  // ---- the CTA's pieces: those of a segment follow each other (warp 0's first, its last, warp 1's
  // first, ...), only its last can be a warp's first
  if (lane == 0) open[2 * warp] = open_first, open[2 * warp + 1] = open_last;
  __syncthreads();
  // each lane a piece: which of them are of its segment
  static_assert(2 * W <= 32, "a lane for each piece");
  const int2 piece = lane < 2 * W ? open[lane] : make_int2(-1, 0);
  const unsigned alike = __match_any_sync(0xffffffffu, piece.x >= 0 ? piece.x : -1 - lane);
  // a thread for each piece and head: the segment's maximum and sum, the piece's share
#pragma unroll 1
  for (int e = threadIdx.x; e < 2 * W * 8 * NT; e += W * 32) {
    const int p = e / (8 * NT);
    const unsigned mask = __shfl_sync(0xffffffffu, alike, p);
    const float2* ml = stats + e % (8 * NT);
    float top = kAttnNone, sum = 0.0f;
#pragma unroll 4
    for (int q = 0; q < 2 * W; ++q)
      if ((mask >> q) & 1) top = fmaxf(top, ml[q * (8 * NT)].x);
#pragma unroll 4
    for (int q = 0; q < 2 * W; ++q)
      if ((mask >> q) & 1) sum += ex2(ml[q * (8 * NT)].x - top) * ml[q * (8 * NT)].y;
    factor[e] = ex2(stats[e].x - top) * stats[e].y * attn_inverse(sum);
    total[e] = make_float2(top, sum);
  }
  __syncthreads();
  unsigned leaders = __ballot_sync(0xffffffffu, piece.x >= 0 && (alike & ((1u << lane) - 1)) == 0);
#pragma unroll 1
  for (; leaders; leaders &= leaders - 1) {
    const int p0 = __ffs(leaders) - 1;
    const unsigned mask = __shfl_sync(0xffffffffu, alike, p0);
    const int p1 = 31 - __clz(mask);  // its last piece
    const AttnSegment s = attn_segment(P, __shfl_sync(0xffffffffu, piece.x, p0));
    const int starts = __shfl_sync(0xffffffffu, piece.y, p0) & 1;
    const bool whole = starts && (__shfl_sync(0xffffffffu, piece.y, p1) & 2);
    const int live = min(8 * NT, P.group - s.block * 8 * NT);
    const int slot = 2 * blockIdx.x + starts;  // where it goes on in other CTAs
#pragma unroll
    for (int i0 = 0; i0 < L::kItems / W; ++i0) {
      const int i = i0 * W + warp, n = (i / (2 * MT)) * 8 + 2 * c + (i & 1), at = i * 32 + lane;
      if (n >= live) continue;
      float2 acc = make_float2(0.0f, 0.0f);
      if ((p1 & 1) == 0) {  // a warp's first
        const float2 v = reinterpret_cast<const float2*>(
            P.part_o + (int64_t(blockIdx.x) * W + (p1 >> 1)) * L::kPiece)[at];
        const float f = factor[p1 * (8 * NT) + n];
        acc = make_float2(f * v.x, f * v.y);
      }
#pragma unroll 4
      for (int w = 0; w < W; ++w)
        if ((mask >> (2 * w + 1)) & 1) {
          const float2 v = reinterpret_cast<const float2*>(attn_smem + w * L::kRing)[at];
          const float f = factor[(2 * w + 1) * (8 * NT) + n];
          acc.x += f * v.x;
          acc.y += f * v.y;
        }
      const float2 ml = total[p0 * (8 * NT) + n];
      if (whole) {
        attn_store<TYPE, D>(P, int64_t(s.b) * P.q_heads + s.h * P.group + s.block * 8 * NT + n,
                            (i >> 1) % MT, r, acc, ml);
      } else {
        reinterpret_cast<float2*>(P.part_o + (int64_t(P.ctas) * W + slot) * L::kPiece)[at] = acc;
        if (r == 0 && ((i >> 1) % MT) == 0) P.part_ml[slot * (8 * NT) + n] = ml;
      }
    }
  }
  // sequences without tokens: no warp has them
#pragma unroll 1
  for (int64_t seg = unit; int(blockIdx.x) < P.grid && seg < P.segments; seg += units) {
    const AttnSegment s = attn_segment(P, int(seg));
    if (attn_span(P, s.b).n > 0) continue;
    const int64_t row = int64_t(s.b) * P.q_heads + s.h * P.group + s.block * 8 * NT;
    const int live = min(8 * NT, P.group - s.block * 8 * NT);
#pragma unroll 1
    for (int i = lane; i < live * (D / 2); i += 32) reinterpret_cast<uint32_t*>(P.out + row * D)[i] = 0u;
    if (P.lse && lane < live) P.lse[row + lane] = -INFINITY;
  }
}

// Joins the pieces of segments that several CTAs shared. A CTA for each segment, or, where there are
// more of them, for each CTA of the attention kernel and the segment that goes on behind it, and for
// four of a piece's pairs of values, times PARTS; a part's warps take the pieces in turn. Many CTAs take
// long to launch, few segments have many pieces: two parts where one would make more than kJoinMany CTAs
// an SM (64 sequences of 3 to 8192 tokens, 8 heads: 100.4 us, 103.0 with one part; 33 of 1 to 2000 21.9
// and 24.3; 32 of 24 heads in bf16 140.0 and 143.4), else one (1 x 131072, 64 heads over 8, int8, 55.0 us, 58.6 with
// two; 1 x 2000 9.3 and 10.6; 32 x 8000 of 64 over 4 heads of 64 37.9 and 39.2). A sum of pieces is never
// formed before it is divided, so that values up to fp32's largest stay finite.
constexpr int kJoinWarps = 8, kJoinItems = 4, kJoinMany = 5;

template <int TYPE, int D, int NT, int PARTS>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_join_kernel(const __grid_constant__ AttnParams P) {
  using L = AttnLayout<TYPE, D, NT>;
  __shared__ float2 sums[kJoinWarps][kJoinItems][32];
  __shared__ float2 stats[kJoinWarps][2][4];
  // Which pieces there are is found while the attention kernel runs: it began once the kernels before
  // it were complete, so the lengths are there.
  const AttnScan scan = attn_scan(P);
  const AttnSplit split = attn_split<L::kWarps>(P, scan);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  constexpr int W = L::kWarps;
  const bool by_segment = P.segments <= P.ctas;
  AttnSegment s = {0, 0, 0};
  int64_t first = 0;  // the segment's first weighted tile
  int count = 0;
  if (by_segment) {
    s = attn_segment(P, blockIdx.x);
    const int per = (P.batch + 31) >> 5, owner = int(uint32_t(s.b) / uint32_t(per));
    int before = __shfl_sync(0xffffffffu, scan.incl - scan.mine, owner);
#pragma unroll 1
    for (int i = owner * per; i < s.b; ++i) before += attn_weight(attn_span(P, i));
    count = attn_weight(attn_span(P, s.b));
    first = int64_t(before) * P.heads + int64_t(s.h * P.blocks + s.block) * count;
  } else {
    const int64_t t = attn_begin<W>(P, split, blockIdx.x + 1) - 1;  // the CTA's last tile
    if (t < int64_t(scan.total) * P.heads && (split.rest > 0 || int(blockIdx.x) < P.grid)) {
      const AttnPlace at = attn_find(P, scan, int(fast_div(t, P.by_heads)));
      count = attn_weight(attn_span(P, at.b));
      const uint32_t hb = uint32_t(t - int64_t(at.before) * P.heads) / uint32_t(count);
      s = attn_segment(P, int(hb));
      s.b = at.b;
      first = int64_t(at.before) * P.heads + int64_t(hb) * count;
    }
  }
  const bool some = split.mode == kByTile && count > 0;
  const int c0 = some ? attn_cta<W>(P, split, first + kAttnExtra) : 0;
  const int c1 = some ? attn_cta<W>(P, split, first + count - 1) : 0;
  // (a segment that began in an earlier CTA is joined there)
  const int pieces = some && (by_segment || c0 == int(blockIdx.x)) ? c1 - c0 + 1 : 0;
  wait_for_producers();
  allow_dependents();
  if (pieces < 2) return;
  const int live = min(8 * NT, P.group - s.block * 8 * NT);
  // Pieces whose loads a warp has under way together: two where segments are few and have many (1 x 2000
  // tokens: 9.3 us, 11.5 with one), one where the join's CTAs are many and wait for registers (256 x 300:
  // 33.1 us, 34.1 with two).
  constexpr int kJoinAhead = PARTS == 2 ? 1 : 2;
  constexpr int kTurns = kJoinWarps / PARTS;  // warps of a part
  const int item0 = (blockIdx.y * PARTS + warp % PARTS) * kJoinItems;
  float2 ml[2] = {{kAttnNone, 0.0f}, {kAttnNone, 0.0f}}, acc[kJoinItems];
#pragma unroll
  for (int i = 0; i < kJoinItems; ++i) acc[i] = make_float2(0.0f, 0.0f);
  // (the four items are of one block of eight heads, in turn its heads 2c and 2c + 1)
  const bool in[2] = {(item0 / (2 * L::MT)) * 8 + 2 * c < live, (item0 / (2 * L::MT)) * 8 + 2 * c + 1 < live};
#pragma unroll 1
  for (int p0 = warp / PARTS; p0 < pieces; p0 += kJoinAhead * kTurns) {
    float2 x[kJoinAhead][2], v[kJoinAhead][kJoinItems];
#pragma unroll
    for (int k = 0; k < kJoinAhead; ++k) {
      const int p = p0 + k * kTurns;
      const int slot = 2 * (c0 + p) + (p == 0 ? 1 : 0);  // the first piece is its CTA's last
      const float2* from = reinterpret_cast<const float2*>(
          P.part_o + (int64_t(P.ctas) * W + slot) * L::kPiece) + item0 * 32 + lane;
      const float2* stat = P.part_ml + slot * (8 * NT) + (item0 / (2 * L::MT)) * 8 + 2 * c;
#pragma unroll
      for (int i = 0; i < 2; ++i) x[k][i] = p < pieces && in[i] ? stat[i] : make_float2(kAttnNone, 0.0f);
#pragma unroll
      for (int i = 0; i < kJoinItems; ++i)
        v[k][i] = p < pieces && in[i & 1] ? from[i * 32] : make_float2(0.0f, 0.0f);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = ml[i].x;
#pragma unroll
      for (int k = 0; k < kJoinAhead; ++k) top = fmaxf(top, x[k][i].x);
      float old = ex2(ml[i].x - top) * ml[i].y, sum = old;
#pragma unroll
      for (int k = 0; k < kJoinAhead; ++k) x[k][i].y *= ex2(x[k][i].x - top), sum += x[k][i].y;
      ml[i] = make_float2(top, sum);
      const float inv = attn_inverse(sum);
      old *= inv;
#pragma unroll
      for (int j = i; j < kJoinItems; j += 2) acc[j].x *= old, acc[j].y *= old;
#pragma unroll
      for (int k = 0; k < kJoinAhead; ++k) {
        const float f = x[k][i].y * inv;
#pragma unroll
        for (int j = i; j < kJoinItems; j += 2) acc[j].x += f * v[k][j].x, acc[j].y += f * v[k][j].y;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kJoinItems; ++i) {
    sums[warp][i][lane] = acc[i];
    if (r == 0 && i < 2) stats[warp][i][c] = ml[i];
  }
  __syncthreads();
#pragma unroll
  for (int e = warp; e < PARTS * kJoinItems; e += kJoinWarps) {
    const int part = e / kJoinItems, i = e % kJoinItems;
    const int it = blockIdx.y * (PARTS * kJoinItems) + e, n = (it / (2 * L::MT)) * 8 + 2 * c + (it & 1);
    if (n >= live) continue;
    float top = kAttnNone, sum = 0.0f;
    float2 a = make_float2(0.0f, 0.0f);
    float share[kTurns];
#pragma unroll
    for (int k = 0; k < kTurns; ++k) top = fmaxf(top, stats[k * PARTS + part][i & 1][c].x);
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
      const float2 x = stats[k * PARTS + part][i & 1][c];
      share[k] = ex2(x.x - top) * x.y;
      sum += share[k];
    }
    const float inv = attn_inverse(sum);
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
      const float f = share[k] * inv;
      const float2 x = sums[k * PARTS + part][i][lane];
      a.x += f * x.x;
      a.y += f * x.y;
    }
    attn_store<TYPE, D>(P, int64_t(s.b) * P.q_heads + s.h * P.group + s.block * 8 * NT + n,
                        (it >> 1) % L::MT, r, a, make_float2(top, sum));
  }
}

}  // namespace fp8q
