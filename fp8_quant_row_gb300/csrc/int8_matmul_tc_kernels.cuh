// int8_matmul_tc_kernels.cuh -- the int8 product on the 5th-generation tensor cores (sm_103a).
//
// sm_103a has no 8-bit integer tcgen05 kind (and its legacy integer matrix instruction runs at
// 258 products a clock and SM). An int8 is exactly an fp16, a product of two at most 2^14 and a
// sum of 1024 products at most 2^24: tcgen05.mma kind::f16 with fp32 accumulators adds them
// exactly. So the tiles are brought in as int8 (half the bytes), converted in the SM, multiplied
// as fp16, and every 1024 values of k the accumulators are drained into fp32 registers
// (exact while |sum| <= 2^24; beyond, one rounding for each drain).
//
// The weights' rows (output channels) are the matrix instruction's M side, tokens its N side:
// lane = channel, column = token. A tile is CG * 128 channels x BT tokens:
//
//   CG = 2   a pair of CTAs shares a tile; each brings and converts its own 128 channels and half
//            the tokens (half the operand traffic per product; for many tokens)
//   CG = 1   one CTA; a cluster of `split` CTAs shares the tile's k where there are fewer tiles
//            than SMs, and exchanges partial sums at the end (for few tokens, where bringing the
//            weights in is what counts)
//
//   warpgroup 0          warp 0: TMA, 128 bytes of k for 128 + BT / CG rows per stage, 128-byte
//                        swizzle; warp 1 (first CTA of a pair): issues the matrix instructions
//   warpgroups 1, 2      weights: int8 stage -> fp16 in tensor memory, thread = row; they take
//                        stages in turn
//   warpgroups 3, 4      tokens: int8 stage -> fp16 in shared memory (128-byte swizzled K-major),
//                        in turn
//   warpgroups 5, 6      drain the accumulators, scale, store
//
// Conversion of four int8: flip the sign bits (value + 128), place each byte under the fp16
// exponent of 1024 (1024 + 128 + value, exact), subtract 1152.
//
// Measured on one GB300 (four calls in a CUDA graph, median of five replays, below the power limit):
// 4608 x 36864 x 6144 1043 us, 2002 TFLOP/s (cuBLAS in bf16 at that shape, the same way: 1046);
// 4608 x 6144 x 18432 528 us, 1978 (cuBLAS 537). Called for seconds on end, at the power limit, 1150
// to 1180 and 580 to 600. For a CTA of a pair one stage is 1024 clocks of the tensor cores, and of
// shared memory too (32 KB each of copies in, reads for conversion, converted tokens, and reads by
// the tensor cores): weights go to tensor memory so that this is not more; about 1200 are reached.
// 16 x 36864 x 6144 40 us (85% of HBM), 64 x 6144 x 6144 15 us. What it took, at 4608 x 6144 x 18432
// (here and below both sides of a change are from one session; sessions differ by some percent):
// waits and arrivals without cluster-scope fences 993 -> 630 us; issue from uniform registers and two
// groups of converting warps for either operand 630 -> 560; the accumulators in two halves -> 537.
//
// Every wait is bounded; a wait that runs out records the device error bit, the role stops, and
// the CTA pair meets at the end, where tensor memory is freed and every arrival on its way has landed.
#pragma once

#include <cuda.h>

#include "int8_matmul_kernels.cuh"

namespace fp8q {

constexpr int kTcStep = 128;        // k values per stage
constexpr int kTcChunk = 1024;      // k values per drain
constexpr int kTcThreads = 896;
constexpr int kTcFirstDrain = 20;   // first of the draining warps
constexpr int kTcSmemLimit = 227 * 1024;

template <int CG, int BT>
struct TcLayout {
  // registers a thread: the roles' shares of what the launch gives (72 x 896 threads)
  static constexpr int kRegsIssue = 40, kRegsConvert = BT > 128 ? 40 : 64;
  static constexpr int kRegsDrain = BT > 128 ? 152 : 104;
  static_assert(kRegsIssue + 4 * kRegsConvert + 2 * kRegsDrain <= 7 * 72, "");
  static constexpr int kRowsB = BT / CG;
  // A pair's accumulators are two halves, of the tokens' first and second halves in each CTA, so
  // that one is drained while the other's products run (565 -> 537 us at 4608 x 6144 x 18432).
  // Of 128 tokens they stay whole: 24.5 against 25.6 us at 128 x 6144 x 6144.
  static constexpr int kHalves = BT == 256 ? 2 : 1;
  static constexpr int kRawA = 128 * kTcStep, kRawB = kRowsB * kTcStep, kRaw = kRawA + kRawB;
  static constexpr int kConvB = kRowsB * kTcStep * 2;
  // (four for a pair: 61.5 against 64.4 us at 1024 x 6144 x 6144 of 128 tokens)
  static constexpr int kConvStages = CG == 2 ? 4 : 3;
  static constexpr int kBarBytes = 320;
  static constexpr int kScaleBytes = 2 * BT * 4;  // the token scales of two tiles in turn
  static constexpr int kRawStages0 =
      (kTcSmemLimit - kBarBytes - kScaleBytes - kConvStages * kConvB) / kRaw;
  static constexpr int kRawStages = kRawStages0 > 8 ? 8 : kRawStages0;
  // "Copied in" barriers. The two groups of converting warps take stages in turn, and a wait tells
  // phases apart by parity alone: over an odd ring a group would see only every second phase of a
  // barrier, and pass on the one before when that copy is late. So their ring is even. (Converted
  // stages are freed in order: who waits for one has seen the one two before it freed, so no
  // phase of a ring of three or four goes unseen.)
  static constexpr int kFullBars = kRawStages % 2 ? 2 * kRawStages : kRawStages;
  static constexpr int kBytes = kRawStages * kRaw + kConvStages * kConvB + kBarBytes + kScaleBytes;
  static constexpr int kColsA = BT;  // first column of the converted weights
  static constexpr int kCols = kColsA + kConvStages * 64 <= 256 ? 256 : 512;
  // partial sums, sent and got, over the stages (free by then)
  static_assert(CG == 2 || (2 * BT + 8) * 512 <= kRawStages * kRaw + kConvStages * kConvB, "");
  static_assert(kBytes <= kTcSmemLimit && kRawStages >= 2 && kColsA + kConvStages * 64 <= 512, "");
  static_assert(8 * (kFullBars + kRawStages + 2 * kConvStages + 9) <= kBarBytes, "");
};

// ---- instructions -------------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Address of `addr` (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// `bytes` of this CTA's shared memory to another's, counted by that CTA's barrier.
__device__ __forceinline__ void bulk_send(uint32_t cluster_dst, uint32_t src, uint32_t bytes,
                                          uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, "
      "[%3];" ::"r"(cluster_dst),
      "r"(src), "r"(bytes), "r"(cluster_bar)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}
// Bounded wait that reports when it runs out. (Waits that acquire, and arrivals that release, at
// cluster scope cost 0.4 us a stage here, 993 against 630 us at 4608 x 6144 x 18432; what they
// would order, the other CTA's converted tile, its own proxy fence and the arrival already do.)
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitLimitCycles) {
      report_device_error(kDevErrWaitTimeout);
      return false;
    }
  return true;
}
// The same for a whole warp, whose lanes stay together (what follows are warp-wide instructions):
// every branch is on a vote.
__device__ __forceinline__ bool tc_wait_warp(uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
    if (__any_sync(0xffffffffu, clock64() - t0 > kWaitLimitCycles)) {
      report_device_error(kDevErrWaitTimeout);
      return false;
    }
  return true;
}
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
  if (CG == 2)
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(slot)),
                 "r"(cols)
                 : "memory");
  else
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(slot)),
                 "r"(cols)
                 : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  if (CG == 2) {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
  } else {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
  }
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// D (+)= A (tensor memory) * B (shared memory, descriptor hi:lo), 16 values of k.
template <int CG, bool ADD>
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, uint32_t add) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(ADD ? 1u : add)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(ADD ? 1u : add)
        : "memory");
}
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
// One arrival on `bar` (in both CTAs of a pair) once the matrix instructions so far are done.
template <int CG>
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  if (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_addr(bar)),
        "h"(uint16_t(3))
        : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// Eight columns; the wait is part of the statement, so nothing uses the values before it.
__device__ __forceinline__ void tmem_load8(uint32_t addr, float (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7])
      : "r"(addr)
      : "memory");
}

__device__ __forceinline__ void sts_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float lds_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- kernel -------------------------------------------------------------------------------

struct TcParams {
  MmParams mm;
  int64_t tiles, tiles_n, tiles_m;  // tiles_n: of CG * 128 channels, tiles_m: of BT tokens
  int steps;                        // ceil(k / kTcStep)
  int split, steps_per;             // CG = 1: CTAs that share a tile's k, stages of each
};

// Token tiles are taken in groups of up to 16, inside a group all channel tiles in order, tokens
// fastest: the tiles at work at one time share few rows of either operand.
__device__ __forceinline__ void tc_tile(const TcParams& p, int64_t t, int64_t& tn, int64_t& tm) {
  const int64_t per = 16 * p.tiles_n, g = t / per, in = t - g * per;
  const int64_t left = p.tiles_m - 16 * g, w = left < 16 ? left : 16;
  tn = in / w;
  tm = 16 * g + (in - tn * w);
}

template <int CG, int BT, bool F32>
__global__ void __launch_bounds__(kTcThreads, 1)
    int8_matmul_tc_kernel(const __grid_constant__ CUtensorMap map_w,
                          const __grid_constant__ CUtensorMap map_a, const TcParams p) {
  using L = TcLayout<CG, BT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* raw = smem;
  uint8_t* conv = smem + L::kRawStages * L::kRaw;
  uint64_t* bars = reinterpret_cast<uint64_t*>(conv + L::kConvStages * L::kConvB);
  uint64_t* raw_full = bars;
  uint64_t* raw_empty = raw_full + L::kFullBars;
  uint64_t* conv_full = raw_empty + L::kRawStages;   // first CTA's counts for the pair
  uint64_t* conv_empty = conv_full + L::kConvStages;
  uint64_t* d_full = conv_empty + L::kConvStages;    // one for each half
  uint64_t* d_empty = d_full + 2;                    // the same; first CTA's counts for the pair
  uint64_t* peers_ready = d_empty + 2;               // CG = 1: the others' stages are free
  uint64_t* sums_full = peers_ready + 1;             // CG = 1: the others' sums are here
  uint64_t* sums_laid = sums_full + 1;               // CG = 1: this CTA's sums are in its memory
  uint64_t* idle = sums_laid + 1;                    // all matrix instructions are done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(idle + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t half = CG == 2 ? rank : 0u;         // which 128 channels and tokens of the tile
  const int ctas = CG == 2 ? 2 : p.split;
  const int64_t first = blockIdx.x / unsigned(ctas), stride = gridDim.x / unsigned(ctas);
  const int s0 = CG == 2 ? 0 : int(rank) * p.steps_per;
  const int steps = CG == 2 ? p.steps : min(p.steps_per, p.steps - s0);

  allow_dependents();
  if (threadIdx.x == 64) {  // the copies' descriptions, ahead of their first use
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_w)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_a)) : "memory");
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kFullBars; ++i) mbar_init(&raw_full[i], 1);
    for (int i = 0; i < L::kRawStages; ++i) mbar_init(&raw_empty[i], 8);
    for (int i = 0; i < L::kConvStages; ++i) {
      mbar_init(&conv_full[i], 8 * CG);
      mbar_init(&conv_empty[i], 1);
    }
    for (int h = 0; h < L::kHalves; ++h) {
      mbar_init(&d_full[h], 1);
      mbar_init(&d_empty[h], 8 * CG / L::kHalves);
    }
    mbar_init(peers_ready, CG == 1 && ctas > 1 ? ctas - 1 : 1);
    mbar_init(sums_full, 1);
    mbar_init(sums_laid, 8);
    mbar_init(idle, 1);
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 1) tmem_alloc<CG>(tmem_slot, L::kCols);
  tc_fence_before();
  if (ctas > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  wait_for_producers();

  if (warp < 4) {
    reg_dec<L::kRegsIssue>();
    if (warp == 0 && lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int64_t t = first; t < p.tiles && ok; t += stride) {
        int64_t tn, tm;
        tc_tile(p, t, tn, tm);
        const int yw = int(tn * (128 * CG) + half * 128), ya = int(tm * BT + half * L::kRowsB);
        for (int s = 0; s < steps; ++s, ++it) {
          const uint32_t st = it % L::kRawStages, use = it / L::kRawStages;
          ok = tc_wait(&raw_empty[st], (use & 1) ^ 1);
          if (!ok) break;
          uint8_t* dst = raw + st * L::kRaw;
          uint64_t* full = &raw_full[it % L::kFullBars];
          mbar_arrive_expect_tx(full, L::kRaw);
          tma_load_2d(dst, &map_w, (s0 + s) * kTcStep, yw, full);
          tma_load_2d(dst + L::kRawA, &map_a, (s0 + s) * kTcStep, ya, full);
        }
      }
      // copies still in flight land before the CTA ends
      for (uint32_t i = it > L::kRawStages ? it - L::kRawStages : 0; i < it; ++i)
        tc_wait(&raw_full[i % L::kFullBars], (i / L::kFullBars) & 1);
    } else if (warp == 1 && half == 0) {
      // The whole warp goes through the loop and one lane issues: values that the warp shares
      // stay in uniform registers, where the instructions want them.
      // fp32 accumulators, fp16 operands, K-major, N = BT or half of it, M = CG * 128
      constexpr uint32_t idesc = (1u << 4) | (uint32_t(BT / L::kHalves / 8) << 17) | (uint32_t(CG * 8) << 24);
      // 128-byte swizzle, 1024 bytes between groups of eight rows
      constexpr uint32_t desc_hi = (2u << 29) | (1u << 14) | 64u;
      const uint32_t desc_lo = (1u << 16) | ((smem_addr(conv) & 0x3FFFFu) >> 4);
      const uint32_t d = __shfl_sync(0xffffffffu, tmem, 0);
      const bool leader = elect_lane();
      uint32_t st = 0, use = 0, chunk = 0;
      bool ok = true;
      // One half's products of a stage.
      auto issue = [&](int h, uint32_t stage, bool add) {
        tc_fence_after();
        const uint32_t dh = d + h * (BT / 2), a = d + L::kColsA + stage * 64;
        const uint32_t b = desc_lo + stage * (L::kConvB >> 4) + h * (L::kRowsB / 2 * 8);
        if (leader) {
          tc_mma<CG, false>(dh, a, b, desc_hi, idesc, add);
#pragma unroll
          for (int j = 1; j < kTcStep / 16; ++j)
            tc_mma<CG, true>(dh, a + j * 8, b + (j / 4) * (L::kRowsB * 8) + (j % 4) * 2, desc_hi,
                             idesc, 1);
        }
      };
      constexpr int kPer = kTcChunk / kTcStep;  // stages between drains
      for (int64_t t = first; t < p.tiles && ok; t += stride) {
        for (int s = 0; s < steps;) {
          // With two halves the first two and the last two stages between drains are taken
          // together, first half first: a half is drained during two stages of the other (537 ->
          // 516 us at 4608 x 6144 x 18432, with the fourth converted stage that it needs).
          const int in = s % kPer;
          const bool both = L::kHalves == 2 && (in == 0 || in == kPer - 2) && s + 1 < steps;
          const int n = both ? 2 : 1;
          const bool fresh = in == 0, last = in + n == kPer || s + n == steps;
          const bool wrap = st + 1 == L::kConvStages;
          const uint32_t next = wrap ? 0 : st + 1, next_use = wrap ? use ^ 1 : use;
          ok = tc_wait_warp(&conv_full[st], use);
          if (ok && fresh) ok = tc_wait_warp(&d_empty[0], (chunk & 1) ^ 1);
          if (!ok) break;
          issue(0, st, !fresh);
          if (both) {
            ok = tc_wait_warp(&conv_full[next], next_use);
            if (!ok) break;
            issue(0, next, true);
          }
          if (leader && last) tc_commit<CG>(&d_full[0]);
          if (L::kHalves == 2) {
            if (fresh) ok = tc_wait_warp(&d_empty[1], (chunk & 1) ^ 1);
            if (!ok) break;
            issue(1, st, !fresh);
          }
          if (leader) tc_commit<CG>(&conv_empty[st]);
          st = next, use = next_use;
          if (both) {
            issue(1, st, true);
            if (leader) tc_commit<CG>(&conv_empty[st]);
            if (++st == L::kConvStages) st = 0, use ^= 1;
          }
          if (L::kHalves == 2 && leader && last) tc_commit<CG>(&d_full[1]);
          if (last) ++chunk;
          s += n;
        }
      }
      // matrix instructions still in flight are done before tensor memory is freed
      if (leader) tc_commit<CG>(idle);
      __syncwarp();
      tc_wait_warp(idle, 0);
    }
  } else if (warp < kTcFirstDrain) {
    reg_dec<L::kRegsConvert>();
    bool ok = true;
    const bool weights = warp < 12;
    const uint32_t turn = (warp >> 2) - (weights ? 1 : 3);  // takes the stages of this parity
    const int tid = (warp & 3) * 32 + lane;
    const uint32_t full0 = map_rank(smem_addr(conv_full), rank - half);
    constexpr int kParts = L::kRowsB / 16;  // 16-byte chunks of a token's stage a thread converts
    const int row = weights ? tid : tid % L::kRowsB;
    const int part = weights ? 0 : tid / L::kRowsB * kParts;  // its first chunk
    const uint32_t chunks = weights ? 8 : kParts;
    // its next stage of either ring, its next "copied in" barrier, and the phases that it waits for
    uint32_t rs = turn, cs = turn, full = turn, raw_phase = 0, conv_phase = 1;
    int s = int(turn);
    for (int64_t t = first; t < p.tiles && ok; t += stride) {
      for (; s < steps; s += 2) {
        ok = tc_wait_warp(&raw_full[full], raw_phase);
        if (!ok) break;
        const uint8_t* src = raw + rs * L::kRaw + (weights ? 0 : L::kRawA) + row * 128;
        uint8_t* dst = conv + cs * L::kConvB + row * 128;
        const uint32_t dst_a = tmem + L::kColsA + cs * 64 + (uint32_t(warp & 3) << 21);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // half of this thread's share into registers, so that its loads overlap
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (h * 4 + i < chunks)
              v[i] = *reinterpret_cast<const uint4*>(src + (((part + h * 4 + i) ^ (row & 7)) << 4));
          if (h == 0) {
            ok = tc_wait_warp(&conv_empty[cs], conv_phase);
            if (!ok) break;
            tc_fence_after();
          } else {
            __syncwarp();
            if (lane == 0) mbar_arrive(&raw_empty[rs]);
          }
          __syncwarp();  // the stores to tensor memory below are warp-wide
          if (weights) {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              uint32_t f[16];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                int8_to_f16(v[i + j].x, f[j * 8 + 0], f[j * 8 + 1]);
                int8_to_f16(v[i + j].y, f[j * 8 + 2], f[j * 8 + 3]);
                int8_to_f16(v[i + j].z, f[j * 8 + 4], f[j * 8 + 5]);
                int8_to_f16(v[i + j].w, f[j * 8 + 6], f[j * 8 + 7]);
              }
              tmem_store16(dst_a + h * 32 + i * 8, f);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (h * 4 + i >= kParts) continue;
              const int c = part + h * 4 + i;
              uint4 a, b;
              int8_to_f16(v[i].x, a.x, a.y);
              int8_to_f16(v[i].y, a.z, a.w);
              int8_to_f16(v[i].z, b.x, b.y);
              int8_to_f16(v[i].w, b.z, b.w);
              uint8_t* at = dst + (c >> 2) * (L::kRowsB * 128);
              *reinterpret_cast<uint4*>(at + ((((c & 3) * 2) ^ (row & 7)) << 4)) = a;
              *reinterpret_cast<uint4*>(at + ((((c & 3) * 2 + 1) ^ (row & 7)) << 4)) = b;
            }
          }
        }
        if (!ok) break;
        if (weights) {
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          tc_fence_before();
        } else {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncwarp();
        if (lane == 0) {
          if (CG == 2) mbar_arrive_cluster(full0 + cs * 8);
          else mbar_arrive(&conv_full[cs]);
        }
        rs += 2;
        if (rs >= L::kRawStages) rs -= L::kRawStages;
        full += 2;
        if (full >= L::kFullBars) full -= L::kFullBars, raw_phase ^= 1;
        cs += 2;
        if (cs >= L::kConvStages) cs -= L::kConvStages, conv_phase ^= 1;
      }
      s -= steps;
    }
  } else {
    reg_inc<L::kRegsDrain>();
    constexpr int kAcc = BT / 2;  // token columns of this warp
    const int side = (warp - kTcFirstDrain) >> 2, quarter = warp & 3;
    const uint32_t src = tmem + side * kAcc + (uint32_t(quarter) << 21);
    const uint32_t empty0 = map_rank(smem_addr(&d_empty[side % L::kHalves]), rank - half);
    uint32_t chunk = 0;
    bool ok = true;
    float* scales = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) + L::kBarBytes);
    bool parity = false;
    for (int64_t t = first; t < p.tiles && ok; t += stride) {
      int64_t tn, tm;
      tc_tile(p, t, tn, tm);
      const int64_t n = tn * (128 * CG) + half * 128 + quarter * 32 + lane;
      // the tokens of this warp's columns: two runs of half of them
      const int64_t m0 = tm * BT + side * (L::kHalves == 2 ? kAcc / 2 : kAcc);
      constexpr int kRun = L::kHalves == 2 ? kAcc : kAcc / 2;  // from the first run to the second
      // the scales while the products run
      constexpr int kMine = (kAcc + 31) / 32;
      float as[kMine];
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int c = i * 32 + lane;
        const int64_t m = m0 + c % (kAcc / 2) + (c >= kAcc / 2 ? kRun : 0);
        as[i] = c < kAcc && m < p.mm.m ? p.mm.a_scale[m] : 0.0f;
      }
      float ws = 0.0f, bias = 0.0f;
      if (n < p.mm.n) {
        ws = p.mm.w_scale[n];
        if (p.mm.bias) bias = __uint_as_float(uint32_t(p.mm.bias[n]) << 16);
      }
      float acc[kAcc];
#pragma unroll
      for (int i = 0; i < kAcc; ++i) acc[i] = 0.0f;
      for (int s = 0; s < steps; s += kTcChunk / kTcStep, ++chunk) {
        ok = tc_wait_warp(&d_full[side % L::kHalves], chunk & 1);
        if (!ok) break;
        tc_fence_after();
        // the last products are in: this CTA's stages are free, which the other CTAs of the
        // tile wait to hear
        if (CG == 1 && ctas > 1 && warp == kTcFirstDrain && s + kTcChunk / kTcStep >= steps &&
            lane < ctas && lane != int(rank))
          mbar_arrive_cluster(map_rank(smem_addr(peers_ready), lane));
        __syncwarp();  // the loads from tensor memory below are warp-wide
        if (s == 0) {
          // The four warps of a side store the same values. Their buffer is free: this tile's
          // first products were issued after every warp had drained the tile before, which is
          // after it had finished with the one before that.
#pragma unroll
          for (int i = 0; i < kMine; ++i)
            if (i * 32 + lane < kAcc) scales[side * kAcc + i * 32 + lane] = as[i];
          __syncwarp();
        }
#pragma unroll
        for (int c = 0; c < kAcc / 8; ++c) {
          float v[8];
          tmem_load8(src + c * 8, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[c * 8 + i] += v[i];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2) mbar_arrive_cluster(empty0);
          else mbar_arrive(&d_empty[0]);
        }
      }
      if (!ok) break;
      uint8_t* const o0 = static_cast<uint8_t*>(p.mm.out) + (m0 * p.mm.n + n) * (F32 ? 4 : 2);
      const int64_t step = p.mm.n * (F32 ? 4 : 2);
      if (CG == 1 && ctas > 1) {
        // The cluster has one tile. Each CTA finishes `per` of its columns. It lays its sums out
        // as [column][channel] over its stages (free once all its products are in, as the last
        // drain says), sends each other CTA that one's columns (in one bulk copy, once that one
        // says that its stages are free) and gets its own columns as [CTA][column][channel].
        // (Loops that stay loops: this code runs once, and its instructions come from memory;
        // unrolled over the columns it took 26 us at 128 tokens.)
        const int cols = min(BT, int(p.mm.m - tm * BT)), per = (cols + ctas - 1) / ctas;
        const int own0 = min(int(rank) * per, cols), own1 = min(own0 + per, cols);
        const uint32_t send = smem_addr(raw), get = send + BT * 512;
        const uint32_t at = (quarter * 32 + lane) * 4;
        if (warp == kTcFirstDrain && lane == 0)
          mbar_arrive_expect_tx(sums_full, uint32_t((ctas - 1) * (own1 - own0) * 512));
#pragma unroll
        for (int c = 0; c < kAcc; ++c) sts_f32(send + (side * kAcc + c) * 512 + at, acc[c]);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(sums_laid);
        ok = tc_wait_warp(sums_laid, 0);
        if (warp == kTcFirstDrain) {
          ok = tc_wait_warp(peers_ready, 0) && ok;
          const int to0 = min(lane * per, cols), to1 = min(to0 + per, cols);
          if (ok && lane < ctas && lane != int(rank) && to1 > to0)
            bulk_send(map_rank(get + uint32_t(int(rank) * per * 512), lane), send + to0 * 512,
                      uint32_t((to1 - to0) * 512), map_rank(smem_addr(sums_full), lane));
        }
        ok = tc_wait_warp(sums_full, 0) && ok;
        if (!ok) break;
        asm volatile("fence.acq_rel.cluster;" ::: "memory");
        if (n < p.mm.n) {
          uint8_t* o = o0 + (own0 + side - side * kAcc) * step;
#pragma unroll 1
          for (int col = own0 + side; col < own1; col += 8) {  // four columns at a time
            float v[4] = {};
#pragma unroll 1
            for (int r = 0; r < ctas; ++r) {  // in the order of k
              const uint32_t from = (r == int(rank) ? send + uint32_t(col * 512)
                                                    : get + uint32_t((r * per + col - own0) * 512)) + at;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (col + 2 * i < own1) v[i] += lds_f32(from + i * 1024);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i, o += 2 * step)
              if (col + 2 * i < own1) mm_store<F32>(o, mm_value(v[i], ws, scales[col + 2 * i], bias));
          }
        }
      } else if (n < p.mm.n) {
#pragma unroll
        for (int run = 0; run < 2; ++run) {
          uint8_t* o = o0 + run * kRun * step;
          const int64_t left = p.mm.m - m0 - run * kRun;
          const int cols = left < kAcc / 2 ? int(left) : kAcc / 2;
#pragma unroll
          for (int c = 0; c < kAcc / 2; c += 4) {
            const float4 sc = lds128(
                reinterpret_cast<const float4*>(scales + side * kAcc + run * (kAcc / 2) + c));
#pragma unroll
            for (int i = 0; i < 4; ++i, o += step)
              if (c + i < cols)
                mm_store<F32>(o, mm_value(acc[run * (kAcc / 2) + c + i], ws,
                                          i == 0 ? sc.x : i == 1 ? sc.y : i == 2 ? sc.z : sc.w,
                                          bias));
          }
        }
      }
      scales = parity ? scales - BT : scales + BT;
      parity = !parity;
    }
    if (warp == kTcFirstDrain) {
      // The commits' arrivals, which the first CTA of a pair sends to both, land in either before
      // its shared memory goes to another CTA: the last of each converted stage, and `idle` (those
      // on d_full the draining warps have seen). Here, since only after the last drain are they
      // at most a few stages away, whatever the product's length: the waits are bounded.
      bool landed = tc_wait_warp(idle, 0) && ok;
      const uint32_t uses = uint32_t((p.tiles - first + stride - 1) / stride) * uint32_t(steps);
      for (uint32_t i = uses > L::kConvStages ? uses - L::kConvStages : 0; i < uses && landed; ++i)
        landed = tc_wait_warp(&conv_empty[i % L::kConvStages], (i / L::kConvStages) & 1);
    }
  }
  __syncwarp();
  tc_fence_before();
  if (ctas > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_free<CG>(tmem, L::kCols);
}

}  // namespace fp8q
