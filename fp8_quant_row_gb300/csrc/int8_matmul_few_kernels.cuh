// int8_matmul_few_kernels.cuh -- the int8 product for few tokens (sm_103a): every weight is read
// once and used for at most 8 * NT tokens, so the weights' bytes bound it.
//
// A CTA of eight warps takes 16 output channels at a time; `split` of its warps share a channel
// group's k, interleaved by 128 values, so that together they read a kilobyte of each row at
// about one time (DRAM pages: at 36864 x 6144, 42.6 us against 48.8 with a contiguous range for
// each warp). Each lane copies its own 16-byte pieces of the weights (cp.async) through a ring in
// shared memory that it alone writes and reads, two groups of k ahead (4 KB a warp, 96 KB in
// flight on an SM of 24 warps), across channel groups, in the layout of the fp16 matrix instruction m16n8k16: 16 consecutive bytes of a channel per
// lane; which k a fragment's places stand for is free as long as both operands agree. It
// converts (exact) and multiplies; tokens are read and converted the same way and come from the
// L1 cache after the first use. (The integer instruction m16n8k32 runs at a quarter of the fp16
// rate: 258 against 1020 products a clock and SM; eight tokens at the memory's rate need 183.)
// The warps' sums are added through shared memory in a fixed order.
//
// Measured on one GB300 (graph replay over weights larger than the L2 cache): 1 x 6144 x 6144 9.6
// us, 1 x 6144 x 18432 22.0 us, 1 x 2048 x 2048 3.5 us: about 6 TB/s of weights after 3.5 us of
// launch, first loads and last sums. Issue slots are half used (ncu), so the memory bounds it.
#pragma once

#include "int8_matmul_kernels.cuh"

namespace fp8q {

constexpr int kFewWarps = 8;
constexpr int kFewStages = 3;                     // groups of 128 values of k in the ring
constexpr int kFewStageBytes = 4 * 512;           // per warp: 16 channels x 128 values
constexpr int kFewFlush = 1024 / 128;             // groups between drains: sums stay exact
constexpr int kFewRing = kFewWarps * kFewStages * kFewStageBytes;

template <int NT>
constexpr int few_smem_bytes() {
  return kFewRing + 2 * kFewWarps * NT * 4 * 32 * 4;  // the ring, two buffers of sums
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16 bytes to shared memory, zeros where `in` is false.
__device__ __forceinline__ void cp_async16_if(uint32_t dst, const int8_t* src, bool in) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}

// rounds: channel groups of 16 a team of `split` warps takes, one grid apart.
template <int NT, bool F32>
__global__ void __launch_bounds__(kFewWarps * 32, 3)
    int8_matmul_few_kernel(MmParams p, int split, int rounds) {
  extern __shared__ uint4 few_smem[];
  allow_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int teams = kFewWarps / split;
  const int64_t team = int64_t(blockIdx.x) * teams + warp / split;  // and so on, one grid apart
  const int64_t stride = int64_t(gridDim.x) * teams;
  const int k = int(p.k), per = ((k + 127) / 128 + split - 1) / split;  // groups of k a warp
  const int k0 = (warp % split) * 128 + t * 16, step = split * 128;
  const int8_t* a[NT];  // tokens past the last are read as the last, their results not stored
#pragma unroll
  for (int j = 0; j < NT; ++j) a[j] = p.a + min(int64_t(j * 8 + g), p.m - 1) * p.lda;
  const uint4* ring = few_smem + warp * (kFewStages * kFewStageBytes / 16) + lane;
  const uint32_t ring_addr = smem_addr(ring);
  float* part = reinterpret_cast<float*>(few_smem) + kFewRing / 4;
  wait_for_producers();

  // The next group to copy: two segments of 64 values, each two pieces of 16 bytes a lane.
  int64_t ft = team;
  int fr = 0, fi = 0, fs = 0;
  const int8_t *w0 = nullptr, *w1 = nullptr;
  auto fetch = [&]() {
    if (fr < rounds) {
      if (fi == 0) {
        w0 = p.w + min(ft * 16 + g, p.n - 1) * p.k;
        w1 = p.w + min(ft * 16 + g + 8, p.n - 1) * p.k;
      }
      const uint32_t dst = ring_addr + fs * kFewStageBytes;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int off = k0 + fi * step + h * 64;
        const bool in = off < k;
        cp_async16_if(dst + h * 1024, w0 + (in ? off : 0), in);
        cp_async16_if(dst + h * 1024 + 512, w1 + (in ? off : 0), in);
      }
      if (++fi == per) fi = 0, ++fr, ft += stride;
    }
    fs = (fs + 1) % kFewStages;
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kFewStages - 1; ++i) fetch();

  // This lane's tokens of group i, loaded one group ahead (past k the weights are zero; no
  // read-only loads: the kernel before may write the tokens while this one has begun).
  uint4 an[2][NT];
  auto tokens = [&](int i) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int off = k0 + i * step + h * 64;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        an[h][j] = *reinterpret_cast<const uint4*>(a[j] + (off < k ? off : 0));
    }
  };
  tokens(0);

  int cs = 0;
  for (int r = 0; r < rounds; ++r) {
    float sum[NT][4] = {};
    float acc[NT][4] = {};
    for (int i = 0; i < per; ++i) {
      uint4 av[2][NT];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < NT; ++j) av[h][j] = an[h][j];
      tokens(i + 1 < per ? i + 1 : 0);
      fetch();
      cp_async_wait<kFewStages - 1>();
      const uint4* stage = ring + cs * (kFewStageBytes / 16);
      cs = (cs + 1) % kFewStages;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 wx = stage[h * 64], wy = stage[h * 64 + 32];
        const uint32_t x[4] = {wx.x, wx.y, wx.z, wx.w}, y[4] = {wy.x, wy.y, wy.z, wy.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t f[4];
          int8_to_f16(x[q], f[0], f[2]);
          int8_to_f16(y[q], f[1], f[3]);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint4 v = av[h][j];
            uint32_t b0, b1;
            int8_to_f16(q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w, b0, b1);
            mma_f16(acc[j], f[0], f[1], f[2], f[3], b0, b1);
          }
        }
      }
      if ((i + 1) % kFewFlush == 0) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) sum[j][c] += acc[j][c], acc[j][c] = 0.0f;
      }
    }
    // two buffers in turn: one barrier between the writing and the reading of each is enough
    float* buf = part + (r & 1) * (kFewWarps * NT * 4 * 32);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        buf[(warp * NT * 4 + j * 4 + c) * 32 + lane] = sum[j][c] + acc[j][c];
    __syncthreads();
    // a team's values, one (register, lane) pair each, over its `split` warps
    const int64_t n0 = (team + r * stride) * 16;
    for (int e = (warp % split) * 32 + lane; e < NT * 4 * 32; e += split * 32) {
      float v = 0.0f;
      for (int s = 0; s < split; ++s) v += buf[(warp - warp % split + s) * NT * 4 * 32 + e];
      const int i = e >> 5, l = e & 31;
      const int64_t n = n0 + (l >> 2) + ((i & 2) ? 8 : 0);
      const int64_t m = (i >> 2) * 8 + (l & 3) * 2 + (i & 1);
      if (n < p.n && m < p.m)
        mm_store<F32>(static_cast<uint8_t*>(p.out) + (m * p.n + n) * (F32 ? 4 : 2),
                      mm_value(v, p.w_scale[n], p.a_scale[m],
                               p.bias ? __uint_as_float(uint32_t(p.bias[n]) << 16) : 0.0f));
    }
  }
  cp_async_wait<0>();
}

}  // namespace fp8q
