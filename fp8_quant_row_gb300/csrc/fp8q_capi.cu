// fp8q_capi.cu -- host side of libfp8q: argument validation, device checks, launch shapes.
//
// Every entry point validates synchronously and returns a status before anything is
// enqueued; it then launches exactly one kernel on the caller's stream. Nothing here
// allocates device memory or synchronises, so the calls can be captured in CUDA graphs
// once the per-device launch caches below are warm (first call on a device queries
// attributes).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>

#include <cuda_runtime.h>

#include "fp8q.h"
#include "elementwise_kernels.cuh"
#include "int8_matmul_few_kernels.cuh"
#include "int8_matmul_kernels.cuh"
#include "int8_matmul_tc_kernels.cuh"
#include "nss_kernels.cuh"
#include "nss_ws_kernels.cuh"
#include "nvfp4_kernels.cuh"
#include "qkv_kernels.cuh"
#include "row_quant_kernels.cuh"

namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxLnCols = 32768;
constexpr int64_t kMaxEwCols = int64_t(1) << 30;
constexpr int64_t kMaxSiluCols = int64_t(1) << 20;
constexpr int64_t kMaxMmK = 131056;  // |sum| < 2^31

thread_local int g_last_cuda_error = 0;
thread_local char g_last_detail[160] = "";

struct DeviceInfo {
  int major = 0, minor = 0, sms = 0, smem_optin = 0;
  bool ok = false;
};

DeviceInfo g_dev[kMaxDevices];
std::once_flag g_dev_once[kMaxDevices];

// Records which runtime call failed (thread-local) and returns FP8Q_ERR_CUDA.
fp8q_status cuda_fail(cudaError_t e, const char* site, long long arg = -1) {
  g_last_cuda_error = int(e);
  std::snprintf(g_last_detail, sizeof g_last_detail, "%s(%lld): %s", site, arg,
                cudaGetErrorName(e));
  return FP8Q_ERR_CUDA;
}

// Current device, checked to be compute capability 10.3.
fp8q_status current_device(const DeviceInfo** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return FP8Q_ERR_UNSUPPORTED;
  std::call_once(g_dev_once[dev], [dev] {
    DeviceInfo& d = g_dev[dev];
    d.ok = cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor, dev) == cudaSuccess &&
           cudaDeviceGetAttribute(&d.minor, cudaDevAttrComputeCapabilityMinor, dev) == cudaSuccess &&
           cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
           cudaDeviceGetAttribute(&d.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) ==
               cudaSuccess;
  });
  const DeviceInfo& d = g_dev[dev];
  if (!d.ok) return cuda_fail(cudaErrorInvalidDevice, "cudaDeviceGetAttribute", dev);
  if (d.major != 10 || d.minor != 3) return FP8Q_ERR_UNSUPPORTED;
  *out = &d;
  return FP8Q_OK;
}

// Resident CTAs per SM of a kernel at a block size and a dynamic shared-memory size, cached per
// device. (The row kernels are launched with several block sizes, and wide rows with a
// shared-memory size for each width: a table of 2048 sets of eight, in which the next entry of a
// full set is replaced, so that what a process calls stays known however many widths it has seen.
// With 1200 entries spread evenly, some set has nine with a probability of 3e-5.)
struct OccEntry {
  int dev, threads;
  const void* fn;
  size_t smem;
  int blocks;
};
constexpr int kOccSets = 2048, kOccWays = 8;
struct OccSet {
  OccEntry entry[kOccWays];  // fn null where free
  int next;
};
OccSet g_occ[kOccSets];

OccSet& occ_set(int dev, const void* fn, int threads, size_t smem) {
  uint64_t h = uint64_t(reinterpret_cast<uintptr_t>(fn));
  for (uint64_t v : {uint64_t(smem), uint64_t(threads), uint64_t(dev)})
    h = (h ^ (h >> 29) ^ v) * 0x9E3779B97F4A7C15u;  // odd, 2^64 / golden ratio
  return g_occ[(h >> 40) % kOccSets];
}

// Dynamic shared-memory limit set on each (device, function): the limit is a property of the
// function, not of a launch, so it only ever grows to the largest size launched (a launch
// above the current limit is rejected; a smaller size seen later must not lower it).
struct SmemLimit {
  const void* fn;
  size_t limit;
};
constexpr int kMaxLimits = 256;  // more than the library has kernels
struct SmemLimits {
  SmemLimit entry[kMaxLimits];
  int n;
};
SmemLimits g_lim[kMaxDevices];
std::mutex g_occ_mu;

fp8q_status raise_smem_limit(int dev, const void* fn, size_t smem) {
  SmemLimits& lim = g_lim[dev];
  SmemLimit* entry = nullptr;
  for (int i = 0; i < lim.n; ++i)
    if (lim.entry[i].fn == fn) entry = &lim.entry[i];
  if (entry && entry->limit >= smem) return FP8Q_OK;
  if (!entry && lim.n == kMaxLimits) return FP8Q_ERR_UNSUPPORTED;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(MaxDynamicSharedMemorySize)", (long long)smem);
  if (!entry) entry = &lim.entry[lim.n++];
  *entry = SmemLimit{fn, smem};
  return FP8Q_OK;
}

fp8q_status blocks_per_sm(const void* fn, int threads, size_t smem, int* blocks) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return FP8Q_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_occ_mu);
  // Checked on every call: the cached occupancy below says nothing about the current limit.
  if (smem > 48 * 1024) {
    const fp8q_status st = raise_smem_limit(dev, fn, smem);
    if (st != FP8Q_OK) return st;
  }
  OccSet& set = occ_set(dev, fn, threads, smem);
  for (const OccEntry& o : set.entry)
    if (o.fn == fn && o.dev == dev && o.threads == threads && o.smem == smem) {
      *blocks = o.blocks;
      return FP8Q_OK;
    }
  int b = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, fn, threads, smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveBlocksPerMultiprocessor", (long long)smem);
  set.entry[set.next] = OccEntry{dev, threads, fn, smem, b};
  set.next = (set.next + 1) % kOccWays;
  *blocks = b;
  return FP8Q_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// Bytes spanned by `tokens` rows of `width` BF16 values at a stride of `ld` values.
size_t strided_bytes(int64_t tokens, int64_t ld, int64_t width) {
  return tokens > 0 ? size_t((tokens - 1) * ld + width) * 2 : 0;
}

struct Range {
  const void* p;
  size_t bytes;
};

bool overlap(Range a, Range b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

bool same(Range a, Range b) { return a.p == b.p && a.bytes == b.bytes; }

// One launch; the status is this launch's own (cudaLaunchKernelEx's return value), so an
// unrelated pending error of another library on the same thread is never reported as ours.
// Launches allow programmatic dependent launch: a kernel may be scheduled while the previous
// kernel in the stream drains, and every kernel executes griddepcontrol.wait before its first
// global-memory access, so producer -> consumer ordering is unchanged.
template <typename... Args>
fp8q_status launch(void (*fn)(Args...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                   Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, args...);
  if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernelEx", (long long)smem);
  return FP8Q_OK;
}

// ------------------------------------------------------------------------------------------
// LayerNorm family
// ------------------------------------------------------------------------------------------

template <int V, int WPR, bool RESID, bool HAS_BIAS>
fp8q_status launch_tuned(const fp8q::NssParams& p, const DeviceInfo& dev, int64_t n_mod,
                         cudaStream_t stream, bool* launched) {
  using L = fp8q::TunedLayout<V, WPR, RESID>;
  auto* fn = fp8q::nss_tuned_kernel<V, WPR, RESID, HAS_BIAS>;
  *launched = false;
  // As many warps per CTA (one CTA per SM) as the shared-memory ring allows, up to 24 where
  // the kernel is built for it; below 16 rows per SM at most 16 (width 3072, two warps per
  // row, 16 -> 24 warps: 2048 rows 10.41 -> 10.70 us, 3072 rows 13.25 -> 13.06 us, 4608 rows
  // 16.85 -> 16.59 us).
  int nw = fp8q::tuned_threads<V, WPR, RESID>() / 32;
  if (p.rows < 16 * int64_t(dev.sms) && nw > fp8q::kTunedMaxThreads / 32)
    nw = fp8q::kTunedMaxThreads / 32;
  while (nw >= WPR && L::smem_bytes(nw) > size_t(dev.smem_optin)) nw -= WPR;
  nw -= nw % WPR;
  if (nw < WPR) return FP8Q_OK;
  if (fp8q::kMaxTableUnitsPerThread * nw * 32 < WPR * V * 32) return FP8Q_OK;
  const size_t smem = L::smem_bytes(nw);
  int bps = 0;
  fp8q_status st = blocks_per_sm(reinterpret_cast<const void*>(fn), nw * 32, smem, &bps);
  if (st != FP8Q_OK) return st;
  if (bps <= 0) return FP8Q_OK;
  const int rows_per_iter = nw / WPR;
  int64_t need = (p.rows + rows_per_iter - 1) / rows_per_iter;
  // Fewer rows than a full wave: spread them over all SMs rather than filling a few CTAs, so
  // each SM's rows finish sooner (a warp or a warp pair computes a whole row).
  if (need < dev.sms) need = p.rows < dev.sms ? p.rows : dev.sms;
  const int64_t cap = int64_t(dev.sms) * bps;
  int64_t grid = need > n_mod ? need : n_mod;
  if (grid > cap) grid = cap;
  // Every CTA must sit inside one modulation group (single-row table).
  if (n_mod > grid) return FP8Q_OK;
  *launched = true;
  return launch(fn, dim3(unsigned(grid)), dim3(nw * 32), smem, stream, p, n_mod);
}

// Warp-specialised kernel: one CTA per SM (never more CTAs than rows), each owning a block
// of rows that it streams through a ring of WsLayout::kStages row stages.
constexpr int kWsDepth = 1 << 30;  // rows in flight per CTA (no limit beyond the ring)

template <int C, int NS, int NO>
fp8q_status launch_ws(const fp8q::NssParams& p, const DeviceInfo& dev, int64_t n_mod,
                      cudaStream_t stream, bool* launched) {
  using L = fp8q::WsLayout<C, NS, NO>;
  auto* fn = fp8q::nss_ws_kernel<C, NS, NO>;
  *launched = false;
  int64_t grid = std::min<int64_t>(dev.sms, p.rows);
  if (n_mod > grid) return FP8Q_OK;  // every CTA must sit inside one modulation group
  if (L::kSmemBytes > size_t(dev.smem_optin)) return FP8Q_OK;
  int bps = 0;
  fp8q_status st = blocks_per_sm(reinterpret_cast<const void*>(fn), L::kThreads, L::kSmemBytes, &bps);
  if (st != FP8Q_OK) return st;
  if (bps <= 0) return FP8Q_OK;
  *launched = true;
  return launch(fn, dim3(unsigned(grid)), dim3(L::kThreads), L::kSmemBytes, stream, p, n_mod,
                kWsDepth);
}

template <bool RESID, bool HAS_BIAS>
fp8q_status launch_generic(const fp8q::NssParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  auto* fn = fp8q::nss_generic_kernel<RESID, HAS_BIAS>;
  const size_t smem = size_t(p.cols) * 2;
  int bps = 0;
  fp8q_status st = blocks_per_sm(reinterpret_cast<const void*>(fn), fp8q::kNssThreads, smem, &bps);
  if (st != FP8Q_OK) return st;
  if (bps <= 0) return cuda_fail(cudaErrorInvalidConfiguration, "occupancy", (long long)smem);
  int64_t grid = int64_t(dev.sms) * bps;
  if (grid > p.rows) grid = p.rows;
  return launch(fn, dim3(unsigned(grid)), dim3(fp8q::kNssThreads), smem, stream, p);
}

template <bool RESID, bool HAS_BIAS>
fp8q_status dispatch_ln(const fp8q::NssParams& p, const DeviceInfo& dev, int64_t n_mod,
                        cudaStream_t stream) {
  bool launched = false;
  fp8q_status st = FP8Q_OK;
  // Up to two rows per SM the CTA-per-row kernel (eight warps share a row) has the lower
  // latency (width 3072, against the tuned kernel with two warps per row: 4.19 vs 4.58 us at
  // 153 rows, 4.53 vs 4.83 at 256; above, 4.91 vs 5.25 at 400, 5.26 vs 6.12 at 512).
  // At width 3072 two warps share a row up to 48 rows per SM: each warp's chain of per-row
  // work is half as long, which pays while a warp has few rows (width 3072, one vs two warps
  // per row: 1024 rows 9.02 -> 7.44 us, 4608 rows 16.97 -> 16.74 us, 6144 rows 21.16 ->
  // 20.54 us, but 9216 rows 27.47 -> 28.14 us). The residual variant always uses two: its
  // ring stages hold two rows' worth of input (x and residual), and half rows per warp let
  // twice as many warps fit in shared memory.
  if (p.rows <= 2 * int64_t(dev.sms)) return launch_generic<RESID, HAS_BIAS>(p, dev, stream);
  if (!RESID && p.cols == 3072) {
    st = launch_ws<3072, 7, 3>(p, dev, n_mod, stream, &launched);
    if (st != FP8Q_OK || launched) return st;
  }
  if (p.cols == 3072 && (RESID || p.rows <= 48 * int64_t(dev.sms)))
    st = launch_tuned<6, 2, RESID, HAS_BIAS>(p, dev, n_mod, stream, &launched);
  else if (p.cols == 3072)
    st = launch_tuned<12, 1, RESID, HAS_BIAS>(p, dev, n_mod, stream, &launched);
  else if (p.cols == 6144)
    st = launch_tuned<12, 2, RESID, HAS_BIAS>(p, dev, n_mod, stream, &launched);
  if (st != FP8Q_OK || launched) return st;
  return launch_generic<RESID, HAS_BIAS>(p, dev, stream);
}

fp8q_status check_ln_shape(int64_t rows, int64_t cols, int64_t mod_rows, float eps) {
  if (rows < 0 || mod_rows < 0) return FP8Q_ERR_SHAPE;
  if (cols < 8 || cols > kMaxLnCols || cols % 8 != 0) return FP8Q_ERR_SHAPE;
  if (!std::isfinite(eps) || eps < 0.0f) return FP8Q_ERR_VALUE;
  return FP8Q_OK;
}

int64_t mod_count(int64_t rows, int64_t mod_rows) {
  return mod_rows > 0 ? (rows + mod_rows - 1) / mod_rows : 1;
}

// ------------------------------------------------------------------------------------------
// 8-bit rows with a scale each, and their product
// ------------------------------------------------------------------------------------------

// Threads of a row whose chunks of eight values are held in registers, up to `most` a thread. With
// no more than two rows an SM a row gets a thread for each chunk, for its latency.
struct RowShape {
  int per_row, cpt, threads;
  bool many;
};

RowShape row_shape(int64_t rows, int chunks, int most, int sms) {
  RowShape s;
  s.many = rows > 2 * sms;
  s.per_row = 32;
  const int limit = s.many ? 256 : 1024, want = s.many ? most : 1;
  while (s.per_row < limit && s.per_row * want < chunks) s.per_row *= 2;
  s.cpt = (chunks + s.per_row - 1) / s.per_row;
  s.threads = s.per_row > 32 ? s.per_row : 128;
  return s;
}

// As many CTAs as are resident at once, each going from row to row; one row a CTA where not `many`.
template <typename Params>
fp8q_status launch_rows(void (*fn)(Params, int), const Params& p, const RowShape& s,
                        const DeviceInfo& dev, cudaStream_t stream) {
  int64_t ctas = (p.rows + s.threads / s.per_row - 1) / (s.threads / s.per_row);
  if (s.many) {
    int bps = 0;
    const fp8q_status st = blocks_per_sm(reinterpret_cast<const void*>(fn), s.threads, 0, &bps);
    if (st != FP8Q_OK) return st;
    ctas = std::min(ctas, int64_t(dev.sms) * std::max(bps, 1));
  }
  return launch(fn, dim3(unsigned(ctas)), dim3(s.threads), 0, stream, p, s.per_row);
}

// Threads of a row in shared memory. An SM wants over a thousand threads, and several rows, at
// work: 256 threads a row where five rows and more fit (10240 columns, 4608 rows: 37.2 us against
// 39.0 with 512), 512 where two to four do (18432 columns: 65.0 against 67.6 with 256), 1024 for
// one.
int wide_threads(size_t smem, const DeviceInfo& dev) {
  const size_t fit = size_t(dev.smem_optin) / (smem + 1024);
  return fit >= 5 ? 256 : fit >= 2 ? 512 : 1024;
}

template <typename Params>
fp8q_status launch_wide(void (*fn)(Params), int threads, size_t smem, const Params& p,
                        const DeviceInfo& dev, cudaStream_t stream) {
  int bps = 0;
  const fp8q_status st = blocks_per_sm(reinterpret_cast<const void*>(fn), threads, smem, &bps);
  if (st != FP8Q_OK) return st;
  const int64_t ctas = std::min<int64_t>(p.rows, int64_t(dev.sms) * std::max(bps, 1));
  return launch(fn, dim3(unsigned(ctas)), dim3(threads), smem, stream, p);
}

template <bool INT8, bool RESID, int CPT>
fp8q_status launch_rms_rows(const fp8q::RmsParams& p, const RowShape& s, const DeviceInfo& dev,
                            cudaStream_t stream) {
  return s.many ? launch_rows(fp8q::rms_norm_quant_kernel<INT8, RESID, CPT, true>, p, s, dev, stream)
                : launch_rows(fp8q::rms_norm_quant_kernel<INT8, RESID, CPT, false>, p, s, dev, stream);
}

template <bool INT8, bool RESID>
fp8q_status launch_rms(const fp8q::RmsParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  const RowShape s = row_shape(p.rows, p.cols / 8, 4, dev.sms);
  switch (s.cpt) {
    case 1: return launch_rms_rows<INT8, RESID, 1>(p, s, dev, stream);
    case 2: return launch_rms_rows<INT8, RESID, 2>(p, s, dev, stream);
    case 3: return launch_rms_rows<INT8, RESID, 3>(p, s, dev, stream);
    case 4: return launch_rms_rows<INT8, RESID, 4>(p, s, dev, stream);
    default: break;
  }
  const size_t smem = size_t(p.cols) * 4 + fp8q::kRqRedBytes;
  switch (wide_threads(smem, dev)) {
    case 256:
      return launch_wide(fp8q::rms_norm_quant_wide_kernel<INT8, RESID, 256>, 256, smem, p, dev, stream);
    case 512:
      return launch_wide(fp8q::rms_norm_quant_wide_kernel<INT8, RESID, 512>, 512, smem, p, dev, stream);
    default:
      return launch_wide(fp8q::rms_norm_quant_wide_kernel<INT8, RESID, 1024>, 1024, smem, p, dev, stream);
  }
}

template <bool INT8, int CPT>
fp8q_status launch_silu_rows(const fp8q::SiluParams& p, const RowShape& s, const DeviceInfo& dev,
                             cudaStream_t stream) {
  return s.many ? launch_rows(fp8q::silu_mul_quant_kernel<INT8, CPT, true>, p, s, dev, stream)
                : launch_rows(fp8q::silu_mul_quant_kernel<INT8, CPT, false>, p, s, dev, stream);
}

template <bool INT8>
fp8q_status launch_silu(const fp8q::SiluParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  // Four chunks a thread leave room for two CTAs an SM: with many rows shared memory is faster from
  // there (8192 columns, 4608 rows: 30.8 us against 32.1).
  const RowShape s = row_shape(p.rows, p.cols / 8, 3, dev.sms);
  switch (s.cpt) {
    case 1: return launch_silu_rows<INT8, 1>(p, s, dev, stream);
    case 2: return launch_silu_rows<INT8, 2>(p, s, dev, stream);
    case 3: return launch_silu_rows<INT8, 3>(p, s, dev, stream);
    case 4:
      if (s.many) break;
      return launch_rows(fp8q::silu_mul_quant_kernel<INT8, 4, false>, p, s, dev, stream);
    default: break;
  }
  const size_t smem = size_t(p.cols) * 4 + fp8q::kRqRedBytes;
  if (smem > size_t(dev.smem_optin))
    return launch_wide(fp8q::silu_mul_quant_wide_kernel<INT8, false, 512>, 512,
                       fp8q::kRqRedBytes, p, dev, stream);
  switch (wide_threads(smem, dev)) {
    case 256:
      return launch_wide(fp8q::silu_mul_quant_wide_kernel<INT8, true, 256>, 256, smem, p, dev, stream);
    case 512:
      return launch_wide(fp8q::silu_mul_quant_wide_kernel<INT8, true, 512>, 512, smem, p, dev, stream);
    default:
      return launch_wide(fp8q::silu_mul_quant_wide_kernel<INT8, true, 1024>, 1024, smem, p, dev, stream);
  }
}

// The driver's tensor-map encoder, through the runtime (the library links no libcuda).
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

fp8q_status encode_tiled(EncodeTiled* fn) {
  static std::once_flag once;
  static void* entry = nullptr;
  static cudaError_t err = cudaSuccess;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult found;
    err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &entry, 12000,
                                           cudaEnableDefault, &found);
    if (err == cudaSuccess && found != cudaDriverEntryPointSuccess) err = cudaErrorSymbolNotFound;
  });
  if (err != cudaSuccess) return cuda_fail(err, "cudaGetDriverEntryPointByVersion");
  *fn = reinterpret_cast<EncodeTiled>(entry);
  return FP8Q_OK;
}

// Tensor map of int8 rows [rows, k] at stride ld: boxes of 128 values of k x `box` rows, 128-byte
// swizzle; values past k and rows past `rows` read as zero.
fp8q_status int8_map(CUtensorMap* map, const int8_t* p, int64_t rows, int64_t k, int64_t ld,
                     int box) {
  EncodeTiled fn = nullptr;
  const fp8q_status st = encode_tiled(&fn);
  if (st != FP8Q_OK) return st;
  const cuuint64_t dims[2] = {cuuint64_t(k), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(ld)};
  const cuuint32_t boxes[2] = {cuuint32_t(fp8q::kTcStep), cuuint32_t(box)};
  const cuuint32_t steps[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p), dims,
                        strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return cuda_fail(cudaErrorInvalidValue, "cuTensorMapEncodeTiled", r);
  return FP8Q_OK;
}

// Clusters of 2 to 8 CTAs that are resident at one time with one CTA an SM, asked once per device.
// (A cluster stays within one GPC, so larger ones do not fill all SMs: 46 of three CTAs, 36 of
// four, 15 of eight.)
struct ClusterFit {
  std::once_flag once;
  int fit[9] = {};
  fp8q_status status = FP8Q_OK;
};
ClusterFit g_cluster[kMaxDevices];

fp8q_status cluster_fit(const int** fit) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return FP8Q_ERR_UNSUPPORTED;
  ClusterFit& c = g_cluster[dev];
  std::call_once(c.once, [&c] {
    using L = fp8q::TcLayout<1, 128>;
    auto* fn = fp8q::int8_matmul_tc_kernel<1, 128, false>;
    int bps = 0;
    c.status = blocks_per_sm(reinterpret_cast<const void*>(fn), fp8q::kTcThreads, L::kBytes, &bps);
    for (int size = 2; size <= 8 && c.status == FP8Q_OK; ++size) {
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = unsigned(size);
      attr.val.clusterDim.y = 1;
      attr.val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(unsigned(size));
      cfg.blockDim = dim3(fp8q::kTcThreads);
      cfg.dynamicSmemBytes = L::kBytes;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      const cudaError_t err = cudaOccupancyMaxActiveClusters(&c.fit[size], fn, &cfg);
      if (err != cudaSuccess) c.status = cuda_fail(err, "cudaOccupancyMaxActiveClusters", size);
    }
  });
  *fit = c.fit;
  return c.status;
}

// Tiles of a CG x BT kernel for this product and an estimate of its time in us: rounds of tiles
// times a tile's stages, plus a launch's fixed part (fitted to 13 token counts at six weight
// shapes; the choice is within 10% of the best measured at nearly all of them).
constexpr double kTcFixed = 4.0, kTcExchange = 0.8, kTcColumn = 0.02;  // sums' exchange

template <int CG, int BT>
constexpr double tc_stage_us() {
  return CG == 2 ? (BT == 256 ? 0.617 : 0.375) : BT == 128 ? 0.44 : BT == 64 ? 0.37 : 0.35;
}

template <int CG, int BT>
fp8q::TcParams plan_tc(const fp8q::MmParams& mm, const DeviceInfo& dev, const int* fit,
                       double* cost) {
  fp8q::TcParams p;
  p.mm = mm;
  p.tiles_n = (mm.n + 128 * CG - 1) / (128 * CG);
  p.tiles_m = (mm.m + BT - 1) / BT;
  p.tiles = p.tiles_n * p.tiles_m;
  p.steps = int((mm.k + fp8q::kTcStep - 1) / fp8q::kTcStep);
  p.split = 1;
  p.steps_per = p.steps;
  // Fewer tiles than SMs: CTAs of a cluster share a tile's k, each with two stages at least, as
  // many as leave all clusters resident at once.
  if (CG == 1) {
    int s = int(std::min<int64_t>({8, dev.sms / p.tiles, p.steps / 2}));
    while (s > 1 && fit[s] < p.tiles) --s;
    if (s > 1) {
      p.steps_per = (p.steps + s - 1) / s;
      p.split = (p.steps + p.steps_per - 1) / p.steps_per;
    }
  }
  const int64_t slots = dev.sms / CG;
  const double rounds = p.split > 1 ? 1.0 : double((p.tiles + slots - 1) / slots);
  *cost = rounds * p.steps_per * tc_stage_us<CG, BT>() + kTcFixed +
          (p.split > 1 ? kTcExchange + kTcColumn * double(std::min<int64_t>(mm.m, BT)) : 0.0);
  return p;
}

template <int CG, int BT, bool F32>
fp8q_status launch_tc(const fp8q::MmParams& mm, const DeviceInfo& dev, cudaStream_t stream) {
  using L = fp8q::TcLayout<CG, BT>;
  auto* fn = fp8q::int8_matmul_tc_kernel<CG, BT, F32>;
  const int* fit = nullptr;
  fp8q_status st = cluster_fit(&fit);
  if (st != FP8Q_OK) return st;
  double cost = 0.0;
  const fp8q::TcParams p = plan_tc<CG, BT>(mm, dev, fit, &cost);
  int bps = 0;
  st = blocks_per_sm(reinterpret_cast<const void*>(fn), fp8q::kTcThreads, L::kBytes, &bps);
  if (st != FP8Q_OK) return st;
  const int ctas = CG == 2 ? 2 : p.split;
  CUtensorMap map_w, map_a;
  st = int8_map(&map_w, mm.w, mm.n, mm.k, mm.k, 128);
  if (st != FP8Q_OK) return st;
  st = int8_map(&map_a, mm.a, mm.m, mm.k, mm.lda, L::kRowsB);
  if (st != FP8Q_OK) return st;
  const int64_t grid = ctas * std::min<int64_t>(p.tiles, dev.sms / ctas);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(fp8q::kTcThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, map_w, map_a, p);
  if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernelEx", (long long)L::kBytes);
  return FP8Q_OK;
}

template <int NT, bool F32>
fp8q_status launch_few(const fp8q::MmParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  const int64_t groups = (p.n + 15) / 16;  // of 16 channels
  auto* fn = fp8q::int8_matmul_few_kernel<NT, F32>;
  const size_t smem = fp8q::few_smem_bytes<NT>();
  int bps = 0;
  fp8q_status st =
      blocks_per_sm(reinterpret_cast<const void*>(fn), fp8q::kFewWarps * 32, smem, &bps);
  if (st != FP8Q_OK) return st;
  int split = fp8q::kFewWarps;  // warps that share a group's k, each with 128 values at least
  while (split > 1 && p.k < split * 128) split /= 2;
  // no more CTAs than are resident at once, each with the same number of groups (one more or less
  // by the last): they draw on the memory evenly and end together
  const int64_t per_cta = fp8q::kFewWarps / split;
  const int64_t slots = dev.sms * std::max(bps, 1) * per_cta, rounds = (groups + slots - 1) / slots;
  const int64_t grid = (groups + rounds * per_cta - 1) / (rounds * per_cta);
  return launch(fn, dim3(unsigned(grid)), dim3(fp8q::kFewWarps * 32), smem, stream, p, split,
                int(rounds));
}

template <int CG, int BT>
void consider_tc(const fp8q::MmParams& mm, const DeviceInfo& dev, const int* fit, double* best,
                 int* which) {
  double cost = 0.0;
  plan_tc<CG, BT>(mm, dev, fit, &cost);
  if (cost < *best) *best = cost, *which = CG * 1000 + BT;
}

// The kernel with the least estimated time. Measured (us; 8 and 16: the kernel for few tokens,
// CGxBT: the tensor-memory kernel), at 6144 x 6144 weights:
//   tokens      8     16   1x32   1x64  1x128  2x128  2x256
//        8    9.5   11.9   12.9   13.8   17.4   21.8   33.2
//       16          12.1   13.0   14.0   17.4   21.9   33.2
//       32                 13.3   14.2   16.2   21.9   33.5
//       64                 18.8   14.8   17.1   22.2   33.7
//      128                 34.4   21.6   18.3   22.1   34.0
//      256                 49.6   39.0   25.6   22.8   34.1
//      450                 80.4   56.6   46.9   40.7   35.1
//     1024                171.9  108.3   67.8   58.3   63.2
//     4608                709.5  407.2  258.7  221.4  183.4
// at 36864 x 6144, 8 tokens: 42.2 / 55.2 / 39.5 / 45.6 / 65.1 / 42.7 / 64.5, 128 tokens: 1x128 51.0,
// 2x128 44.5, 2x256 66.0; at 2048 x 2048, 8 tokens: 3.6 / 4.4 / 6.1, 200 tokens: 1x64 8.9, 2x128 10.6.
template <bool F32>
fp8q_status launch_int8_matmul(const fp8q::MmParams& p, const DeviceInfo& dev,
                               cudaStream_t stream) {
  double best = 1e30;
  int which = 0;
  // bytes at the rate that many channel groups reach, and how unevenly few groups fall on the SMs
  const int64_t groups = (p.n + 15) / 16, per_sm = (groups + dev.sms - 1) / dev.sms;
  const double uneven = per_sm <= 2 ? double(per_sm * dev.sms) / double(groups) : 1.0;
  const double weights = double(p.n) * double(p.k) * std::min(uneven, 2.0);
  if (p.m <= 8) best = 3.0 + weights / 5.9e6, which = 8;
  else if (p.m <= 16) best = 3.0 + weights / 4.2e6, which = 16;
  const int* fit = nullptr;
  const fp8q_status st = cluster_fit(&fit);
  if (st != FP8Q_OK) return st;
  if (p.m <= 512) consider_tc<1, 32>(p, dev, fit, &best, &which);
  if (p.m > 32 && p.m <= 512) consider_tc<1, 64>(p, dev, fit, &best, &which);
  if (p.m > 64 && p.m <= 1024) consider_tc<1, 128>(p, dev, fit, &best, &which);
  if (p.m > 64) consider_tc<2, 128>(p, dev, fit, &best, &which);
  if (p.m > 128) consider_tc<2, 256>(p, dev, fit, &best, &which);
  switch (which) {
    case 8: return launch_few<1, F32>(p, dev, stream);
    case 16: return launch_few<2, F32>(p, dev, stream);
    case 1032: return launch_tc<1, 32, F32>(p, dev, stream);
    case 1064: return launch_tc<1, 64, F32>(p, dev, stream);
    case 1128: return launch_tc<1, 128, F32>(p, dev, stream);
    case 2128: return launch_tc<2, 128, F32>(p, dev, stream);
    default: return launch_tc<2, 256, F32>(p, dev, stream);
  }
}

}  // namespace

extern "C" {

fp8q_status fp8q_nss_fp8(void* y_bf16, uint8_t* q_e4m3, const void* x_bf16,
                         const void* scale_bf16, const void* shift_bf16, int64_t mod_rows,
                         const float* input_scale, int64_t rows, int64_t cols, float eps,
                         cudaStream_t stream) {
  fp8q_status st = check_ln_shape(rows, cols, mod_rows, eps);
  if (st != FP8Q_OK || rows == 0) return st;
  if (!y_bf16 || !q_e4m3 || !x_bf16 || !scale_bf16 || !shift_bf16 || !input_scale)
    return FP8Q_ERR_NULL;
  if (!aligned16(y_bf16) || !aligned16(q_e4m3) || !aligned16(x_bf16) || !aligned16(scale_bf16) ||
      !aligned16(shift_bf16))
    return FP8Q_ERR_ALIGN;
  const int64_t n_mod = mod_count(rows, mod_rows);
  const size_t n = size_t(rows) * size_t(cols);
  const Range y{y_bf16, n * 2}, q{q_e4m3, n}, x{x_bf16, n * 2};
  const Range sc{scale_bf16, size_t(n_mod) * cols * 2}, sh{shift_bf16, size_t(n_mod) * cols * 2};
  const Range is{input_scale, 4};
  for (Range out : {y, q})
    for (Range in : {x, sc, sh, is})
      if (overlap(out, in)) return FP8Q_ERR_ALIAS;
  if (overlap(y, q)) return FP8Q_ERR_ALIAS;
  const DeviceInfo* dev = nullptr;
  st = current_device(&dev);
  if (st != FP8Q_OK) return st;
  fp8q::NssParams p{};
  p.x = static_cast<const uint16_t*>(x_bf16);
  p.scale = static_cast<const uint16_t*>(scale_bf16);
  p.shift = static_cast<const uint16_t*>(shift_bf16);
  p.y = static_cast<uint16_t*>(y_bf16);
  p.q = q_e4m3;
  p.input_scale = input_scale;
  p.rows = rows;
  p.mod_rows = mod_rows;
  p.cols = int(cols);
  p.eps = eps;
  return dispatch_ln<false, false>(p, *dev, n_mod, stream);
}

fp8q_status fp8q_scale_residual_nss_fp8(void* residual_out, void* y_bf16, uint8_t* q_e4m3,
                                        const void* x_bf16, const void* residual_bf16,
                                        const void* bias_bf16, const void* gate_bf16,
                                        const void* scale_bf16, const void* shift_bf16,
                                        int64_t mod_rows, const float* input_scale,
                                        int64_t rows, int64_t cols, float eps,
                                        cudaStream_t stream) {
  fp8q_status st = check_ln_shape(rows, cols, mod_rows, eps);
  if (st != FP8Q_OK || rows == 0) return st;
  if (!residual_out || !y_bf16 || !q_e4m3 || !x_bf16 || !residual_bf16 || !gate_bf16 ||
      !scale_bf16 || !shift_bf16 || !input_scale)
    return FP8Q_ERR_NULL;
  if (!aligned16(residual_out) || !aligned16(y_bf16) || !aligned16(q_e4m3) ||
      !aligned16(x_bf16) || !aligned16(residual_bf16) || !aligned16(gate_bf16) ||
      !aligned16(scale_bf16) || !aligned16(shift_bf16) || (bias_bf16 && !aligned16(bias_bf16)))
    return FP8Q_ERR_ALIGN;
  const int64_t n_mod = mod_count(rows, mod_rows);
  const size_t n = size_t(rows) * size_t(cols);
  const size_t mod_bytes = size_t(n_mod) * cols * 2;
  const Range ro{residual_out, n * 2}, y{y_bf16, n * 2}, q{q_e4m3, n};
  const Range x{x_bf16, n * 2}, res{residual_bf16, n * 2}, b{bias_bf16, size_t(cols) * 2};
  const Range g{gate_bf16, mod_bytes}, sc{scale_bf16, mod_bytes}, sh{shift_bf16, mod_bytes};
  const Range is{input_scale, 4};
  for (Range out : {ro, y, q})
    for (Range in : {x, res, b, g, sc, sh, is}) {
      if (out.p == ro.p && same(ro, res) && in.p == res.p) continue;  // in-place residual
      if (overlap(out, in)) return FP8Q_ERR_ALIAS;
    }
  if (overlap(ro, y) || overlap(ro, q) || overlap(y, q)) return FP8Q_ERR_ALIAS;
  const DeviceInfo* dev = nullptr;
  st = current_device(&dev);
  if (st != FP8Q_OK) return st;
  fp8q::NssParams p{};
  p.x = static_cast<const uint16_t*>(x_bf16);
  p.residual = static_cast<const uint16_t*>(residual_bf16);
  p.bias = static_cast<const uint16_t*>(bias_bf16);
  p.gate = static_cast<const uint16_t*>(gate_bf16);
  p.scale = static_cast<const uint16_t*>(scale_bf16);
  p.shift = static_cast<const uint16_t*>(shift_bf16);
  p.residual_out = static_cast<uint16_t*>(residual_out);
  p.y = static_cast<uint16_t*>(y_bf16);
  p.q = q_e4m3;
  p.input_scale = input_scale;
  p.rows = rows;
  p.mod_rows = mod_rows;
  p.cols = int(cols);
  p.eps = eps;
  if (bias_bf16) return dispatch_ln<true, true>(p, *dev, n_mod, stream);
  return dispatch_ln<true, false>(p, *dev, n_mod, stream);
}

fp8q_status fp8q_bias_mul_add(void* y_bf16, const void* x_bf16, const void* bias_bf16,
                              const void* gate_bf16, const void* residual_bf16, int64_t rows,
                              int64_t cols, cudaStream_t stream) {
  if (rows < 0 || cols < 8 || cols % 8 != 0 || cols > kMaxEwCols) return FP8Q_ERR_SHAPE;
  if (rows == 0) return FP8Q_OK;
  if (!y_bf16 || !x_bf16 || !bias_bf16 || !gate_bf16 || !residual_bf16) return FP8Q_ERR_NULL;
  if (!aligned16(y_bf16) || !aligned16(x_bf16) || !aligned16(bias_bf16) ||
      !aligned16(gate_bf16) || !aligned16(residual_bf16))
    return FP8Q_ERR_ALIGN;
  const size_t n = size_t(rows) * size_t(cols);
  const Range y{y_bf16, n * 2}, x{x_bf16, n * 2}, res{residual_bf16, n * 2};
  const Range b{bias_bf16, size_t(cols) * 2}, g{gate_bf16, size_t(cols) * 2};
  // Elementwise: y may be exactly x or exactly residual; partial overlaps are rejected.
  if ((overlap(y, x) && !same(y, x)) || (overlap(y, res) && !same(y, res)) || overlap(y, b) ||
      overlap(y, g))
    return FP8Q_ERR_ALIAS;
  const DeviceInfo* dev = nullptr;
  fp8q_status st = current_device(&dev);
  if (st != FP8Q_OK) return st;
  const int chunks = int(cols / 8);
  const int per_cta = fp8q::kEwThreads * fp8q::kBmaUnroll;
  const unsigned gy = unsigned((chunks + per_cta - 1) / per_cta);
  if (gy > 65535u) return FP8Q_ERR_SHAPE;
  // Two rows per CTA once one row per CTA would need more than one wave of resident CTAs.
  auto* fn1 = fp8q::bias_mul_add_kernel<1>;
  auto* fn2 = fp8q::bias_mul_add_kernel<2>;
  int bps = 0;
  st = blocks_per_sm(reinterpret_cast<const void*>(fn2), fp8q::kEwThreads, 0, &bps);
  if (st != FP8Q_OK) return st;
  const int64_t wave = int64_t(dev->sms) * (bps > 0 ? bps : 1);
  const bool two = rows * int64_t(gy) > wave;
  const int64_t gx64 = two ? (rows + 1) / 2 : rows;
  const unsigned gx = unsigned(gx64 < 0x7FFFFFFF ? gx64 : 0x7FFFFFFF);
  auto* yp = static_cast<uint16_t*>(y_bf16);
  auto* xp = static_cast<const uint16_t*>(x_bf16);
  auto* bp = static_cast<const uint16_t*>(bias_bf16);
  auto* gp = static_cast<const uint16_t*>(gate_bf16);
  auto* rp = static_cast<const uint16_t*>(residual_bf16);
  if (two)
    return launch(fn2, dim3(gx, gy), dim3(fp8q::kEwThreads), 0, stream, yp, xp, bp, gp, rp, rows,
                  int(cols));
  return launch(fn1, dim3(gx, gy), dim3(fp8q::kEwThreads), 0, stream, yp, xp, bp, gp, rp, rows,
                int(cols));
}

fp8q_status fp8q_token_cat_fp8(uint8_t* q_e4m3, const void* a_bf16, int64_t a_cols,
                               const void* m_bf16, int64_t m_cols, const float* input_scale,
                               int64_t rows, cudaStream_t stream) {
  if (rows < 0 || a_cols < 16 || m_cols < 16 || a_cols % 16 != 0 || m_cols % 16 != 0 ||
      a_cols + m_cols > kMaxEwCols)
    return FP8Q_ERR_SHAPE;
  if (rows == 0) return FP8Q_OK;
  if (!q_e4m3 || !a_bf16 || !m_bf16 || !input_scale) return FP8Q_ERR_NULL;
  if (!aligned16(q_e4m3) || !aligned16(a_bf16) || !aligned16(m_bf16)) return FP8Q_ERR_ALIGN;
  const Range q{q_e4m3, size_t(rows) * size_t(a_cols + m_cols)};
  const Range a{a_bf16, size_t(rows) * size_t(a_cols) * 2};
  const Range m{m_bf16, size_t(rows) * size_t(m_cols) * 2};
  const Range is{input_scale, 4};
  if (overlap(q, a) || overlap(q, m) || overlap(q, is)) return FP8Q_ERR_ALIAS;
  const DeviceInfo* dev = nullptr;
  fp8q_status st = current_device(&dev);
  if (st != FP8Q_OK) return st;
  const int chunks = int((a_cols + m_cols) / 8);
  const int per_cta = fp8q::kEwThreads * fp8q::kCatUnroll;
  const unsigned gy = unsigned((chunks + per_cta - 1) / per_cta);
  const unsigned gx = unsigned(rows < 0x7FFFFFFF ? rows : 0x7FFFFFFF);
  if (gy > 65535u) return FP8Q_ERR_SHAPE;
  return launch(fp8q::token_cat_fp8_kernel, dim3(gx, gy), dim3(fp8q::kEwThreads), 0, stream,
                q_e4m3, static_cast<const uint16_t*>(a_bf16), int(a_cols),
                static_cast<const uint16_t*>(m_bf16), int(m_cols), input_scale, rows);
}

int64_t fp8q_nvfp4_scale_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 16 || cols % 16 != 0 || cols > kMaxEwCols) return -1;
  const int64_t groups = cols / 16;
  return (rows + 127) / 128 * 128 * ((groups + 3) / 4 * 4);
}

fp8q_status fp8q_token_cat_nvfp4(uint8_t* q_fp4, uint8_t* sf_e4m3, const void* a_bf16,
                                 int64_t a_cols, const void* m_bf16, int64_t m_cols,
                                 const float* global_scale, int64_t rows, cudaStream_t stream) {
  if (rows < 0 || a_cols < 64 || m_cols < 64 || a_cols % 64 != 0 || m_cols % 64 != 0 ||
      a_cols + m_cols > kMaxEwCols)
    return FP8Q_ERR_SHAPE;
  if (rows == 0) return FP8Q_OK;
  if (!q_fp4 || !sf_e4m3 || !a_bf16 || !m_bf16 || !global_scale) return FP8Q_ERR_NULL;
  if (!aligned32(q_fp4) || !aligned32(a_bf16) || !aligned32(m_bf16) || !aligned16(sf_e4m3))
    return FP8Q_ERR_ALIGN;
  const int64_t cols = a_cols + m_cols;
  const int64_t rows_pad = (rows + 127) / 128 * 128;
  const Range q{q_fp4, size_t(rows) * size_t(cols / 2)};
  const Range sf{sf_e4m3, size_t(fp8q_nvfp4_scale_bytes(rows, cols))};
  const Range a{a_bf16, size_t(rows) * size_t(a_cols) * 2};
  const Range m{m_bf16, size_t(rows) * size_t(m_cols) * 2};
  const Range gs{global_scale, 4};
  if (overlap(q, a) || overlap(q, m) || overlap(q, gs) || overlap(sf, a) || overlap(sf, m) ||
      overlap(sf, gs) || overlap(q, sf))
    return FP8Q_ERR_ALIAS;
  const DeviceInfo* dev = nullptr;
  fp8q_status st = current_device(&dev);
  if (st != FP8Q_OK) return st;
  const int64_t units = cols / 64;
  const int64_t items = rows_pad / 8 * ((units + 3) / 4);  // warp items (see the kernel)
  const int64_t warps_per_cta = fp8q::kFp4Threads / 32;
  int bps = 0;
  st = blocks_per_sm(reinterpret_cast<const void*>(fp8q::token_cat_nvfp4_kernel),
                     fp8q::kFp4Threads, 0, &bps);
  if (st != FP8Q_OK) return st;
  // One item per warp (short CTAs, one after another) unless that is under two waves of
  // resident CTAs: then a persistent grid of exactly one wave spreads the items evenly over
  // all warps (FLUX.2 widths: 512 tokens 8.16 -> 7.69 us; at 4096 tokens and above one item
  // per warp is faster, 42.5 against 47.7 us persistent).
  const int64_t blocks = (items + warps_per_cta - 1) / warps_per_cta;
  const int64_t wave = int64_t(dev->sms) * std::max(bps, 1);
  const int64_t grid = blocks < 2 * wave ? std::min(blocks, wave) : blocks;
  if (grid > 0x7FFFFFFF) return FP8Q_ERR_SHAPE;
  return launch(fp8q::token_cat_nvfp4_kernel, dim3(unsigned(grid)), dim3(fp8q::kFp4Threads), 0,
                stream, q_fp4, sf_e4m3, static_cast<const uint16_t*>(a_bf16), int(a_cols / 64),
                static_cast<const uint16_t*>(m_bf16), int(m_cols / 64), global_scale, rows,
                rows_pad);
}

fp8q_status fp8q_qkv_epilogue(void* joint_q, void* joint_k, void* joint_v,
                              const fp8q_qkv_stream* txt, const fp8q_qkv_stream* img,
                              int64_t heads, cudaStream_t stream) {
  if (!txt || !img) return FP8Q_ERR_NULL;
  if (heads < 1 || heads > 4096) return FP8Q_ERR_SHAPE;
  const int64_t width = heads * fp8q::kHeadDim;
  const fp8q_qkv_stream* st[2] = {txt, img};
  for (const fp8q_qkv_stream* s : st) {
    if (s->tokens < 0 || (s->tokens > 0 && (s->ld < width || s->ld % 16 != 0)))
      return FP8Q_ERR_SHAPE;
  }
  const int64_t total = txt->tokens + img->tokens;
  if (total == 0) return FP8Q_OK;
  for (const fp8q_qkv_stream* s : st) {
    if (s->tokens == 0) continue;
    if (!(s->eps > 0.0f) || !std::isfinite(s->eps)) return FP8Q_ERR_VALUE;
  }
  if (!joint_q || !joint_k || !joint_v) return FP8Q_ERR_NULL;
  for (const fp8q_qkv_stream* s : st) {
    if (s->tokens == 0) continue;
    if (!s->q || !s->k || !s->v || !s->q_weight || !s->k_weight || !s->cos_sin)
      return FP8Q_ERR_NULL;
    if (!aligned32(s->q) || !aligned32(s->k) || !aligned32(s->v) || !aligned32(s->q_weight) ||
        !aligned32(s->k_weight) || !aligned32(s->cos_sin))
      return FP8Q_ERR_ALIGN;
  }
  if (!aligned32(joint_q) || !aligned32(joint_k) || !aligned32(joint_v)) return FP8Q_ERR_ALIGN;
  const size_t out_bytes = size_t(total) * size_t(width) * 2;
  const Range outs[3] = {{joint_q, out_bytes}, {joint_k, out_bytes}, {joint_v, out_bytes}};
  for (int i = 0; i < 3; ++i) {
    for (int j = i + 1; j < 3; ++j)
      if (overlap(outs[i], outs[j])) return FP8Q_ERR_ALIAS;
    for (const fp8q_qkv_stream* s : st) {
      if (s->tokens == 0) continue;
      const Range ins[6] = {{s->q, strided_bytes(s->tokens, s->ld, width)},
                            {s->k, strided_bytes(s->tokens, s->ld, width)},
                            {s->v, strided_bytes(s->tokens, s->ld, width)},
                            {s->q_weight, size_t(fp8q::kHeadDim) * 2},
                            {s->k_weight, size_t(fp8q::kHeadDim) * 2},
                            {s->cos_sin, size_t(s->tokens) * fp8q::kHeadDim * 4}};
      for (const Range& r : ins)
        if (overlap(outs[i], r)) return FP8Q_ERR_ALIAS;
    }
  }
  const DeviceInfo* dev = nullptr;
  fp8q_status stt = current_device(&dev);
  if (stt != FP8Q_OK) return stt;
  fp8q::QkvParams p;
  p.jq = static_cast<uint16_t*>(joint_q);
  p.jk = static_cast<uint16_t*>(joint_k);
  p.jv = static_cast<uint16_t*>(joint_v);
  fp8q::QkvStream* dstp[2] = {&p.txt, &p.img};
  for (int i = 0; i < 2; ++i) {
    dstp[i]->q = static_cast<const uint16_t*>(st[i]->q);
    dstp[i]->k = static_cast<const uint16_t*>(st[i]->k);
    dstp[i]->v = static_cast<const uint16_t*>(st[i]->v);
    dstp[i]->wq = static_cast<const uint16_t*>(st[i]->q_weight);
    dstp[i]->wk = static_cast<const uint16_t*>(st[i]->k_weight);
    dstp[i]->cos_sin = st[i]->cos_sin;
    dstp[i]->ld = st[i]->ld;
    dstp[i]->tokens = st[i]->tokens;
    dstp[i]->eps = st[i]->eps;
  }
  p.heads = int(heads);
  if (heads <= fp8q::kQkvMaxWsHeads) {
    // warp-specialised: one CTA per SM (never more CTAs than tokens), a ring of whole tokens
    const size_t per_stage = fp8q::qws_stage_bytes(int(heads)) + 20;
    const int64_t fit = (int64_t(dev->smem_optin) - fp8q::kQkvWeightBytes - 16) / int64_t(per_stage);
    const int stages = int(std::min<int64_t>(fit, fp8q::kQwsMaxStages));
    if (stages >= 2) {
      const size_t smem = fp8q::qws_smem_bytes(int(heads), stages);
      const int nw = fp8q::qws_qk_warps(int(heads));
      auto* fn = nw == 16 ? fp8q::qkv_ws_kernel<16> : fp8q::qkv_ws_kernel<13>;
      const int threads = fp8q::qws_threads(nw);
      int bps = 0;
      stt = blocks_per_sm(reinterpret_cast<const void*>(fn), threads, smem, &bps);
      if (stt != FP8Q_OK) return stt;
      if (bps > 0) {
        const int64_t grid = std::min<int64_t>(total, dev->sms);
        return launch(fn, dim3(unsigned(grid)), dim3(threads), smem, stream, p, stages);
      }
    }
  }
  const unsigned gx = unsigned(total < 0x7FFFFFFF ? total : 0x7FFFFFFF);
  return launch(fp8q::qkv_epilogue_kernel, dim3(gx), dim3(fp8q::kQkvWarps * 32), 0, stream, p);
}

fp8q_status fp8q_rms_norm_quant(void* residual_out, void* q, float* q_scale, const void* x_bf16,
                                const void* residual_bf16, const void* weight_bf16, int q_type,
                                int64_t rows, int64_t cols, float eps, cudaStream_t stream) {
  fp8q_status st = check_ln_shape(rows, cols, 0, eps);
  if (st != FP8Q_OK) return st;
  if (rows > INT64_MAX / cols / 4) return FP8Q_ERR_SHAPE;
  if (q_type != FP8Q_INT8 && q_type != FP8Q_E4M3) return FP8Q_ERR_VALUE;
  if (rows == 0) return FP8Q_OK;
  if (!q || !q_scale || !x_bf16 || !weight_bf16 || !residual_out != !residual_bf16)
    return FP8Q_ERR_NULL;
  if (!aligned16(q) || !aligned16(x_bf16) || !aligned16(weight_bf16) || !aligned4(q_scale) ||
      (residual_bf16 && (!aligned16(residual_out) || !aligned16(residual_bf16))))
    return FP8Q_ERR_ALIGN;
  const size_t n = size_t(rows) * size_t(cols);
  const Range ro{residual_out, n * 2}, qr{q, n}, sr{q_scale, size_t(rows) * 4};
  const Range x{x_bf16, n * 2}, res{residual_bf16, n * 2}, w{weight_bf16, size_t(cols) * 2};
  for (Range out : {ro, qr, sr})
    for (Range in : {x, res, w}) {
      if (out.p == ro.p && same(ro, res) && in.p == res.p) continue;  // in-place residual
      if (overlap(out, in)) return FP8Q_ERR_ALIAS;
    }
  if (overlap(ro, qr) || overlap(ro, sr) || overlap(qr, sr)) return FP8Q_ERR_ALIAS;
  const DeviceInfo* dev = nullptr;
  st = current_device(&dev);
  if (st != FP8Q_OK) return st;
  fp8q::RmsParams p{};
  p.x = static_cast<const uint16_t*>(x_bf16);
  p.residual = static_cast<const uint16_t*>(residual_bf16);
  p.weight = static_cast<const uint16_t*>(weight_bf16);
  p.h = static_cast<uint16_t*>(residual_out);
  p.q = static_cast<uint8_t*>(q);
  p.scale = q_scale;
  p.rows = rows;
  p.cols = int(cols);
  p.eps = eps;
  if (q_type == FP8Q_INT8)
    return residual_bf16 ? launch_rms<true, true>(p, *dev, stream)
                         : launch_rms<true, false>(p, *dev, stream);
  return residual_bf16 ? launch_rms<false, true>(p, *dev, stream)
                       : launch_rms<false, false>(p, *dev, stream);
}

fp8q_status fp8q_silu_mul_quant(void* q, float* q_scale, const void* gate_bf16,
                                const void* up_bf16, int64_t ld, int q_type, int64_t rows,
                                int64_t cols, cudaStream_t stream) {
  if (rows < 0 || cols < 8 || cols % 8 != 0 || cols > kMaxSiluCols) return FP8Q_ERR_SHAPE;
  if (ld < cols || ld % 8 != 0 || ld > kMaxEwCols || rows > INT64_MAX / ld / 4)
    return FP8Q_ERR_SHAPE;
  if (q_type != FP8Q_INT8 && q_type != FP8Q_E4M3) return FP8Q_ERR_VALUE;
  if (rows == 0) return FP8Q_OK;
  if (!q || !q_scale || !gate_bf16 || !up_bf16) return FP8Q_ERR_NULL;
  if (!aligned16(q) || !aligned16(gate_bf16) || !aligned16(up_bf16) || !aligned4(q_scale))
    return FP8Q_ERR_ALIGN;
  const Range qr{q, size_t(rows) * size_t(cols)}, sr{q_scale, size_t(rows) * 4};
  const Range g{gate_bf16, strided_bytes(rows, ld, cols)};
  const Range u{up_bf16, strided_bytes(rows, ld, cols)};
  for (Range out : {qr, sr})
    if (overlap(out, g) || overlap(out, u)) return FP8Q_ERR_ALIAS;
  if (overlap(qr, sr)) return FP8Q_ERR_ALIAS;
  const DeviceInfo* dev = nullptr;
  fp8q_status st = current_device(&dev);
  if (st != FP8Q_OK) return st;
  fp8q::SiluParams p{};
  p.gate = static_cast<const uint16_t*>(gate_bf16);
  p.up = static_cast<const uint16_t*>(up_bf16);
  p.ld = ld;
  p.q = static_cast<uint8_t*>(q);
  p.scale = q_scale;
  p.rows = rows;
  p.cols = int(cols);
  return q_type == FP8Q_INT8 ? launch_silu<true>(p, *dev, stream)
                             : launch_silu<false>(p, *dev, stream);
}

fp8q_status fp8q_int8_matmul(void* out, const int8_t* a, int64_t lda, const float* a_scale,
                             const int8_t* w, const float* w_scale, const void* bias_bf16,
                             int out_type, int64_t m, int64_t n, int64_t k, cudaStream_t stream) {
  if (m < 0 || n < 1 || n > INT32_MAX || m > INT32_MAX || k < 16 || k % 16 != 0 || k > kMaxMmK ||
      lda < k || lda % 16 != 0 || lda > kMaxEwCols)
    return FP8Q_ERR_SHAPE;
  if (out_type != FP8Q_OUT_BF16 && out_type != FP8Q_OUT_FP32) return FP8Q_ERR_VALUE;
  if (m == 0) return FP8Q_OK;
  if (!out || !a || !a_scale || !w || !w_scale) return FP8Q_ERR_NULL;
  const size_t width = out_type == FP8Q_OUT_FP32 ? 4 : 2;
  if (!aligned16(a) || !aligned16(w) || !aligned4(a_scale) || !aligned4(w_scale) ||
      (reinterpret_cast<uintptr_t>(out) & (width - 1)) != 0 ||
      (reinterpret_cast<uintptr_t>(bias_bf16) & 1) != 0)
    return FP8Q_ERR_ALIGN;
  const Range o{out, size_t(m) * size_t(n) * width};
  for (Range in : {Range{a, size_t(m - 1) * size_t(lda) + size_t(k)},
                   Range{w, size_t(n) * size_t(k)}, Range{a_scale, size_t(m) * 4},
                   Range{w_scale, size_t(n) * 4}, Range{bias_bf16, size_t(n) * 2}})
    if (overlap(o, in)) return FP8Q_ERR_ALIAS;
  const DeviceInfo* dev = nullptr;
  fp8q_status st = current_device(&dev);
  if (st != FP8Q_OK) return st;
  fp8q::MmParams p{};
  p.a = a;
  p.w = w;
  p.a_scale = a_scale;
  p.w_scale = w_scale;
  p.bias = static_cast<const uint16_t*>(bias_bf16);
  p.out = out;
  p.lda = lda;
  p.m = m;
  p.n = n;
  p.k = k;
  return out_type == FP8Q_OUT_FP32 ? launch_int8_matmul<true>(p, *dev, stream)
                                   : launch_int8_matmul<false>(p, *dev, stream);
}

fp8q_status fp8q_device_error(unsigned int* bits) {
  if (!bits) return FP8Q_ERR_NULL;
  const DeviceInfo* dev = nullptr;
  fp8q_status st = current_device(&dev);
  if (st != FP8Q_OK) return st;
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, fp8q::g_device_error, sizeof v);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyFromSymbol(g_device_error)");
  const unsigned int zero = 0;
  e = cudaMemcpyToSymbol(fp8q::g_device_error, &zero, sizeof zero);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyToSymbol(g_device_error)");
  *bits = v;
  return FP8Q_OK;
}

const char* fp8q_status_string(int status) {
  switch (status) {
    case FP8Q_OK: return "ok";
    case FP8Q_ERR_NULL: return "null pointer";
    case FP8Q_ERR_ALIGN: return "pointer not aligned (16 bytes; 32 for NVFP4 and QKV data)";
    case FP8Q_ERR_SHAPE: return "unsupported shape";
    case FP8Q_ERR_UNSUPPORTED: return "device is not compute capability 10.3 (GB300)";
    case FP8Q_ERR_ALIAS: return "an output overlaps an input or another output";
    case FP8Q_ERR_CUDA: return "CUDA runtime error";
    case FP8Q_ERR_VALUE: return "scalar argument out of range";
    default: return "unknown status";
  }
}

int fp8q_last_cuda_error(void) { return g_last_cuda_error; }

const char* fp8q_last_error_detail(void) { return g_last_detail; }

int fp8q_version(void) { return 0x000300; }

}  // extern "C"
