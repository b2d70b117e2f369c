// host_launch.cuh -- what the entry points share on the host: device checks, launch caches, argument
// checks, the launch itself. One instance for the library's translation units.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "fp8q.h"

namespace fp8q_host {

// Reads and clears the device error word of cache_capi.cu's kernels (each unit has its own).
fp8q_status take_cache_device_error(unsigned int* bits);

constexpr int kMaxDevices = 64;

inline thread_local int g_last_cuda_error = 0;
inline thread_local char g_last_detail[160] = "";

struct DeviceInfo {
  int major = 0, minor = 0, sms = 0, smem_optin = 0;
  bool ok = false;
};

inline DeviceInfo g_dev[kMaxDevices];
inline std::once_flag g_dev_once[kMaxDevices];

// Records which runtime call failed (thread-local) and returns FP8Q_ERR_CUDA.
inline fp8q_status cuda_fail(cudaError_t e, const char* site, long long arg = -1) {
  g_last_cuda_error = int(e);
  std::snprintf(g_last_detail, sizeof g_last_detail, "%s(%lld): %s", site, arg,
                cudaGetErrorName(e));
  return FP8Q_ERR_CUDA;
}

// Current device, checked to be compute capability 10.3.
inline fp8q_status current_device(const DeviceInfo** out) {
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
inline OccSet g_occ[kOccSets];

inline OccSet& occ_set(int dev, const void* fn, int threads, size_t smem) {
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
inline SmemLimits g_lim[kMaxDevices];
inline std::mutex g_occ_mu;

inline fp8q_status raise_smem_limit(int dev, const void* fn, size_t smem) {
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

inline fp8q_status blocks_per_sm(const void* fn, int threads, size_t smem, int* blocks) {
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

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// Bytes spanned by `tokens` rows of `width` BF16 values at a stride of `ld` values.
inline size_t strided_bytes(int64_t tokens, int64_t ld, int64_t width) {
  return tokens > 0 ? size_t((tokens - 1) * ld + width) * 2 : 0;
}

struct Range {
  const void* p;
  size_t bytes;
};

inline bool overlap(Range a, Range b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

inline bool same(Range a, Range b) { return a.p == b.p && a.bytes == b.bytes; }

// One launch; the status is this launch's own (cudaLaunchKernelEx's return value), so an
// unrelated pending error of another library on the same thread is never reported as ours.
// Launches allow programmatic dependent launch: a kernel may be scheduled while the previous
// kernel in the stream drains, and every kernel executes griddepcontrol.wait before its first
// global-memory access, so producer -> consumer ordering is unchanged. One exception: attn_join_kernel
// reads the sequences' lengths before its wait. It follows paged_attention_kernel, which lets it start only
// after its own wait, when whatever wrote the lengths is complete.
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

// The driver's tensor-map encoder, through the runtime (the library links no libcuda).
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline fp8q_status encode_tiled(EncodeTiled* fn) {
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

}  // namespace fp8q_host
