/* A stand-in for the CUDA runtime calls that the library's host side makes, preloaded over the real
 * one: a host without a GPU sees the launch shapes that the library chooses. Nothing runs. */
#include <cuda.h>
#include <cuda_runtime_api.h>

struct fake_launch {
  const void *fn;
  unsigned grid, block, cluster;
  unsigned long smem;
};

#define LAUNCHES 65536
static struct fake_launch launches[LAUNCHES];
static int n_launches, n_queries, n_refused, n_falls, device;

/* dynamic shared-memory limits of (device, function) pairs, as the runtime keeps them */
static struct { int dev; const void *fn; int limit; } limits[65536];
static int n_limits;

static int *limit_of(const void *fn) {
  for (int i = 0; i < n_limits; ++i)
    if (limits[i].dev == device && limits[i].fn == fn) return &limits[i].limit;
  limits[n_limits].dev = device;
  limits[n_limits].fn = fn;
  limits[n_limits].limit = 48 * 1024;
  return &limits[n_limits++].limit;
}

int fake_launches(void) { return n_launches; }
int fake_queries(void) { return n_queries; }
int fake_refused(void) { return n_refused; }
int fake_limit_falls(void) { return n_falls; }
void fake_device(int d) { device = d; }
struct fake_launch fake_launch_at(int i) { return launches[i]; }

/* CTAs of 128 registers a thread on an SM of 65536 registers, 2048 threads and 228 KB. */
static int resident(int threads, size_t smem) {
  int by_regs = 65536 / (128 * threads), by_smem = (int)(233472 / (smem + 1024));
  int by_threads = 2048 / threads, r = by_regs < by_smem ? by_regs : by_smem;
  r = r < by_threads ? r : by_threads;
  return r < 32 ? r : 32;
}

cudaError_t cudaGetDevice(int *d) {
  *d = device;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int *v, enum cudaDeviceAttr a, int d) {
  (void)d;
  *v = a == cudaDevAttrComputeCapabilityMajor   ? 10
       : a == cudaDevAttrComputeCapabilityMinor ? 3
       : a == cudaDevAttrMultiProcessorCount    ? 152
                                                : 232448;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void *fn, enum cudaFuncAttribute a, int v) {
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) {
    if (v < *limit_of(fn)) ++n_falls;
    *limit_of(fn) = v;
  }
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int *n, const void *fn, int threads,
                                                          size_t smem) {
  (void)fn;
  ++n_queries;
  *n = resident(threads, smem);
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *fn, const cudaLaunchConfig_t *c) {
  (void)fn;
  *n = 152 / (int)c->gridDim.x;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *fn, void **args) {
  (void)args;
  if (c->dynamicSmemBytes > (size_t)*limit_of(fn)) {
    ++n_refused;
    return cudaErrorInvalidValue;
  }
  struct fake_launch l = {fn, c->gridDim.x, c->blockDim.x, 1, c->dynamicSmemBytes};
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension)
      l.cluster = c->attrs[i].val.clusterDim.x;
  launches[n_launches++ % LAUNCHES] = l;
  return cudaSuccess;
}
static CUresult encode(void) { return CUDA_SUCCESS; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *name, void **fn, unsigned v,
                                             unsigned long long flags,
                                             enum cudaDriverEntryPointQueryResult *found) {
  (void)name, (void)v, (void)flags;
  *fn = (void *)encode;
  *found = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
