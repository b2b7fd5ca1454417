// cluster.cuh — thread-block clusters: launch and the few PTX operations that the
// accumulated-weight and eviction kernels use (distributed shared memory, barrier).
#pragma once

#include <atomic>

#include "rrq_device.cuh"

namespace rrq {

// All threads of the cluster meet; shared-memory writes before it are seen after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same in two halves, with work between them that the other CTAs need not wait for.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The 32-bit word at this CTA's shared address `addr` in the CTA of rank `rank`.
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr, uint32_t rank) {
  uint32_t v, a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// Lets `kernel` run with `smem` bytes and in clusters of 16, once per device (`done`: a bit per
// device, one word per kernel).
template <typename... KArgs>
cudaError_t allow_kernel(void (*kernel)(KArgs...), int smem, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

// Launch `kernel` in clusters of `size` CTAs along x (up to 16: the opt-in size), with
// programmatic stream serialization allowed.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, unsigned size, size_t smem,
                           cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = size;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// CTAs per cluster for `rows` rows of `n` tokens each: enough for every SM while a CTA keeps
// at least `least` tokens, a power of two, at most 16.
inline unsigned cluster_size(int64_t rows, int64_t n, int64_t least) {
  unsigned c = 1;
  while (c < 16 && rows * c * 2 <= 160 && n >= int64_t(c) * 2 * least) c *= 2;
  return c;
}

}  // namespace rrq
