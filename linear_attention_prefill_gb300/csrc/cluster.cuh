// cluster.cuh - thread-block clusters: barriers, stores into a neighbour's shared memory, launches.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// A block that runs says so at its start, and waits for the others' word before it first writes into
// their shared memory.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// every block of the cluster has arrived, and what they wrote before is seen
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// 16 bytes into the same place of block `rank`'s shared memory
__device__ __forceinline__ void store_to_rank(void* local, unsigned rank, unsigned long long a,
                                              unsigned long long b) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(local));
  uint32_t there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(there), "l"(a), "l"(b) : "memory");
}

// A launch in clusters of `blocks` (1: none) neighbouring blocks.
template <typename Kernel, typename Params>
cudaError_t launch_clusters(Kernel kernel, unsigned grid, unsigned threads, unsigned blocks, const Params& p,
                            cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = blocks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = blocks > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace gdn
