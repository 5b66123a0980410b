// cluster.cuh - thread-block clusters: barriers, stores into a neighbour's shared memory, launches.
#pragma once

#include "gdn_common.cuh"

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

// The same, counted as 16 bytes by the barrier `bar` of that block: the receiver waits for its barrier,
// and nothing of the sender's other accesses is waited for, as a cluster's barrier does.
__device__ __forceinline__ void send_to_rank(void* local, uint64_t* bar, unsigned rank, unsigned long long a,
                                             unsigned long long b) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(local));
  const uint32_t of = static_cast<uint32_t>(__cvta_generic_to_shared(bar));
  uint32_t there, its;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(its) : "r"(of), "r"(rank));
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(there),
               "l"(a), "l"(b), "r"(its)
               : "memory");
}
// Wait for phase `parity` of `bar`, whose bytes come from the cluster; gives up after `limit` cycles (about a
// second) and records that, and from then on (`dead`) no wait of the block lasts.
__device__ __forceinline__ void wait_for_ranks(uint64_t* bar, unsigned parity, unsigned* err, volatile int* dead,
                                               long long limit = 1ll << 31) {
  const auto done = [&] {
    unsigned ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(bar))), "r"(parity)
        : "memory");
    return ok != 0;
  };
  if (done()) return;
  const long long t0 = clock64();
  while (!done()) {
    if (*dead || clock64() - t0 > limit) {
      if (!*dead) record_error(err, kErrWaitTimeout);
      *dead = 1;
      return;
    }
  }
}
// The end of a block that exchanges so: no block leaves before its neighbours have sent what they send.  To one
// that has given up a wait some of that may be on its way still; it takes microseconds, and half a millisecond is
// waited.
__device__ __forceinline__ void leave_ranks(volatile int* dead) {
  cluster_sync();
  if (*dead) {
    const long long t0 = clock64();
    while (clock64() - t0 < (1ll << 20)) {
    }
  }
}

// A launch in clusters of `blocks` (1: none) neighbouring blocks, with `smem` bytes of dynamic memory.  `most`:
// what any launch of the kernel takes, allowed for all of them (another thread may launch it with more).
template <typename Kernel>
cudaError_t allow_clusters(Kernel kernel, unsigned blocks, size_t smem) {
  cudaError_t e = cudaSuccess;
  if (smem) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  // more than 8 is more than every GPU of the family takes
  if (e == cudaSuccess && blocks > 8)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}
struct ClusterConfig {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  ClusterConfig(unsigned grid, unsigned threads, unsigned blocks, size_t smem, cudaStream_t stream) {
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = blocks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = blocks > 1 ? 1 : 0;
  }
};
template <typename Kernel, typename Params>
cudaError_t launch_clusters(Kernel kernel, unsigned grid, unsigned threads, unsigned blocks, const Params& p,
                            cudaStream_t stream, size_t smem = 0, size_t most = 0) {
  const cudaError_t e = allow_clusters(kernel, blocks, most);
  if (e != cudaSuccess) return e;
  const ClusterConfig c(grid, threads, blocks, smem, stream);
  return cudaLaunchKernelEx(&c.cfg, kernel, p);
}

}  // namespace gdn
