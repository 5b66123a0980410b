// layer_norm.cuh - what layer norm's forward and backward share: how rows lie on threads, and the
// sums over a row.
//
// A row is held in registers as vectors of 8 columns (packed pairs), NV a thread.  Rows of up to
// 512 columns take G lanes of a warp; up to 8192 a block; wider ones a cluster of 2 or 4 blocks
// with a slice of the columns each, whose sums go through each other's shared memory.
#pragma once

#include "cluster.cuh"
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {

// Sums over a row of kCount values a thread: G lanes of a warp, or (G = 0) the block and its
// cluster.  `turn` alternates between the sums of a block: their shared memory does, too, so that
// one barrier a sum is enough.
struct LnShared {
  float warp[2][3][32];
  float rank[2][4][4];
};
template <int G, int kCount>
__device__ __forceinline__ void sum_row(float (&v)[kCount], LnShared* s, int& turn, unsigned blocks) {
  constexpr int kLanes = G ? G : 32;
#pragma unroll
  for (int off = kLanes >> 1; off > 0; off >>= 1)
#pragma unroll
    for (int j = 0; j < kCount; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], off);
  if constexpr (G == 0) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < kCount; ++j) s->warp[turn][j][threadIdx.x >> 5] = v[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kCount; ++j) {  // every warp adds the warps' sums (16 at most)
      v[j] = lane < warps ? s->warp[turn][j][lane] : 0.f;
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) v[j] += __shfl_xor_sync(0xffffffffu, v[j], off);
      v[j] = __shfl_sync(0xffffffffu, v[j], 0);
    }
    if (blocks > 1) {
      if (threadIdx.x < blocks) {  // this block's sums into the others' memory
        static_assert(kCount <= 4, "two pairs a store");
        float q[4] = {};
#pragma unroll
        for (int j = 0; j < kCount; ++j) q[j] = v[j];
        store_to_rank(&s->rank[turn][cluster_rank()][0], threadIdx.x, pack2(q[0], q[1]), pack2(q[2], q[3]));
      }
      __syncwarp();
      cluster_sync();
#pragma unroll
      for (int j = 0; j < kCount; ++j) {
        v[j] = 0.f;
        for (unsigned k = 0; k < blocks; ++k) v[j] += s->rank[turn][k][j];
      }
    }
    turn ^= 1;
  }
}

// Where a thread's columns are: vector i holds columns first + i * step .. + 8 of the row, n[i] of
// which exist.
template <int G, int NV>
struct LnColumns {
  int first, n[NV];
  __device__ __forceinline__ LnColumns(const LnParams& p, unsigned rank) {
    const int lane = G ? threadIdx.x % (G ? G : 1) : threadIdx.x;
    const int base = (int)rank * p.slice, most = min(p.D - base, p.slice);
    first = base + lane * 8;
#pragma unroll
    for (int i = 0; i < NV; ++i) n[i] = most - (lane + i * step()) * 8;
  }
  static __device__ __forceinline__ int step() { return G ? G : blockDim.x; }
};

// Columns that do not exist become zero.
template <bool kWhole>
__device__ __forceinline__ void mask(f32x2 (&v)[4], int n) {
  if (kWhole) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a, b;
    unpack2(v[j], a, b);
    v[j] = pack2(2 * j < n ? a : 0.f, 2 * j + 1 < n ? b : 0.f);
  }
}
__device__ __forceinline__ float both(f32x2 v) {
  float a, b;
  unpack2(v, a, b);
  return a + b;
}

// The grid of `kernel` for rows on G lanes or blocks: as many blocks as are resident together, each
// takes its rows in turn.
template <typename Kernel>
cudaError_t ln_grid(Kernel kernel, const LnParams& p, int G, int threads, unsigned* grid) {
  int resident = 0;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kernel, threads, 0);
  if (e != cudaSuccess) return e;
  const long long per_block = G ? threads / G : 1, units = (p.rows + per_block - 1) / per_block;
  const long long most = (long long)(resident < 1 ? 1 : resident) * kSms / p.blocks;
  *grid = (unsigned)((units < most ? units : most) * p.blocks);
  return cudaSuccess;
}

}  // namespace gdn
