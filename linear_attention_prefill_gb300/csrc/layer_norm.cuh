// layer_norm.cuh - what layer norm's forward and backward share: how rows lie on threads, and the
// sums over a row.
//
// A row is held in registers as vectors of 8 columns (packed pairs), NV a thread.  Rows of up to
// 512 columns take G lanes of a warp; up to 8192 a block; wider ones a cluster of 2 or 4 blocks
// with a slice of the columns each, whose sums go through each other's shared memory.  Many rows of whole
// vectors that one block takes arrive through a ring of shared memory.
#pragma once

#include <atomic>
#include <cstddef>

#include "cluster.cuh"
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {

// Sums over the block of kCount (1, 2, 4 or 8) values a thread.  Lanes halve the values that they go on
// with at each step: 8 values take 9 shuffles, not 40, and as many again over the warps' sums.  `turn`
// alternates, and the shared memory with it, so that one barrier a sum is enough.
struct alignas(16) LnShared {
  float warp[2][8][32];
  float rank[2][4][4];  // (written by 16 bytes)
};
static_assert(alignof(LnShared) % 16 == 0 && offsetof(LnShared, rank) % 16 == 0, "stores of 16 bytes into `rank`");
template <int kCount>
__device__ __forceinline__ float scatter_sums(float (&v)[kCount], int lane) {  // the lane's one of them
  int off = 16;
#pragma unroll
  for (int half = kCount / 2; half > 0; half >>= 1, off >>= 1) {
    const bool high = lane & off;
#pragma unroll
    for (int j = 0; j < half; ++j) {
      const float send = high ? v[j] : v[j + half], keep = high ? v[j + half] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, send, off);
    }
  }
#pragma unroll
  for (; off > 0; off >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
  return v[0];  // value lane / (32 / kCount)
}
template <int kCount>
__device__ __forceinline__ void sum_block(float (&v)[kCount], LnShared* s, int& turn) {
  constexpr int kLanes = 32 / kCount;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const float mine = scatter_sums(v, lane);
  if (lane % kLanes == 0) s->warp[turn][lane / kLanes][threadIdx.x >> 5] = mine;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kCount; ++j) v[j] = lane < warps ? s->warp[turn][j][lane] : 0.f;
  const float sum = scatter_sums(v, lane);
#pragma unroll
  for (int j = 0; j < kCount; ++j) v[j] = __shfl_sync(0xffffffffu, sum, j * kLanes);
  turn ^= 1;
}
// Sums over a row: G lanes of a warp, or (G = 0) the block and its cluster.
template <int G, int kCount>
__device__ __forceinline__ void sum_row(float (&v)[kCount], LnShared* s, int& turn, unsigned blocks) {
  if constexpr (G > 0) {
#pragma unroll
    for (int off = G >> 1; off > 0; off >>= 1)
#pragma unroll
      for (int j = 0; j < kCount; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], off);
  } else {
    const int here = turn;
    sum_block(v, s, turn);
    if (blocks > 1) {
      if (threadIdx.x < blocks) {  // this block's sums into the others' memory
        static_assert(kCount <= 4, "two pairs a store");
        float q[4] = {};
#pragma unroll
        for (int j = 0; j < kCount; ++j) q[j] = v[j];
        store_to_rank(&s->rank[here][cluster_rank()][0], threadIdx.x, pack2(q[0], q[1]), pack2(q[2], q[3]));
      }
      __syncwarp();
      cluster_sync();
#pragma unroll
      for (int j = 0; j < kCount; ++j) {
        v[j] = 0.f;
        for (unsigned k = 0; k < blocks; ++k) v[j] += s->rank[here][k][j];
      }
    }
  }
}

// Where a thread's columns are: vector i holds 8 of them, from (lane + i * lanes) * 8 on.  Whole rows (8-column
// vectors, 16 bytes aligned) are accessed so.  Of other rows a warp's accesses are dense, a column a lane,
// and turned into vectors in shared memory (a chunk of W lanes' vectors at a time): the sums are taken in the
// same order, so that alignment does not change results.
template <bool kWhole, int G, int NV>
struct LnColumns {
  static constexpr int W = G ? G : 32;
  int lane, lanes, base, most, l, chunk;
  float* turn;  // this chunk's 8 W floats
  __device__ __forceinline__ LnColumns(const LnParams& p, unsigned rank, float* scratch) {
    lane = G ? threadIdx.x % (G ? G : 1) : threadIdx.x;
    lanes = G ? G : blockDim.x;
    base = (int)rank * p.slice;
    most = min(p.D - base, p.slice);
    l = threadIdx.x % W;
    chunk = (lane - l) * 8;
    turn = scratch + (threadIdx.x - l) * 8;
  }
  __device__ __forceinline__ bool any(int i) const { return (lane + i * lanes) * 8 < most; }
  // of a row (from its first column on): vector i, or what of its chunk the lane's accesses get
  template <typename T>
  __device__ __forceinline__ Raw8<T> load(const T* row, int i) const {
    Raw8<T> r;
    if (kWhole) {
      if (any(i)) r.load(row + base + (lane + i * lanes) * 8);
    } else {
      const int c = chunk + i * lanes * 8 + l;
      const T* q = row + base + c;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = c + j * W < most ? to_f32(q[j * W]) : 0.f;
      r.set(o);
    }
    return r;
  }
  // the vector, zeros for columns that do not exist
  template <typename T>
  __device__ __forceinline__ void vector(const Raw8<T>& r, int i, f32x2 (&v)[4]) const {
    if (kWhole) {
      if (any(i)) {
        pairs_of(r, v);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = 0ull;
      }
      return;
    }
    float o[8];
    pairs_of(r, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) unpack2(v[j], o[2 * j], o[2 * j + 1]);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) turn[l + j * W] = o[j];
    __syncwarp();
    Raw8<float> x;
    x.load(turn + l * 8);
    pairs_of(x, v);
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int i, const f32x2 (&v)[4], bool some) const {
    if (kWhole) {
      if (some && any(i)) raw_of<T>(v).store(row + base + (lane + i * lanes) * 8);
      return;
    }
    __syncwarp();
    raw_of<float>(v).store(turn + l * 8);
    __syncwarp();
    const int c = chunk + i * lanes * 8 + l;
    T* q = row + base + c;
    if (!some) return;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j * W < most) from_f32(q + j * W, turn[l + j * W]);
  }
  __device__ __forceinline__ void mask(f32x2 (&v)[4], int i) const {  // columns that do not exist become zero
    const int n = most - (lane + i * lanes) * 8;
    if (kWhole) {
      if (n <= 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = 0ull;
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a, b;
      unpack2(v[j], a, b);
      v[j] = pack2(2 * j < n ? a : 0.f, 2 * j + 1 < n ? b : 0.f);
    }
  }
};
__device__ __forceinline__ float both(f32x2 v) {
  float a, b;
  unpack2(v, a, b);
  return a + b;
}
__device__ __forceinline__ float sum8(const f32x2 (&v)[4]) { return both(add2(add2(v[0], v[1]), add2(v[2], v[3]))); }

// Blocks an SM for rows of a block: about `most` threads together, 640 in the gradient.  There it is by the row's
// length alone: how rows are dealt out to blocks decides the order of the parameters' gradients.  The gradient in
// bf16 with 640, 1024 and 320 threads: 65.7, 75.9 and 105 us of 40960 x 1024, 65.2, 77.0 and 95.9 of 16384 x 2560, 97.4,
// 100.3 and 97.4 of 16332 x 2568 (one block, two, one), 71.9, 75.1 and 71.9 of 10240 x 4096.  (ln_partials: the most
// blocks of any length on either side of 2560.)
inline int ln_blocks(int D, int most = 640) {
  const int threads = (D / 8 + 31) / 32 * 32;
  return threads > most / 2 ? 1 : most / threads > 8 ? 8 : most / threads;
}

// As many blocks as are resident together, each takes its rows in turn.  The GPU is asked once for each kernel
// and block.
template <auto kKernel>
cudaError_t ln_resident(int threads, int* blocks) {
  static std::atomic<int> known[33];
  int n = known[threads / 32].load(std::memory_order_relaxed);
  if (!n) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kKernel, threads, 0);
    if (e != cudaSuccess) return e;
    if (n < 1) n = 1;
    known[threads / 32].store(n, std::memory_order_relaxed);
  }
  *blocks = n;
  return cudaSuccess;
}
template <auto kKernel>
cudaError_t ln_grid(const LnParams& p, int G, int threads, unsigned* grid) {
  int resident = 0;
  const cudaError_t e = ln_resident<kKernel>(threads, &resident);
  const long long per_block = G ? threads / G : 1, units = (p.rows + per_block - 1) / per_block;
  const long long most = (long long)resident * kSms / p.blocks;
  *grid = (unsigned)((units < most ? units : most) * p.blocks);
  return e;
}

// Many whole rows: a persistent block whose rows arrive by bulk copies in a ring of shared memory, several rows
// ahead.  G threads have 8 columns each of kRows rows at a time, whose sums share their barriers.
constexpr int kLnRingBytes = 208 * 1024, kLnRingSlots = 16;
struct LnRing {
  int slots, slot_bytes, blocks;  // of a block, of a row, of an SM
};
// Rows for which it pays: every block has a few.  With and without the ring in bf16, forward and gradient: 304 x 2560
// 4.3 and 3.8, 8.4 and 8.9 us; 608 x 2560 4.8 and 4.8, 8.9 and 10.9; 1216 x 2560 6.3 and 6.7, 10.4 and 15.0; 304 x 5120 4.8
// and 4.8, 10.9 and 12.5; 1216 x 5120 9.9 and 10.9, 17.6 and 25.3; 8192 x 5120 54.7 and 68.9, 68.0 and 150.  (Forwards
// at some widths the rows in registers are as fast: 40960 x 1024 65 and 56, 20480 x 2048 57 and 57.)
constexpr long long kLnRingRows = 4 * kSms;
template <typename T>
LnRing ln_ring(const LnParams& p, int tensors, int blocks) {
  LnRing r;
  r.slot_bytes = p.D * (int)sizeof(T) * tensors;
  r.blocks = blocks;
  r.slots = kLnRingBytes / r.blocks / r.slot_bytes;  // (two rows at least)
  if (r.slots > 8) r.slots = 8;
  return r;
}
// The ring's barriers and copies, kCount tensors a row.
template <typename T, int kCount>
struct LnFeed {
  const LnParams& p;
  unsigned char* ring;
  uint64_t* full;
  const LnRing shape;
  __device__ __forceinline__ void start() {
    for (int s = 0; s < shape.slots; ++s) mbar_init(&full[s], 1);
    mbar_fence_init();
    for (int s = 0; s < shape.slots; ++s) fetch(blockIdx.x + (long long)s * gridDim.x, s);
  }
  __device__ __forceinline__ void fetch(long long row, int s) {  // one thread: the row's copies into slot s
    if (row >= p.rows) return;
    const int bytes = p.D * (int)sizeof(T);
    unsigned char* dst = ring + s * shape.slot_bytes;
    mbar_expect_tx(&full[s], shape.slot_bytes);
    bulk_g2s(dst, static_cast<const T*>(p.x) + row * p.x_stride, bytes, &full[s]);
    if (kCount == 2) bulk_g2s(dst + bytes, static_cast<const T*>(p.dy) + row * p.dy_stride, bytes, &full[s]);
    if (p.residual)
      bulk_g2s(dst + kCount * bytes, static_cast<const T*>(p.residual) + row * p.D, bytes, &full[s]);
  }
  // after a lost copy: the copies that are still on their way, from `slot` of `phase` on, behind the `rows` rows from `row` on
  __device__ __forceinline__ void drain(long long row, int rows, int slot, unsigned phase) {
    row += (long long)rows * gridDim.x;
    for (int k = rows; k < shape.slots && row < p.rows; ++k, row += gridDim.x) {
      mbar_wait(&full[slot], phase, p.err);
      if (++slot == shape.slots) slot = 0, phase ^= 1;
    }
  }
  __device__ __forceinline__ const T* row_of(int s) const {
    return reinterpret_cast<const T*>(ring + s * shape.slot_bytes);
  }
};

}  // namespace gdn
