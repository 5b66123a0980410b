// layer_norm.cu - layer norm of rows, with the residual's addition.
//
//   r = x + residual,   y = (r - mean(r)) / sqrt(mean((r - mean(r))^2) + eps) w + b
//
// The mean first, then the squares of what differs from it (one pass over x and x^2 would lose rows
// whose mean is large against their spread), from registers: every tensor crosses HBM once, and
// the next row is loaded meanwhile.  All in fp32; r as the new residual and y are rounded once
// each, and the norm sees r before it is rounded.
//
// HBM bandwidth bounds it: 8192 x 5120 in bf16 with a residual takes 58 us, 5.8 TB/s; a row in registers and
// the next one's loads behind it took 102, for want of bytes in flight.
#include "layer_norm.cuh"

namespace gdn {
namespace {

template <typename T, bool kWhole, int G, int NV, int kThreads>
__global__ void __launch_bounds__(kThreads) ln_fwd_kernel(const LnParams p) {
  __shared__ LnShared s;
  __shared__ __align__(16) float scratch[kWhole ? 4 : kThreads * 8];
  const unsigned blocks = G ? 1 : p.blocks, rank = !G && blocks > 1 ? cluster_rank() : 0;
  if (!G && blocks > 1) cluster_arrive();
  const LnColumns<kWhole, G, NV> col(p, rank, scratch);
  const long long per_block = G ? 128 / (G ? G : 1) : 1;
  const long long rows = (long long)(gridDim.x / blocks) * per_block;
  const long long row0 = blockIdx.x / blocks * per_block + (G ? threadIdx.x / (G ? G : 1) : 0);
  f32x2 w[NV][4], b[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[i][j] = dup2(1.f), b[i][j] = 0ull;
    if (p.w) col.vector(col.load(p.w, i), i, w[i]);
    if (p.b) col.vector(col.load(p.b, i), i, b[i]);
  }
  Raw8<T> x[NV], res[NV];
  auto load = [&](long long row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] = col.load(static_cast<const T*>(p.x) + row * p.x_stride, i);
      if (p.residual) res[i] = col.load(static_cast<const T*>(p.residual) + row * p.D, i);
    }
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i].zero(), res[i].zero();
  if (row0 < p.rows) load(row0);
  int turn = 0;
  if (!G && blocks > 1) cluster_wait();
  // every lane of a warp stays for the sums
  for (long long row = row0; row - (G ? threadIdx.x / (G ? G : 1) : 0) < p.rows; row += rows) {
    const bool some = row < p.rows;
    f32x2 r[NV][4];
    float v[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      col.vector(x[i], i, r[i]);
      if (p.residual) {
        f32x2 q[4];
        col.vector(res[i], i, q);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i][j] = add2(r[i][j], q[j]);
        col.store(static_cast<T*>(p.residual_out) + row * p.D, i, r[i], some);
      }
      v[0] += sum8(r[i]);
    }
    if (row + rows < p.rows) load(row + rows);
    sum_row<G>(v, &s, turn, blocks);
    const f32x2 mean = dup2(-v[0] * p.inv_d);
    v[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      f32x2 sum = 0ull;
#pragma unroll
      for (int j = 0; j < 4; ++j) r[i][j] = add2(r[i][j], mean);
      col.mask(r[i], i);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum = fma2(r[i][j], r[i][j], sum);
      v[0] += both(sum);
    }
    sum_row<G>(v, &s, turn, blocks);
    const f32x2 rstd = dup2(rsqrtf(v[0] * p.inv_d + p.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) r[i][j] = fma2(mul2(r[i][j], rstd), w[i][j], b[i][j]);
      col.store(static_cast<T*>(p.y) + row * p.D, i, r[i], some);
    }
  }
}

// Many whole rows, through the ring.
template <typename T, int kRows>
__global__ void __launch_bounds__(1024) ln_fwd_ring_kernel(const LnParams p, const LnRing shape) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ uint64_t full[kLnRingSlots];
  __shared__ int s_lost;
  __shared__ LnShared s;
  LnFeed<T, 1> feed{p, ring, full, shape};
  const int c = threadIdx.x * 8;
  const bool here = c < p.D;
  f32x2 w[4], b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = dup2(1.f), b[j] = 0ull;
  if (here && p.w) pairs_of(load8(p.w + c, 8, 8), w);
  if (here && p.b) pairs_of(load8(p.b + c, 8, 8), b);
  if (threadIdx.x == 0) s_lost = 0, feed.start();
  __syncthreads();
  int slot = 0, turn = 0;
  unsigned phase = 0;
  for (long long row = blockIdx.x; row < p.rows; row += (long long)kRows * gridDim.x) {
    f32x2 r[kRows][4];
    float v[kRows];
    int from[kRows];
    bool lost = false;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const long long at = row + (long long)k * gridDim.x;
      v[k] = 0.f;
      from[k] = slot;
#pragma unroll
      for (int j = 0; j < 4; ++j) r[k][j] = 0ull;
      if (at >= p.rows) continue;
      lost = lost || !mbar_wait(&full[slot], phase, p.err);
      if (here) {
        const T* in = feed.row_of(slot) + c;
        Raw8<T> x;
        x.load(in);
        pairs_of(x, r[k]);
        if (p.residual) {
          f32x2 q[4];
          x.load(in + p.D);
          pairs_of(x, q);
#pragma unroll
          for (int j = 0; j < 4; ++j) r[k][j] = add2(r[k][j], q[j]);
          raw_of<T>(r[k]).store(static_cast<T*>(p.residual_out) + at * p.D + c);
        }
        v[k] = sum8(r[k]);
      }
      if (++slot == shape.slots) slot = 0, phase ^= 1;
    }
    if (lost) s_lost = 1;
    sum_block(v, &s, turn);
    // a copy that does not arrive within about a second is recorded, and ends the block's work (the sum's
    // barrier tells all threads) once the other copies in flight have arrived
    if (s_lost) {
      feed.drain(row, kRows, slot, phase);
      return;
    }
    if (threadIdx.x == 0) {  // every thread has read the slots
      fence_proxy_async();
#pragma unroll
      for (int k = 0; k < kRows; ++k) feed.fetch(row + ((long long)k + shape.slots) * gridDim.x, from[k]);
    }
    float q[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const f32x2 mean = dup2(-v[k] * p.inv_d);
      f32x2 sum = 0ull;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[k][j] = add2(r[k][j], mean);
        sum = fma2(r[k][j], r[k][j], sum);
      }
      q[k] = here ? both(sum) : 0.f;
    }
    sum_block(q, &s, turn);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const long long at = row + (long long)k * gridDim.x;
      if (at >= p.rows || !here) continue;
      const f32x2 rstd = dup2(rsqrtf(q[k] * p.inv_d + p.eps));
#pragma unroll
      for (int j = 0; j < 4; ++j) r[k][j] = fma2(mul2(r[k][j], rstd), w[j], b[j]);
      raw_of<T>(r[k]).store(static_cast<T*>(p.y) + at * p.D + c);
    }
  }
}

template <typename T, bool kWhole, int G, int NV, int kThreads = 128>
cudaError_t launch(const LnParams& p, cudaStream_t stream) {
  const int threads = G ? 128 : ((p.slice + 8 * NV - 1) / (8 * NV) + 31) / 32 * 32;
  unsigned grid;
  const cudaError_t e = ln_grid<ln_fwd_kernel<T, kWhole, G, NV, kThreads>>(p, G, threads, &grid);
  return e == cudaSuccess ? launch_clusters(ln_fwd_kernel<T, kWhole, G, NV, kThreads>, grid, threads, p.blocks, p, stream) : e;
}
template <typename T, int kRows>
cudaError_t launch_ring(LnParams p, const LnRing& shape, cudaStream_t stream) {
  const auto kernel = ln_fwd_ring_kernel<T, kRows>;
  const int threads = (p.D / 8 + 31) / 32 * 32, smem = shape.slots * shape.slot_bytes;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLnRingBytes);
  if (e == cudaSuccess) e = device_error_word(&p.err);
  if (e != cudaSuccess) return e;
  const long long most = (long long)shape.blocks * kSms;
  kernel<<<(unsigned)(p.rows < most ? p.rows : most), threads, smem, stream>>>(p, shape);
  return cudaGetLastError();
}
template <typename T, bool kWhole>
cudaError_t launch_t(const LnParams& p, cudaStream_t stream) {
  if (p.D <= 64) return launch<T, kWhole, 8, 1>(p, stream);
  if (p.D <= 128) return launch<T, kWhole, 16, 1>(p, stream);
  if (p.D <= 256) return launch<T, kWhole, 32, 1>(p, stream);
  if (p.D <= 512) return launch<T, kWhole, 32, 2>(p, stream);
  if (kWhole && p.blocks == 1 && p.rows >= kLnRingRows) {
    // Two blocks an SM up to 704 threads together in bf16, 640 in fp32, whose rows leave the ring fewer places: 16332 x
    // 2568 takes 56 us in bf16 with two and 82 with one, 14894 x 2816 64 and 75, 8166 x 2568 in fp32 62 and 56.
    const LnRing shape = ln_ring<T>(p, p.residual ? 2 : 1, ln_blocks(p.D, sizeof(T) == 2 ? 704 : 640));
    // Two rows a sum where two more are on their way meanwhile.  Two and one in bf16: 64 and 73 us of 65536 x 640, 57
    // and 67 of 20480 x 2048, 55 and 62 of 8192 x 5120; 65 and 59 of 40960 x 1024, 64 and 58 of 6826 x 6144.
    if (shape.slots >= 4) return launch_ring<T, 2>(p, shape, stream);
    return launch_ring<T, 1>(p, shape, stream);
  }
  if (p.slice <= 8 * 512) return launch<T, kWhole, 0, 1, 512>(p, stream);
  return launch<T, kWhole, 0, 1, kLnMaxThreads>(p, stream);
}

}  // namespace

cudaError_t launch_layer_norm(const LnParams& p, bool f32, cudaStream_t stream) {
  if (f32) return p.whole ? launch_t<float, true>(p, stream) : launch_t<float, false>(p, stream);
  return p.whole ? launch_t<__nv_bfloat16, true>(p, stream) : launch_t<__nv_bfloat16, false>(p, stream);
}

}  // namespace gdn
