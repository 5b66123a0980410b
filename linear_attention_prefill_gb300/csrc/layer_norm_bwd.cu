// layer_norm_bwd.cu - the gradient of layer norm.
//
//   xh = (x - mean) rstd,  u = dy w:   dx = rstd (u - mean(u) - xh mean(u xh)) + dres,
//   dw = sum over rows of dy xh,   db = sum over rows of dy
//
// Mean and rstd are taken from x again: the row is in registers for the gradient anyway, and a sum
// more costs no traffic.  A block keeps its columns for all its rows, so dw and db grow in its
// registers (fp32) over the rows that it walks; each block leaves one partial sum, which a second
// launch adds up in a fixed order.
//
// 8192 x 5120 in bf16 with dres takes 70 us, 4.8 TB/s, 9 of them for dw and db: memory and issue (59 % of its
// slots) bound it together.
#include "layer_norm.cuh"

namespace gdn {
namespace {

template <typename T, bool kWhole, int G, int NV, bool kParams, int kThreads>
__global__ void __launch_bounds__(kThreads, 1) ln_bwd_kernel(const LnParams p) {
  __shared__ LnShared s;
  __shared__ __align__(16) float scratch[kWhole && !(kParams && G) ? 4 : kThreads * 8];
  const unsigned blocks = G ? 1 : p.blocks, rank = !G && blocks > 1 ? cluster_rank() : 0;
  if (!G && blocks > 1) cluster_arrive();
  const LnColumns<kWhole, G, NV> col(p, rank, scratch);
  const long long per_block = G ? 128 / (G ? G : 1) : 1;
  const long long rows = (long long)(gridDim.x / blocks) * per_block;
  const long long row0 = blockIdx.x / blocks * per_block + (G ? threadIdx.x / (G ? G : 1) : 0);
  f32x2 w[NV][4], dw[NV][4], db[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[i][j] = dup2(1.f), dw[i][j] = db[i][j] = 0ull;
    if (p.w) col.vector(col.load(p.w, i), i, w[i]);
  }
  Raw8<T> x[NV], dy[NV], res[NV];
  auto load = [&](long long row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] = col.load(static_cast<const T*>(p.x) + row * p.x_stride, i);
      dy[i] = col.load(static_cast<const T*>(p.dy) + row * p.dy_stride, i);
      if (p.residual) res[i] = col.load(static_cast<const T*>(p.residual) + row * p.D, i);
    }
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i].zero(), dy[i].zero(), res[i].zero();
  if (row0 < p.rows) load(row0);
  int turn = 0;
  if (!G && blocks > 1) cluster_wait();
  // every lane of a warp stays for the sums
  for (long long row = row0; row - (G ? threadIdx.x / (G ? G : 1) : 0) < p.rows; row += rows) {
    const bool some = row < p.rows;
    f32x2 r[NV][4], u[NV][4];
    Raw8<T> extra[NV];
    float m[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      col.vector(x[i], i, r[i]);
      col.vector(dy[i], i, u[i]);
      extra[i] = res[i];
      m[0] += sum8(r[i]);
    }
    if (row + rows < p.rows) load(row + rows);
    sum_row<G>(m, &s, turn, blocks);
    const f32x2 mean = dup2(-m[0] * p.inv_d);
    float v[4] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      f32x2 ss = 0ull, su = 0ull, sx = 0ull;
#pragma unroll
      for (int j = 0; j < 4; ++j) r[i][j] = add2(r[i][j], mean);
      col.mask(r[i], i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 uw = mul2(u[i][j], w[i][j]);
        ss = fma2(r[i][j], r[i][j], ss);
        su = fma2(u[i][j], w[i][j], su);
        sx = fma2(uw, r[i][j], sx);
      }
      v[0] += both(ss), v[1] += both(su), v[2] += both(sx);
    }
    sum_row<G>(v, &s, turn, blocks);
    const float rs = rsqrtf(v[0] * p.inv_d + p.eps);
    const f32x2 rstd = dup2(rs), c1 = dup2(-v[1] * p.inv_d), c2 = dup2(-v[2] * p.inv_d * rs);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      f32x2 d[4];
      if (p.residual) {
        col.vector(extra[i], i, d);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = 0ull;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 xh = mul2(r[i][j], rstd);
        if (kParams && some) {
          dw[i][j] = fma2(u[i][j], xh, dw[i][j]);
          db[i][j] = add2(db[i][j], u[i][j]);
        }
        d[j] = fma2(rstd, fma2(xh, c2, fma2(u[i][j], w[i][j], c1)), d[j]);
      }
      col.store(static_cast<T*>(p.y) + row * p.D, i, d, some);
    }
  }
  if (kParams) griddep_launch_dependents();
  if constexpr (kParams && G == 0) {  // [blocks, 2, D]
    float* out = p.partial + (long long)(blockIdx.x / blocks) * 2 * p.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      col.store(out, i, dw[i], true);
      col.store(out + p.D, i, db[i], true);
    }
  }
  if constexpr (kParams && G > 0) {  // the block's rows in order: G lanes of each have the same columns
#pragma unroll
    for (int k = 0; k < 2 * NV; ++k) {
      __syncthreads();
      raw_of<float>(k & 1 ? db[k / 2] : dw[k / 2]).store(scratch + threadIdx.x * 8);
      __syncthreads();
      for (int c = threadIdx.x; c < G * 8; c += 128) {
        float sum = 0.f;
        for (int q = 0; q < 128 / G; ++q) sum += scratch[q * G * 8 + c];
        const int at = k / 2 * G * 8 + c;
        if (at < p.D) p.partial[((long long)blockIdx.x * 2 + (k & 1)) * p.D + at] = sum;
      }
    }
  }
}

// Many whole rows, through the ring: two at a time, whose sums share their barriers.
template <typename T, int kRows, bool kParams, int kThreads>
__global__ void __launch_bounds__(kThreads) ln_bwd_ring_kernel(const LnParams p, const LnRing shape) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ uint64_t full[kLnRingSlots];
  __shared__ int s_lost;
  __shared__ LnShared s;
  LnFeed<T, 2> feed{p, ring, full, shape};
  const int c = threadIdx.x * 8;
  const bool here = c < p.D;
  f32x2 w[4], dw[4], db[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = dup2(1.f), dw[j] = db[j] = 0ull;
  if (here && p.w) pairs_of(load8(p.w + c, 8, 8), w);
  if (threadIdx.x == 0) s_lost = 0, feed.start();
  __syncthreads();
  int slot = 0, turn = 0;
  unsigned phase = 0;
  for (long long row = blockIdx.x; row < p.rows; row += (long long)kRows * gridDim.x) {
    f32x2 r[kRows][4], u[kRows][4];
    Raw8<T> extra[kRows];
    float v[kRows];
    int from[kRows];
    bool lost = false;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      v[k] = 0.f;
      from[k] = slot;
#pragma unroll
      for (int j = 0; j < 4; ++j) r[k][j] = u[k][j] = 0ull;
      if (row + (long long)k * gridDim.x >= p.rows) continue;
      lost = lost || !mbar_wait(&full[slot], phase, p.err);
      if (here) {
        const T* in = feed.row_of(slot) + c;
        Raw8<T> x;
        x.load(in);
        pairs_of(x, r[k]);
        x.load(in + p.D);
        pairs_of(x, u[k]);
        if (p.residual) extra[k].load(in + 2 * p.D);
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
      break;
    }
    if (threadIdx.x == 0) {  // every thread has read the slots
      fence_proxy_async();
#pragma unroll
      for (int k = 0; k < kRows; ++k) feed.fetch(row + ((long long)k + shape.slots) * gridDim.x, from[k]);
    }
    constexpr int kSums = kRows == 2 ? 8 : 4;
    float q[kSums] = {};
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const f32x2 mean = dup2(-v[k] * p.inv_d);
      f32x2 ss = 0ull, su = 0ull, sx = 0ull;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[k][j] = add2(r[k][j], mean);
        const f32x2 uw = mul2(u[k][j], w[j]);
        ss = fma2(r[k][j], r[k][j], ss);
        su = fma2(u[k][j], w[j], su);
        sx = fma2(uw, r[k][j], sx);
      }
      if (here) q[4 * k] = both(ss), q[4 * k + 1] = both(su), q[4 * k + 2] = both(sx);
    }
    sum_block(q, &s, turn);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const long long at = row + (long long)k * gridDim.x;
      if (at >= p.rows || !here) continue;
      const float rs = rsqrtf(q[4 * k] * p.inv_d + p.eps);
      const f32x2 rstd = dup2(rs), c1 = dup2(-q[4 * k + 1] * p.inv_d), c2 = dup2(-q[4 * k + 2] * p.inv_d * rs);
      f32x2 d[4];
      if (p.residual) {
        pairs_of(extra[k], d);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = 0ull;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 xh = mul2(r[k][j], rstd);
        if (kParams) {
          dw[j] = fma2(u[k][j], xh, dw[j]);
          db[j] = add2(db[j], u[k][j]);
        }
        d[j] = fma2(rstd, fma2(xh, c2, fma2(u[k][j], w[j], c1)), d[j]);
      }
      raw_of<T>(d).store(static_cast<T*>(p.y) + at * p.D + c);
    }
  }
  if (kParams) {
    griddep_launch_dependents();
    if (here) {
      float* out = p.partial + (long long)blockIdx.x * 2 * p.D + c;
      raw_of<float>(dw).store(out);
      raw_of<float>(db).store(out + p.D);
    }
  }
}

template <typename T, bool kWhole, int G, int NV, bool kParams, int kThreads = 128>
cudaError_t launch(const LnParams& p, cudaStream_t stream) {
  const int threads = G ? 128 : ((p.slice + 8 * NV - 1) / (8 * NV) + 31) / 32 * 32;
  unsigned grid;
  cudaError_t e = ln_grid<ln_bwd_kernel<T, kWhole, G, NV, kParams, kThreads>>(p, G, threads, &grid);
  if (e != cudaSuccess) return e;
  if (kParams) {  // (by the sizes alone)
    const long long per_block = G ? 128 / (G ? G : 1) : 1, units = (p.rows + per_block - 1) / per_block;
    const long long most = (long long)kSms * (G ? 8 : ln_blocks(p.D)) / p.blocks;
    grid = (unsigned)((units < most ? units : most) * p.blocks);
  }
  if (p.rows) e = launch_clusters(ln_bwd_kernel<T, kWhole, G, NV, kParams, kThreads>, grid, threads, p.blocks, p, stream);
  if (e != cudaSuccess || !kParams) return e;
  return launch_column_sums(p.partial, p.dw, p.db, (int)(grid / p.blocks), p.D, stream);
}
template <typename T, int kRows, bool kParams, int kThreads>
cudaError_t launch_ring(LnParams p, const LnRing& shape, cudaStream_t stream) {
  const auto kernel = ln_bwd_ring_kernel<T, kRows, kParams, kThreads>;
  const int threads = (p.D / 8 + 31) / 32 * 32, smem = shape.slots * shape.slot_bytes;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLnRingBytes);
  if (e == cudaSuccess) e = device_error_word(&p.err);
  if (e != cudaSuccess) return e;
  const long long most = (long long)shape.blocks * kSms;
  const unsigned grid = (unsigned)(p.rows < most ? p.rows : most);
  kernel<<<grid, threads, smem, stream>>>(p, shape);
  e = cudaGetLastError();
  if (e != cudaSuccess || !kParams) return e;
  return launch_column_sums(p.partial, p.dw, p.db, (int)grid, p.D, stream);
}
template <typename T, bool kWhole, bool kParams>
cudaError_t launch_t(const LnParams& p, cudaStream_t stream) {
  if (p.D <= 64) return launch<T, kWhole, 8, 1, kParams>(p, stream);
  if (p.D <= 128) return launch<T, kWhole, 16, 1, kParams>(p, stream);
  if (p.D <= 256) return launch<T, kWhole, 32, 1, kParams>(p, stream);
  if (p.D <= 512) return launch<T, kWhole, 32, 2, kParams>(p, stream);
  if (kWhole && p.blocks == 1 && p.rows >= kLnRingRows) {
    const LnRing shape = ln_ring<T>(p, p.residual ? 3 : 2, ln_blocks(p.D));
    // Two rows take 90 registers, which 640 threads have; 704 have 80 (8192 x 5120 compiled so takes 76 us for 68), wider
    // rows fewer.  Two and one in bf16: 65 and 77 us of 16384 x 2560, 68 and 82 of 8192 x 5120, 81 and 87 of 8179 x 5128,
    // 79 and 81 of 7447 x 5632.
    if (shape.slots >= 4 && p.D <= 8 * 640) return launch_ring<T, 2, kParams, 640>(p, shape, stream);
    if (shape.slots >= 4 && p.D <= 8 * 704) return launch_ring<T, 2, kParams, 704>(p, shape, stream);
    return launch_ring<T, 1, kParams, 1024>(p, shape, stream);
  }
  if (p.slice <= 8 * 512) return launch<T, kWhole, 0, 1, kParams, 512>(p, stream);
  return launch<T, kWhole, 0, 1, kParams, kLnMaxThreads>(p, stream);
}
template <typename T>
cudaError_t launch_type(const LnParams& p, cudaStream_t stream) {
  if (p.dw) return p.whole ? launch_t<T, true, true>(p, stream) : launch_t<T, false, true>(p, stream);
  return p.whole ? launch_t<T, true, false>(p, stream) : launch_t<T, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_layer_norm_bwd(const LnParams& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_type<float>(p, stream) : launch_type<__nv_bfloat16>(p, stream);
}

}  // namespace gdn
