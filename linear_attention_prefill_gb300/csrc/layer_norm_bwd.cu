// layer_norm_bwd.cu - the gradient of layer norm.
//
//   xh = (x - mean) rstd,  u = dy w:   dx = rstd (u - mean(u) - xh mean(u xh)) + dres,
//   dw = sum over rows of dy xh,   db = sum over rows of dy
//
// Mean and rstd are taken from x again: the row is in registers for the gradient anyway, and a sum
// more costs no traffic.  A block keeps its columns for all its rows, so dw and db grow in its
// registers (fp32) over the rows that it walks; each block leaves one partial sum, which a second
// launch adds up in a fixed order.
#include "layer_norm.cuh"

namespace gdn {
namespace {

template <typename T, bool kWhole, int G, int NV, bool kParams>
__global__ void __launch_bounds__(G ? 128 : kLnMaxThreads, 1) ln_bwd_kernel(const LnParams p) {
  __shared__ LnShared s;
  const unsigned blocks = G ? 1 : p.blocks, rank = !G && blocks > 1 ? cluster_rank() : 0;
  if (!G && blocks > 1) cluster_arrive();
  const LnColumns<G, NV> col(p, rank);
  const int by = kWhole ? 8 : p.by, step = LnColumns<G, NV>::step() * 8;
  const long long per_block = G ? 128 / (G ? G : 1) : 1;
  const long long rows = (long long)(gridDim.x / blocks) * per_block;
  const long long row0 = blockIdx.x / blocks * per_block + (G ? threadIdx.x / (G ? G : 1) : 0);
  f32x2 w[NV][4], dw[NV][4], db[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[i][j] = dup2(1.f), dw[i][j] = db[i][j] = 0ull;
    if (col.n[i] > 0 && p.w) pairs_of(load8(p.w + col.first + i * step, col.n[i], by), w[i]);
  }
  Raw8<T> x[NV], dy[NV], res[NV];
  auto load = [&](long long row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (col.n[i] <= 0) continue;
      x[i] = load8(static_cast<const T*>(p.x) + row * p.x_stride + col.first + i * step, col.n[i], by);
      dy[i] = load8(static_cast<const T*>(p.dy) + row * p.dy_stride + col.first + i * step, col.n[i], by);
      if (p.residual)
        res[i] = load8(static_cast<const T*>(p.residual) + row * p.D + col.first + i * step, col.n[i], by);
    }
  };
  if (row0 < p.rows) load(row0);
  int turn = 0;
  if (!G && blocks > 1) cluster_wait();
  // every lane of a warp stays for the sums
  for (long long row = row0; row - (G ? threadIdx.x / (G ? G : 1) : 0) < p.rows; row += rows) {
    const bool some = row < p.rows;
    f32x2 r[NV][4], u[NV][4], sum = 0ull;
    Raw8<T> extra[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) r[i][j] = u[i][j] = 0ull;
      if (!some || col.n[i] <= 0) continue;
      pairs_of(x[i], r[i]);
      pairs_of(dy[i], u[i]);
      if (p.residual) extra[i] = res[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) sum = add2(sum, r[i][j]);
    }
    if (row + rows < p.rows) load(row + rows);
    float m[1] = {both(sum)};
    sum_row<G>(m, &s, turn, blocks);
    const f32x2 mean = dup2(-m[0] * p.inv_d);
    f32x2 ss = 0ull, su = 0ull, sx = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!some || col.n[i] <= 0) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) r[i][j] = add2(r[i][j], mean);
      mask<kWhole>(r[i], col.n[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 uw = mul2(u[i][j], w[i][j]);
        ss = fma2(r[i][j], r[i][j], ss);
        su = add2(su, uw);
        sx = fma2(uw, r[i][j], sx);
      }
    }
    float v[3] = {both(ss), both(su), both(sx)};
    sum_row<G>(v, &s, turn, blocks);
    const float rs = rsqrtf(v[0] * p.inv_d + p.eps);
    const f32x2 rstd = dup2(rs), c1 = dup2(-v[1] * p.inv_d), c2 = dup2(-v[2] * p.inv_d * rs);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!some || col.n[i] <= 0) continue;
      f32x2 d[4];
      if (p.residual) {
        pairs_of(extra[i], d);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = 0ull;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 xh = mul2(r[i][j], rstd);
        if (kParams) {
          dw[i][j] = fma2(u[i][j], xh, dw[i][j]);
          db[i][j] = add2(db[i][j], u[i][j]);
        }
        d[j] = fma2(rstd, fma2(xh, c2, fma2(u[i][j], w[i][j], c1)), d[j]);
      }
      store8(static_cast<T*>(p.y) + row * p.D + col.first + i * step, raw_of<T>(d), col.n[i], by);
    }
  }
  if constexpr (kParams && G == 0) {  // [blocks, 2, D]
    float* out = p.partial + (long long)(blockIdx.x / blocks) * 2 * p.D + col.first;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (col.n[i] <= 0) continue;
      const Raw8<float> a = raw_of<float>(dw[i]), c = raw_of<float>(db[i]);
      if (kWhole) {
        a.store(out + i * step);
        c.store(out + p.D + i * step);
      } else {
        a.store_n(out + i * step, col.n[i]);
        c.store_n(out + p.D + i * step, col.n[i]);
      }
    }
  }
  if constexpr (kParams && G > 0) {  // the block's rows in order: G lanes of each have the same columns
    __shared__ float s_sum[128 * 8];
#pragma unroll
    for (int k = 0; k < 2 * NV; ++k) {
      float o[8];
      raw_of<float>(k & 1 ? db[k / 2] : dw[k / 2]).get(o);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) s_sum[threadIdx.x * 8 + j] = o[j];
      __syncthreads();
      for (int c = threadIdx.x; c < G * 8; c += 128) {
        float sum = 0.f;
        for (int q = 0; q < 128 / G; ++q) sum += s_sum[q * G * 8 + c];
        const int at = k / 2 * G * 8 + c;
        if (at < p.D) p.partial[((long long)blockIdx.x * 2 + (k & 1)) * p.D + at] = sum;
      }
    }
  }
}

template <typename T, bool kWhole, int G, int NV, bool kParams>
cudaError_t launch(const LnParams& p, cudaStream_t stream) {
  const int threads = G ? 128 : ((p.slice + 8 * NV - 1) / (8 * NV) + 31) / 32 * 32;
  unsigned grid;
  const auto kernel = ln_bwd_kernel<T, kWhole, G, NV, kParams>;
  cudaError_t e = ln_grid(kernel, p, G, threads, &grid);
  if (e != cudaSuccess) return e;
  if (kParams && grid / p.blocks > (unsigned)ln_partials(p.D)) grid = ln_partials(p.D) * p.blocks;
  if (p.rows) e = launch_clusters(kernel, grid, threads, p.blocks, p, stream);
  if (e != cudaSuccess || !kParams) return e;
  return launch_column_sums(p.partial, p.dw, p.db, (int)(grid / p.blocks), p.D, stream);
}
template <typename T, bool kWhole, bool kParams>
cudaError_t launch_t(const LnParams& p, cudaStream_t stream) {
  if (p.D <= 64) return launch<T, kWhole, 8, 1, kParams>(p, stream);
  if (p.D <= 128) return launch<T, kWhole, 16, 1, kParams>(p, stream);
  if (p.D <= 256) return launch<T, kWhole, 32, 1, kParams>(p, stream);
  if (p.D <= 512) return launch<T, kWhole, 32, 2, kParams>(p, stream);
  return p.slice <= 8 * kLnMaxThreads ? launch<T, kWhole, 0, 1, kParams>(p, stream)
                                      : launch<T, kWhole, 0, 2, kParams>(p, stream);
}
template <typename T>
cudaError_t launch_type(const LnParams& p, cudaStream_t stream) {
  if (p.dw) return p.by == 8 ? launch_t<T, true, true>(p, stream) : launch_t<T, false, true>(p, stream);
  return p.by == 8 ? launch_t<T, true, false>(p, stream) : launch_t<T, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_layer_norm_bwd(const LnParams& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_type<float>(p, stream) : launch_type<__nv_bfloat16>(p, stream);
}

}  // namespace gdn
