// layer_norm.cu - layer norm of rows, with the residual's addition.
//
//   r = x + residual,   y = (r - mean(r)) / sqrt(mean((r - mean(r))^2) + eps) w + b
//
// The mean first, then the squares of what differs from it (one pass over x and x^2 would lose rows
// whose mean is large against their spread), from registers: every tensor crosses HBM once, and
// the next row is loaded meanwhile.  All in fp32; r as the new residual and y are rounded once
// each, and the norm sees r before it is rounded.
#include "layer_norm.cuh"

namespace gdn {
namespace {

template <typename T, bool kWhole, int G, int NV>
__global__ void __launch_bounds__(G ? 128 : kLnMaxThreads) ln_fwd_kernel(const LnParams p) {
  __shared__ LnShared s;
  const unsigned blocks = G ? 1 : p.blocks, rank = !G && blocks > 1 ? cluster_rank() : 0;
  if (!G && blocks > 1) cluster_arrive();
  const LnColumns<G, NV> col(p, rank);
  const int by = kWhole ? 8 : p.by, step = LnColumns<G, NV>::step() * 8;
  const long long per_block = G ? 128 / (G ? G : 1) : 1;
  const long long rows = (long long)(gridDim.x / blocks) * per_block;
  const long long row0 = blockIdx.x / blocks * per_block + (G ? threadIdx.x / (G ? G : 1) : 0);
  f32x2 w[NV][4], b[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[i][j] = dup2(1.f), b[i][j] = 0ull;
    if (col.n[i] <= 0) continue;
    if (p.w) pairs_of(load8(p.w + col.first + i * step, col.n[i], by), w[i]);
    if (p.b) pairs_of(load8(p.b + col.first + i * step, col.n[i], by), b[i]);
  }
  Raw8<T> x[NV], res[NV];
  auto load = [&](long long row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (col.n[i] <= 0) continue;
      x[i] = load8(static_cast<const T*>(p.x) + row * p.x_stride + col.first + i * step, col.n[i], by);
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
    f32x2 r[NV][4], sum = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!some || col.n[i] <= 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i][j] = 0ull;
        continue;
      }
      pairs_of(x[i], r[i]);
      if (p.residual) {
        f32x2 q[4];
        pairs_of(res[i], q);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i][j] = add2(r[i][j], q[j]);
        store8(static_cast<T*>(p.residual_out) + row * p.D + col.first + i * step, raw_of<T>(r[i]), col.n[i], by);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sum = add2(sum, r[i][j]);
    }
    if (row + rows < p.rows) load(row + rows);
    float v[1] = {both(sum)};
    sum_row<G>(v, &s, turn, blocks);
    const f32x2 mean = dup2(-v[0] * p.inv_d);
    sum = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!some || col.n[i] <= 0) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) r[i][j] = add2(r[i][j], mean);
      mask<kWhole>(r[i], col.n[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum = fma2(r[i][j], r[i][j], sum);
    }
    v[0] = both(sum);
    sum_row<G>(v, &s, turn, blocks);
    const f32x2 rstd = dup2(rsqrtf(v[0] * p.inv_d + p.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!some || col.n[i] <= 0) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) r[i][j] = fma2(mul2(r[i][j], rstd), w[i][j], b[i][j]);
      store8(static_cast<T*>(p.y) + row * p.D + col.first + i * step, raw_of<T>(r[i]), col.n[i], by);
    }
  }
}

template <typename T, bool kWhole, int G, int NV>
cudaError_t launch(const LnParams& p, cudaStream_t stream) {
  const int threads = G ? 128 : ((p.slice + 8 * NV - 1) / (8 * NV) + 31) / 32 * 32;
  unsigned grid;
  const auto kernel = ln_fwd_kernel<T, kWhole, G, NV>;
  const cudaError_t e = ln_grid(kernel, p, G, threads, &grid);
  return e == cudaSuccess ? launch_clusters(kernel, grid, threads, p.blocks, p, stream) : e;
}
template <typename T, bool kWhole>
cudaError_t launch_t(const LnParams& p, cudaStream_t stream) {
  if (p.D <= 64) return launch<T, kWhole, 8, 1>(p, stream);
  if (p.D <= 128) return launch<T, kWhole, 16, 1>(p, stream);
  if (p.D <= 256) return launch<T, kWhole, 32, 1>(p, stream);
  if (p.D <= 512) return launch<T, kWhole, 32, 2>(p, stream);
  return p.slice <= 8 * kLnMaxThreads ? launch<T, kWhole, 0, 1>(p, stream) : launch<T, kWhole, 0, 2>(p, stream);
}

}  // namespace

cudaError_t launch_layer_norm(const LnParams& p, bool f32, cudaStream_t stream) {
  if (f32) return p.by == 8 ? launch_t<float, true>(p, stream) : launch_t<float, false>(p, stream);
  return p.by == 8 ? launch_t<__nv_bfloat16, true>(p, stream) : launch_t<__nv_bfloat16, false>(p, stream);
}

}  // namespace gdn
