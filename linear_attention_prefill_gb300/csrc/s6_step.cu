// s6_step.cu - one token of the S6 recurrence per sequence (the decode step of s6_scan.cuh).
//
// A lane takes four states of one channel for kSeqs sequences at once: reads them, writes
// them back; the LPC lanes of a channel add their parts of y by shuffles.  The states are read
// and written once, 128 bytes a channel at Ns = 16, and HBM bandwidth bounds it: four
// sequences a lane keep enough reads in flight and share A (one sequence measured 2.6 TB/s);
// few sequences take one, and launch latency is all there is.
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {
namespace {

template <typename T, int LPC, int kSeqs>
__global__ void __launch_bounds__(256) s6_step_kernel(const S6Params p, int per_row) {
  const int bx = blockIdx.x % per_row;
  const int first = blockIdx.x / per_row * kSeqs;
  const int id = bx * 256 + threadIdx.x;
  const bool some = id / LPC < p.dim;  // lanes behind the last channel only join the shuffles
  const int ch = some ? id / LPC : p.dim - 1, n0 = id % LPC * 4;
  const int nst = some ? max(0, min(4, p.Ns - n0)) : 0;
  const long long hrow = (long long)ch * p.Ns + n0, hsize = (long long)p.dim * p.Ns;
  float4 h[kSeqs], b[kSeqs], c[kSeqs];
  float x[kSeqs], d[kSeqs], z[kSeqs];
  const float4 a = load_h(p.A + hrow, nst, p.Ns);
#pragma unroll
  for (int i = 0; i < kSeqs; ++i) {
    const long long n = first + i < p.N ? first + i : p.N - 1;
    h[i] = load_h(p.hT + n * hsize + hrow, nst, p.Ns);
    x[i] = to_f32(static_cast<const T*>(p.x)[n * p.x_stride + ch]);
    d[i] = to_f32(static_cast<const T*>(p.dt)[n * p.dt_stride + ch]);
    z[i] = p.z ? to_f32(static_cast<const T*>(p.z)[n * p.z_stride + ch]) : 0.f;
    Raw4<T> rb, rc;
    rb.zero();
    rc.zero();
    if (nst > 0) {
      rb.load(static_cast<const T*>(p.B) + n * p.b_stride + n0, nst, p.vec_bc);
      rc.load(static_cast<const T*>(p.C) + n * p.c_stride + n0, nst, p.vec_bc);
    }
    b[i] = rb.get();
    c[i] = rc.get();
  }
  const float bias = p.dt_bias ? p.dt_bias[ch] : 0.f, skip = p.D ? p.D[ch] : 0.f;
#pragma unroll
  for (int i = 0; i < kSeqs; ++i) {
    const int n = first + i;
    const float dl = p.softplus ? softplus(d[i] + bias) : d[i] + bias;
    const float u = dl * x[i];
    float4 o;
    o.x = fmaf(ex2(dl * (a.x * kLog2e)), h[i].x, u * b[i].x);
    o.y = fmaf(ex2(dl * (a.y * kLog2e)), h[i].y, u * b[i].y);
    o.z = fmaf(ex2(dl * (a.z * kLog2e)), h[i].z, u * b[i].z);
    o.w = fmaf(ex2(dl * (a.w * kLog2e)), h[i].w, u * b[i].w);
    if (n < p.N) store_h(p.hT + n * hsize + hrow, o, nst, p.Ns);
    float y = 0.f;  // only of states that exist
    if (nst > 0) y = c[i].x * o.x;
    if (nst > 1) y = fmaf(c[i].y, o.y, y);
    if (nst > 2) y = fmaf(c[i].z, o.z, y);
    if (nst > 3) y = fmaf(c[i].w, o.w, y);
#pragma unroll
    for (int off = LPC / 2; off > 0; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
    if (some && n < p.N && id % LPC == 0) {
      if (p.D) y = fmaf(skip, x[i], y);
      if (p.z) y *= silu(z[i]);
      from_f32(static_cast<T*>(p.y) + (long long)n * p.dim + ch, y);
    }
  }
}

template <typename T, int LPC>
cudaError_t launch_step_l(const S6Params& p, cudaStream_t stream) {
  const int per_row = (int)(((long long)p.dim * LPC + 255) / 256);
  // four sequences a lane once that still leaves two blocks per SM
  if ((long long)per_row * p.N >= 8 * kSms)
    s6_step_kernel<T, LPC, 4>
        <<<(unsigned)((long long)per_row * ((p.N + 3) / 4)), 256, 0, stream>>>(p, per_row);
  else
    s6_step_kernel<T, LPC, 1><<<(unsigned)((long long)per_row * p.N), 256, 0, stream>>>(p, per_row);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_step_t(const S6Params& p, cudaStream_t stream) {
  if (p.Ns <= 4) return launch_step_l<T, 1>(p, stream);
  if (p.Ns <= 8) return launch_step_l<T, 2>(p, stream);
  if (p.Ns <= 16) return launch_step_l<T, 4>(p, stream);
  if (p.Ns <= 32) return launch_step_l<T, 8>(p, stream);
  return launch_step_l<T, 16>(p, stream);
}

}  // namespace

cudaError_t launch_s6_step(const S6Params& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_step_t<float>(p, stream) : launch_step_t<__nv_bfloat16>(p, stream);
}

}  // namespace gdn
