// rms_norm.cu - RMS norm of rows: before a layer's projections (with the residual's addition,
// into 16 bits or e4m3 with scales), and of each head after a forward (with its gate).
//
//   r = x + residual,   y = r / sqrt(mean(r^2) + eps) w silu(gate),
//   e4m3: scale = max|y| / 448 over each group of columns (at least 2^-126; 1 for a group of
//   zeros), q = y / scale rounded to nearest even.
//
// r is added, normed and quantised in fp32; it is rounded once to be stored as the new
// residual, and y once on the way out.  HBM bandwidth bounds it: every tensor crosses once,
// with the row held in registers between the sum of squares and the output.  A thread
// holds vectors of 8 columns, so a group of 32, 64 or 128 columns is 4, 8 or 16 lanes.
#include <cuda_fp8.h>

#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {
namespace {

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Four e4m3 of y * inv, saturating.
__device__ __forceinline__ uint32_t e4m3x4(const float* y, float inv) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[1] * inv), "f"(y[0] * inv));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[3] * inv), "f"(y[2] * inv));
  return lo | ((uint32_t)hi << 16);
}

// Sum or maximum over the G threads of a row: G <= 32 lanes of a warp, or the whole block.
template <bool kMax>
__device__ __forceinline__ float combine(float a, float b) {
  return kMax ? max_nan(a, b) : a + b;
}
template <bool kMax, bool kBlock>
__device__ __forceinline__ float reduce_row(float v, int G, float* s) {
  const int lanes = kBlock ? 32 : G;
  for (int off = lanes >> 1; off > 0; off >>= 1)
    v = combine<kMax>(v, __shfl_xor_sync(0xffffffffu, v, off));
  if (!kBlock) return v;
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s[0];
  for (int i = 1; i < warps; ++i) v = combine<kMax>(v, s[i]);
  return v;
}

// One row per G threads (kBlock: per block), NV vectors of 8 columns a thread: vector
// i * G + (thread of the row).
template <typename T, bool kFp8, bool kBlock, int NV>
__global__ void __launch_bounds__(kBlock ? 1024 : 128) norm_kernel(const NormParams p, int G) {
  __shared__ float s_red[2][32];
  const int lane = kBlock ? threadIdx.x : threadIdx.x % G;
  const int per_block = kBlock ? 1 : blockDim.x / G;
  const long long row = (long long)blockIdx.x * per_block + (kBlock ? 0 : threadIdx.x / G);
  const bool some = row < p.rows;
  const long long rr = some ? row : 0;
  const long long token = rr / p.heads;
  const int head = (int)(rr % p.heads);
  const T* x = static_cast<const T*>(p.x) + token * p.x_stride + (long long)head * p.D;
  const T* gate = static_cast<const T*>(p.gate) + token * p.gate_stride + (long long)head * p.D;
  const bool vec = p.vec;

  Raw8<T> xr[NV], rr8[NV];
  float r[NV][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + lane) * 8, n = some ? p.D - c : 0;
    xr[i].zero();
    rr8[i].zero();
    if (n > 0) {
      xr[i] = load8(x + c, n, vec);
      if (p.residual)
        rr8[i] = load8(static_cast<const T*>(p.residual) + rr * p.D + c, n, vec);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + lane) * 8, n = some ? p.D - c : 0;
    xr[i].get(r[i]);
    if (p.residual) {
      float q[8];
      rr8[i].get(q);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[i][j] += q[j];
      Raw8<T> o;
      o.set(r[i]);
      if (n > 0) store8(static_cast<T*>(p.residual_out) + rr * p.D + c, o, n, vec);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(r[i][j], r[i][j], ss);
  }
  ss = reduce_row<false, kBlock>(ss, G, s_red[0]);
  const float rstd = rsqrtf(ss / (float)p.D + p.eps);

  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + lane) * 8, n = some ? p.D - c : 0;
    if (n > 0) {
      float w[8];
      load8(p.w + c, n, vec).get(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[i][j] = r[i][j] * rstd * w[j];
      if (p.gate) {
        float g[8];
        load8(gate + c, n, vec).get(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] *= silu(g[j]);
      }
      if (!kFp8) {
        Raw8<T> o;
        o.set(r[i]);
        store8(static_cast<T*>(p.y) + rr * p.D + c, o, n, vec);
      }
    }
    if (kFp8) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) m = max_nan(m, fabsf(r[i][j]));
      if (p.group < p.D) {  // the lanes of the group: group / 8 neighbours
        for (int off = p.group >> 4; off > 0; off >>= 1)
          m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        const float scale = m == 0.f ? 1.f : max_nan(__fdiv_rn(m, 448.f), 1.17549435e-38f);
        if (n > 0) {
          const float inv = __frcp_rn(scale);
          uint8_t* q = static_cast<uint8_t*>(p.y) + rr * p.D + c;
          const uint2 v = make_uint2(e4m3x4(&r[i][0], inv), e4m3x4(&r[i][4], inv));
          if (vec) {
            *reinterpret_cast<uint2*>(q) = v;
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j < n) q[j] = (uint8_t)((j < 4 ? v.x : v.y) >> (8 * (j & 3)));
          }
          const int groups = (p.D + p.group - 1) / p.group;
          if (c % p.group == 0) p.scales[rr * groups + c / p.group] = scale;
        }
      } else {
        amax = max_nan(amax, m);
      }
    }
  }
  if (kFp8 && p.group >= p.D) {  // one scale a row
    amax = reduce_row<true, kBlock>(amax, G, s_red[1]);
    const float scale = amax == 0.f ? 1.f : max_nan(__fdiv_rn(amax, 448.f), 1.17549435e-38f);
    const float inv = __frcp_rn(scale);
    if (some && lane == 0) p.scales[rr] = scale;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * G + lane) * 8, n = some ? p.D - c : 0;
      if (n <= 0) continue;
      uint8_t* q = static_cast<uint8_t*>(p.y) + rr * p.D + c;
      const uint2 v = make_uint2(e4m3x4(&r[i][0], inv), e4m3x4(&r[i][4], inv));
      if (vec) {
        *reinterpret_cast<uint2*>(q) = v;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) q[j] = (uint8_t)((j < 4 ? v.x : v.y) >> (8 * (j & 3)));
      }
    }
  }
}

template <typename T, bool kFp8>
cudaError_t launch_t(const NormParams& p, cudaStream_t stream) {
  const int nvec = (p.D + 7) / 8;
  if (nvec <= 128) {  // rows within a warp, 128 threads a block
    int G = 4;
    while (G < nvec && G < 32) G *= 2;
    const int rows = 128 / G;
    const unsigned grid = (unsigned)((p.rows + rows - 1) / rows);
    if (nvec <= 32) norm_kernel<T, kFp8, false, 1><<<grid, 128, 0, stream>>>(p, G);
    else if (nvec <= 64) norm_kernel<T, kFp8, false, 2><<<grid, 128, 0, stream>>>(p, G);
    else norm_kernel<T, kFp8, false, 4><<<grid, 128, 0, stream>>>(p, G);
    return cudaGetLastError();
  }
  const int nv = nvec <= 1024 ? (p.rows <= 152 ? 1 : 2) : nvec <= 2048 ? 2 : 4;
  const int G = ((nvec + nv - 1) / nv + 31) / 32 * 32;
  if (nv == 1) norm_kernel<T, kFp8, true, 1><<<(unsigned)p.rows, G, 0, stream>>>(p, G);
  else if (nv == 2) norm_kernel<T, kFp8, true, 2><<<(unsigned)p.rows, G, 0, stream>>>(p, G);
  else norm_kernel<T, kFp8, true, 4><<<(unsigned)p.rows, G, 0, stream>>>(p, G);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, bool f32, bool fp8, cudaStream_t stream) {
  if (f32) return fp8 ? launch_t<float, true>(p, stream) : launch_t<float, false>(p, stream);
  return fp8 ? launch_t<__nv_bfloat16, true>(p, stream) : launch_t<__nv_bfloat16, false>(p, stream);
}

}  // namespace gdn
