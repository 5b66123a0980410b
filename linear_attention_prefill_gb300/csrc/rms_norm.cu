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

// The columns' e4m3 of one vector.
__device__ __forceinline__ void store_e4m3(uint8_t* q, const float (&r)[8], float inv, int n,
                                           bool vec) {
  const uint2 v = make_uint2(e4m3x4(&r[0], inv), e4m3x4(&r[4], inv));
  if (vec) {
    *reinterpret_cast<uint2*>(q) = v;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) q[j] = (uint8_t)((j < 4 ? v.x : v.y) >> (8 * (j & 3)));
  }
}
__device__ __forceinline__ float scale_of(float amax) {
  return amax == 0.f ? 1.f : max_nan(__fdiv_rn(amax, 448.f), 1.17549435e-38f);
}

// One row per G threads (kBlock: per block), NV vectors of 8 columns a thread: vector
// i * G + (thread of the row).  Rows within a warp: a block walks rows, the next one is
// loaded while the present one is reduced, and w stays in registers.  A row per block: one
// row each, as many blocks side by side as fit (beyond 8192 columns a block of up to 1024
// threads has registers for the row only, and loads w and the gate late).
template <typename T, bool kFp8, bool kBlock, int NV>
__global__ void __launch_bounds__(!kBlock ? 128 : NV == 4 ? 1024 : 1024 / NV)
    norm_kernel(const NormParams p, int G) {
  constexpr bool kWide = kBlock && NV == 4, kLoop = !kBlock;
  __shared__ float s_red[2][2][32];  // by turns, so that one barrier a reduction is enough
  const int lane = kBlock ? threadIdx.x : threadIdx.x % G;
  const int per_block = kBlock ? 1 : blockDim.x / G;
  const long long step = (long long)gridDim.x * per_block;
  const bool vec = p.vec;
  int n[NV];  // columns of this thread's vectors that exist
  float w[kWide ? 1 : NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + lane) * 8;
    n[i] = p.D - c;
    if (!kWide && n[i] > 0) load8(p.w + c, n[i], vec).get(w[i]);
  }
  Raw8<T> x_next[NV], r_next[NV], g_next[kWide ? 1 : NV];
  auto load_row = [&](long long row) {
    const long long token = row / p.heads;
    const long long col = (row - token * p.heads) * p.D;
    const T* x = static_cast<const T*>(p.x) + token * p.x_stride + col;
    const T* r = static_cast<const T*>(p.residual) + row * p.D;
    const T* g = static_cast<const T*>(p.gate) + token * p.gate_stride + col;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * G + lane) * 8;
      if (n[i] > 0) {
        x_next[i] = load8(x + c, n[i], vec);
        if (p.residual) r_next[i] = load8(r + c, n[i], vec);
        if (!kWide && p.gate) g_next[i] = load8(g + c, n[i], vec);
      }
    }
  };
  const long long row0 = (long long)blockIdx.x * per_block + (kBlock ? 0 : threadIdx.x / G);
  if (!kWide && row0 < p.rows) load_row(row0);
  int turn = 0;
  // every thread of a warp stays for the shuffles: rows are per block, or guarded by `some`
  for (long long base = (long long)blockIdx.x * per_block; base < p.rows;
       base = kLoop ? base + step : p.rows, turn ^= 1) {
    const long long row = base + (kBlock ? 0 : threadIdx.x / G);
    const bool some = row < p.rows;
    float r[NV][8];
    Raw8<T> g[kWide ? 1 : NV];
    float ss = 0.f;
    if (kWide) load_row(row);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!kWide) g[i] = g_next[i];
      if (!some || n[i] <= 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = 0.f;
        continue;
      }
      x_next[i].get(r[i]);
      if (p.residual) {
        float q[8];
        r_next[i].get(q);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] += q[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(r[i][j], r[i][j], ss);
    }
    if (kLoop && row + step < p.rows) load_row(row + step);
    if (p.residual && some) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * G + lane) * 8;
        Raw8<T> o;
        o.set(r[i]);
        if (n[i] > 0) store8(static_cast<T*>(p.residual_out) + row * p.D + c, o, n[i], vec);
      }
    }
    ss = reduce_row<false, kBlock>(ss, G, s_red[0][turn]);
    const float rstd = rsqrtf(ss / (float)p.D + p.eps);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * G + lane) * 8;
      const bool here = some && n[i] > 0;
      if (here) {
        if (kWide) load8(p.w + c, n[i], vec).get(w[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = r[i][j] * rstd * w[kWide ? 0 : i][j];
        if (p.gate) {
          float q[8];
          if (kWide) {
            const long long token = row / p.heads;
            g[0] = load8(static_cast<const T*>(p.gate) + token * p.gate_stride +
                             (row - token * p.heads) * p.D + c,
                         n[i], vec);
          }
          g[kWide ? 0 : i].get(q);
#pragma unroll
          for (int j = 0; j < 8; ++j) r[i][j] *= silu(q[j]);
        }
        if (!kFp8) {
          Raw8<T> o;
          o.set(r[i]);
          store8(static_cast<T*>(p.y) + row * p.D + c, o, n[i], vec);
        }
      }
      if (kFp8) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (here && j < n[i]) m = max_nan(m, fabsf(r[i][j]));
        if (p.group < p.D) {  // the lanes of the group: group / 8 neighbours
          for (int off = p.group >> 4; off > 0; off >>= 1)
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
          if (here) {
            const float scale = scale_of(m);
            store_e4m3(static_cast<uint8_t*>(p.y) + row * p.D + c, r[i], __frcp_rn(scale), n[i], vec);
            const int groups = (p.D + p.group - 1) / p.group;
            if (c % p.group == 0) p.scales[row * groups + c / p.group] = scale;
          }
        } else {
          amax = max_nan(amax, m);
        }
      }
    }
    if (kFp8 && p.group >= p.D) {  // one scale a row
      amax = reduce_row<true, kBlock>(amax, G, s_red[1][turn]);
      const float scale = scale_of(amax), inv = __frcp_rn(scale);
      if (some && lane == 0) p.scales[row] = scale;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (some && n[i] > 0)
          store_e4m3(static_cast<uint8_t*>(p.y) + row * p.D + (i * G + lane) * 8, r[i], inv, n[i], vec);
    }
  }
}

template <typename T, bool kFp8, bool kBlock, int NV>
cudaError_t launch_k(const NormParams& p, int threads, int G, cudaStream_t stream) {
  const long long per_block = kBlock ? 1 : threads / G;
  const long long blocks = (p.rows + per_block - 1) / per_block;
  // rows within a warp: as many blocks as fit side by side, each takes its rows in turn
  const long long most = kBlock ? blocks : 12ll * kSms;
  norm_kernel<T, kFp8, kBlock, NV>
      <<<(unsigned)(blocks < most ? blocks : most), threads, 0, stream>>>(p, G);
  return cudaGetLastError();
}

template <typename T, bool kFp8>
cudaError_t launch_t(const NormParams& p, cudaStream_t stream) {
  const int nvec = (p.D + 7) / 8;
  if (nvec <= 64) {  // rows within a warp, 128 threads a block
    int G = 4;
    while (G < nvec && G < 32) G *= 2;
    if (nvec <= 32) return launch_k<T, kFp8, false, 1>(p, 128, G, stream);
    return launch_k<T, kFp8, false, 2>(p, 128, G, stream);
  }
  // one vector a thread for few rows (latency), two for many; four for the widest
  const int nv = nvec > 1024 ? 4 : p.rows <= 152 ? 1 : 2;
  const int G = ((nvec + nv - 1) / nv + 31) / 32 * 32;
  if (nv == 1) return launch_k<T, kFp8, true, 1>(p, G, G, stream);
  if (nv == 2) return launch_k<T, kFp8, true, 2>(p, G, G, stream);
  return launch_k<T, kFp8, true, 4>(p, G, G, stream);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, bool f32, bool fp8, cudaStream_t stream) {
  if (f32) return fp8 ? launch_t<float, true>(p, stream) : launch_t<float, false>(p, stream);
  return fp8 ? launch_t<__nv_bfloat16, true>(p, stream) : launch_t<__nv_bfloat16, false>(p, stream);
}

}  // namespace gdn
