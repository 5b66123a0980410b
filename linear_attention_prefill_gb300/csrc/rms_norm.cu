// rms_norm.cu - RMS norm of rows: before a layer's projections (with the residual's addition,
// into 16 bits or e4m3 with scales), and of each head after a forward (with its gate).
//
//   r = x + residual,   y = r / sqrt(mean(r^2) + eps) w silu(gate),
//   e4m3: scale = max|y| / 448 over each group of columns (at least 2^-126; 1 for a group of
//   zeros), q = y times the scale's reciprocal (rcp.approx), rounded to nearest even.
//
// SiLU behind the norm is the only gate: a Gated DeltaNet layer's.
//
// r is added, normed and quantised in fp32; it is rounded once to be stored as the new
// residual, and y once on the way out.  HBM bandwidth bounds it: every tensor crosses once,
// with the row held in registers between the sum of squares and the output.  A thread
// holds vectors of 8 columns as packed pairs, so a group of 32, 64 or 128 columns is 4, 8 or 16
// lanes.  Rows of up to 512 columns stay within a warp (65536 gated heads of 128, bf16, 50 MB:
// 11.6 us in a graph, 4.3 TB/s); wider ones take a block each (16 rows of 2560 with residual into
// e4m3: 2.1 us) or, many of them, a ring of bulk copies (8192 x 5120 with residual into e4m3, 295
// MB: 52 us, 5.7 TB/s).  Kernels of whole vectors are apart from those for other rows: with both
// in one the compiler left fewer loads in flight (13.4 us against 12.4 for the heads, a call).
#include "gdn_common.cuh"
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {
namespace {

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_abs(const f32x2 (&v)[4]) {
  float a[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) unpack2(v[j], a[2 * j], a[2 * j + 1]);
#pragma unroll
  for (int j = 0; j < 8; ++j) a[j] = fabsf(a[j]);
  return max_nan(max_nan(max_nan(a[0], a[1]), max_nan(a[2], a[3])),
                 max_nan(max_nan(a[4], a[5]), max_nan(a[6], a[7])));
}

// Two e4m3, saturating.
__device__ __forceinline__ uint32_t e4m3x2(f32x2 v) {
  float a, b;
  unpack2(v, a, b);
  uint16_t q;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(q) : "f"(b), "f"(a));
  return q;
}
// One vector's e4m3 of y * inv.
__device__ __forceinline__ void store_e4m3(uint8_t* q, const f32x2 (&y)[4], float inv, int n,
                                           int by) {
  const f32x2 s = dup2(inv);
  const uint2 v = make_uint2(e4m3x2(mul2(y[0], s)) | (e4m3x2(mul2(y[1], s)) << 16),
                             e4m3x2(mul2(y[2], s)) | (e4m3x2(mul2(y[3], s)) << 16));
  if (by == 8) {
    *reinterpret_cast<uint2*>(q) = v;
  } else if (by == 4) {
    if (n > 0) reinterpret_cast<uint32_t*>(q)[0] = v.x;
    if (n > 4) reinterpret_cast<uint32_t*>(q)[1] = v.y;
  } else if (by == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (2 * j < n) reinterpret_cast<uint16_t*>(q)[j] = (uint16_t)((j < 2 ? v.x : v.y) >> (16 * (j & 1)));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) q[j] = (uint8_t)((j < 4 ? v.x : v.y) >> (8 * (j & 3)));
  }
}
// max|y| -> scale; the reciprocal and the product by 1 / 448 are within an ulp each
__device__ __forceinline__ float scale_of(float m) {
  return m == 0.f ? 1.f : m < 5.2666e-36f ? 1.17549435e-38f : m * (1.f / 448.f);
}

// Sum or maximum over the G threads of a row: G <= 32 lanes of a warp, or the whole block.
template <bool kMax>
__device__ __forceinline__ float combine(float a, float b) {
  return kMax ? max_nan(a, b) : a + b;
}
template <bool kMax, bool kBlock>
__device__ __forceinline__ float reduce_row(float v, int G, float* s) {
  if (kBlock) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      v = combine<kMax>(v, __shfl_xor_sync(0xffffffffu, v, off));
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    const int warps = blockDim.x >> 5;  // every warp adds the warps' results
    v = (threadIdx.x & 31) < warps ? s[threadIdx.x & 31] : 0.f;
    for (int off = warps > 16 ? 16 : warps > 8 ? 8 : warps > 4 ? 4 : 2; off > 0; off >>= 1)
      v = combine<kMax>(v, __shfl_xor_sync(0xffffffffu, v, off));
    return __shfl_sync(0xffffffffu, v, 0);
  }
#pragma unroll
  for (int off = G >> 1; off > 0; off >>= 1)
    v = combine<kMax>(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// What a row is after its sum of squares is known: y of every vector, stored.  r: the row's
// vectors; load_w(i), load_gate(i): vector i of w and of the gate; n[i]: columns that exist
// (whole vectors with kWhole, where p.by is 8); some: there is a row; at: its
// first element of the lane in the outputs, scales: its scales.
template <typename T, bool kFp8, bool kBlock, bool kWhole, int NV, typename LoadW, typename LoadGate>
__device__ __forceinline__ void finish(const NormParams& p, long long at, float* scales, bool some,
                                       int G, int lane, f32x2 (&r)[NV][4], const int (&n)[NV], float ss,
                                       float* s_max, LoadW load_w, LoadGate load_gate) {
  const int by = kWhole ? 8 : p.by;
  const f32x2 rstd = dup2(rsqrtf(ss * p.inv_d + p.eps));
  T* y = static_cast<T*>(p.y) + at;
  uint8_t* y8 = static_cast<uint8_t*>(p.y) + at;
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool here = some && n[i] > 0;
    if (here) {
      f32x2 q[4];
      load_w(i, q);
#pragma unroll
      for (int j = 0; j < 4; ++j) r[i][j] = mul2(mul2(r[i][j], rstd), q[j]);
      if (p.gate) {
        load_gate(i, q);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i][j] = mul2(r[i][j], silu2(q[j]));
      }
      if (!kFp8) store8(y + i * G * 8, raw_of<T>(r[i]), n[i], by);
    }
    if (kFp8) {
      float m = 0.f;
      if (here) {
        if (by != 8) {  // columns that do not exist were read as zeros, but a row of NaN has none
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float a, b;
            unpack2(r[i][j], a, b);
            r[i][j] = pack2(2 * j < n[i] ? a : 0.f, 2 * j + 1 < n[i] ? b : 0.f);
          }
        }
        m = max_abs(r[i]);
      }
      if (p.group < p.D) {  // the lanes of the group: group / 8 neighbours
        for (int off = p.group >> 4; off > 0; off >>= 1)
          m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (here) {
          const float scale = scale_of(m);
          store_e4m3(y8 + i * G * 8, r[i], rcp(scale), n[i], by);
          const int c = (i * G + lane) * 8;
          if ((c & (p.group - 1)) == 0) scales[c >> p.group_log] = scale;
        }
      } else {
        amax = max_nan(amax, m);
      }
    }
  }
  if (kFp8 && p.group >= p.D) {  // one scale a row
    amax = reduce_row<true, kBlock>(amax, G, s_max);
    const float scale = scale_of(amax), inv = rcp(scale);
    if (some && lane == 0) *scales = scale;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (some && n[i] > 0) store_e4m3(y8 + i * G * 8, r[i], inv, n[i], by);
  }
}

// x + residual of one vector, the residual's update stored; adds the squares to ss.
template <typename T, bool kWhole>
__device__ __forceinline__ void take(const NormParams& p, T* out, const Raw8<T>& x,
                                     const Raw8<T>& res, int n, f32x2 (&r)[4], f32x2& ss) {
  pairs_of(x, r);
  if (p.residual) {
    f32x2 q[4];
    pairs_of(res, q);
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = add2(r[j], q[j]);
    store8(out, raw_of<T>(r), n, kWhole ? 8 : p.by);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) ss = fma2(r[j], r[j], ss);
}

// Rows within a warp: G lanes a row, NV vectors of 8 columns a lane: vector i * G + lane.  A
// block walks its rows, the next one is loaded while the present one is reduced, and w stays in
// registers.
template <typename T, bool kFp8, bool kWhole, int G, int NV>
__global__ void __launch_bounds__(128) norm_warp_kernel(const NormParams p) {
  constexpr int per_block = 128 / G;
  const int lane = threadIdx.x % G;
  const unsigned step = gridDim.x * per_block, rows = (unsigned)p.rows;  // (rows fit 31 bits)
  const int by = kWhole ? 8 : p.by;
  int n[NV];
  f32x2 w[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + lane) * 8;
    n[i] = p.D - c;
    if (n[i] > 0) pairs_of(load8(p.w + c, n[i], by), w[i]);
  }
  Raw8<T> x[NV], res[NV], gate[NV];
  const unsigned row0 = blockIdx.x * per_block + threadIdx.x / G;
  long long at = (long long)row0 * p.D + lane * 8;  // of the present row in the dense tensors
  const long long step_at = (long long)step * p.D;
  float* scales = p.scales + (long long)row0 * p.groups;
  const T* xp = static_cast<const T*>(p.x) + lane * 8;
  const T* gp = static_cast<const T*>(p.gate) + lane * 8;
  const T* rp = static_cast<const T*>(p.residual) + at;
  const bool heads = p.heads > 1;  // else a row's place moves on by a constant
  if (!heads) xp += row0 * p.x_stride, gp += row0 * p.gate_stride;
  auto load_row = [&](unsigned row) {
    const T *xr = xp, *gr = gp;
    if (heads) {
      // (with a 64-bit quotient 131072 heads of 64: 12.7 us against 10.9)
      const unsigned token = row / (unsigned)p.heads;
      const int col = (int)(row - token * p.heads) * p.D;
      xr += token * p.x_stride + col;
      gr += token * p.gate_stride + col;
    } else {
      xp += step * p.x_stride;
      gp += step * p.gate_stride;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (n[i] <= 0) continue;
      x[i] = load8(xr + i * G * 8, n[i], by);
      if (p.residual) res[i] = load8(rp + i * G * 8, n[i], by);
      if (p.gate) gate[i] = load8(gr + i * G * 8, n[i], by);
    }
    rp += step_at;
  };
  if (row0 < rows) load_row(row0);
  // every lane of a warp stays for the shuffles
  for (unsigned row = row0; row - threadIdx.x / G < rows; row += step) {
    const bool some = row < rows;
    T* out = static_cast<T*>(p.residual_out) + at;
    f32x2 r[NV][4], ss = 0ull;
    Raw8<T> g[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (some && n[i] > 0) {
        take<T, kWhole>(p, out + i * G * 8, x[i], res[i], n[i], r[i], ss);
        g[i] = gate[i];
      }
    }
    if (row + step < rows) load_row(row + step);
    float s0, s1;
    unpack2(ss, s0, s1);
    const float sum = reduce_row<false, false>(s0 + s1, G, nullptr);
    finish<T, kFp8, false, kWhole, NV>(
        p, at, scales, some, G, lane, r, n, sum, nullptr,
        [&](int i, f32x2 (&q)[4]) {
#pragma unroll
          for (int j = 0; j < 4; ++j) q[j] = w[i][j];
        },
        [&](int i, f32x2 (&q)[4]) { pairs_of(g[i], q); });
    at += step_at;
    if (kFp8) scales += (long long)step * p.groups;
  }
}

// A row per block of G threads, NV vectors a thread.  Up to 8192 columns w and the gate are
// loaded with the row; wider blocks (up to 1024 threads) have registers for the row only, and of
// fp32 rows not even that: 64 registers a thread spill 144 to 396 bytes (2048 x 16384: bf16 32.8 us,
// 4.1 TB/s; fp32 61.8, 4.3).
template <typename T, bool kFp8, bool kWhole, int NV>
__global__ void __launch_bounds__(NV == 4 ? 1024 : 1024 / NV, 1)
    norm_block_kernel(const NormParams p, int G) {
  constexpr bool kWide = NV == 4;
  __shared__ float s_sum[32], s_max[32];
  const int lane = threadIdx.x;
  const int by = kWhole ? 8 : p.by;
  const long long row = blockIdx.x;
  const long long token = p.heads == 1 ? row : (unsigned)row / (unsigned)p.heads;
  const long long col = (row - token * p.heads) * p.D + lane * 8;
  const T* xp = static_cast<const T*>(p.x) + token * p.x_stride + col;
  const T* gp = static_cast<const T*>(p.gate) + token * p.gate_stride + col;
  int n[NV];
  Raw8<T> x[NV], res[NV], g[kWide ? 1 : NV];
  Raw8<float> w[kWide ? 1 : NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + lane) * 8;
    n[i] = p.D - c;
    if (n[i] <= 0) continue;
    x[i] = load8(xp + i * G * 8, n[i], by);
    if (p.residual) res[i] = load8(static_cast<const T*>(p.residual) + row * p.D + c, n[i], by);
  }
  if (!kWide) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (n[i] <= 0) continue;
      if (p.gate) g[i] = load8(gp + i * G * 8, n[i], by);
      w[i] = load8(p.w + (i * G + lane) * 8, n[i], by);
    }
  }
  f32x2 r[NV][4], ss = 0ull;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (n[i] > 0)
      take<T, kWhole>(p, static_cast<T*>(p.residual_out) + row * p.D + (i * G + lane) * 8, x[i], res[i], n[i],
           r[i], ss);
  float s0, s1;
  unpack2(ss, s0, s1);
  const float sum = reduce_row<false, true>(s0 + s1, G, s_sum);
  finish<T, kFp8, true, kWhole, NV>(
      p, row * p.D + lane * 8, p.scales + row * p.groups, true, G, lane, r, n, sum, s_max,
      [&](int i, f32x2 (&q)[4]) {
        if (kWide) w[0] = load8(p.w + (i * G + lane) * 8, n[i], by);
        pairs_of(w[kWide ? 0 : i], q);
      },
      [&](int i, f32x2 (&q)[4]) {
        if (kWide) g[0] = load8(gp + i * G * 8, n[i], by);
        pairs_of(g[kWide ? 0 : i], q);
      });
}

// Many wide rows: a persistent block whose rows arrive by bulk copies in a ring of shared
// memory, several rows ahead, so that no row's arrival is waited for and none is held in
// registers.  G threads have vectors i * G + thread.
constexpr int kRingThreads = 512, kRingBytes = 220 * 1024;
template <typename T, bool kFp8, int NV>
__global__ void __maxnreg__(NV == 1 ? 64 : NV > 2 ? 128 : sizeof(T) == 4 ? 96 : 80)
    norm_ring_kernel(const NormParams p, int G, int slots, int slot_bytes) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ uint64_t full[16];
  __shared__ float s_sum[2][32], s_max[2][32];  // by turns: one barrier a reduction is enough
  const int tid = threadIdx.x;
  const int row_bytes = p.D * (int)sizeof(T);
  const int res_at = row_bytes, gate_at = row_bytes * (p.residual ? 2 : 1);
  int n[NV];
  Raw8<float> w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + tid) * 8;
    n[i] = p.D - c;
    if (n[i] > 0) w[i].load(p.w + c);
  }
  auto fetch = [&](long long row, int s) {  // one thread: the row's copies into slot s
    const long long token = p.heads == 1 ? row : (unsigned)row / (unsigned)p.heads;
    const long long col = (row - token * p.heads) * p.D;
    unsigned char* dst = ring + s * slot_bytes;
    mbar_expect_tx(&full[s], slot_bytes);
    bulk_g2s(dst, static_cast<const T*>(p.x) + token * p.x_stride + col, row_bytes, &full[s]);
    if (p.residual)
      bulk_g2s(dst + res_at, static_cast<const T*>(p.residual) + row * p.D, row_bytes, &full[s]);
    if (p.gate)
      bulk_g2s(dst + gate_at, static_cast<const T*>(p.gate) + token * p.gate_stride + col, row_bytes,
               &full[s]);
  };
  if (tid == 0) {
    for (int s = 0; s < slots; ++s) mbar_init(&full[s], 1);
    mbar_fence_init();
    for (int s = 0; s < slots; ++s) {
      const long long row = blockIdx.x + (long long)s * gridDim.x;
      if (row < p.rows) fetch(row, s);
    }
  }
  __syncthreads();
  int s = 0, turn = 0;
  unsigned phase = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    // a copy that does not arrive within about a second ends the block's work: it is recorded,
    // and the other copies in flight are waited for before the block leaves
    if (!mbar_wait(&full[s], phase, p.err)) {
      for (int k = 1; k < slots; ++k) {
        const int t = (s + k) % slots;
        if (row + (long long)k * gridDim.x < p.rows) mbar_wait(&full[t], t > s ? phase : phase ^ 1, p.err);
      }
      break;
    }
    const T* at = reinterpret_cast<const T*>(ring + s * slot_bytes) + tid * 8;
    T* out = static_cast<T*>(p.residual_out) + row * p.D + tid * 8;
    f32x2 r[NV][4], ss = 0ull;
    Raw8<T> g[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (n[i] <= 0) continue;
      const T* q = at + i * G * 8;
      Raw8<T> x, res;
      x.load(q);
      if (p.residual) res.load(q + p.D);
      if (p.gate) g[i].load(q + (p.residual ? 2 : 1) * p.D);
      take<T, true>(p, out + i * G * 8, x, res, 8, r[i], ss);
    }
    float s0, s1;
    unpack2(ss, s0, s1);
    const float sum = reduce_row<false, true>(s0 + s1, G, s_sum[turn]);
    // the reduction's barrier: every thread has read the slot
    const long long next = row + (long long)slots * gridDim.x;
    if (tid == 0 && next < p.rows) {
      fence_proxy_async();
      fetch(next, s);
    }
    finish<T, kFp8, true, true, NV>(
        p, row * p.D + tid * 8, p.scales + row * p.groups, true, G, tid, r, n, sum, s_max[turn],
        [&](int i, f32x2 (&q)[4]) { pairs_of(w[i], q); },
        [&](int i, f32x2 (&q)[4]) { pairs_of(g[i], q); });
    if (++s == slots) s = 0, phase ^= 1;
  }
}

template <typename T, bool kFp8, int G, int NV>
cudaError_t launch_warp(const NormParams& p, cudaStream_t stream) {
  const auto kernel = p.by == 8 ? norm_warp_kernel<T, kFp8, true, G, NV> : norm_warp_kernel<T, kFp8, false, G, NV>;
  static_assert(32 % G == 0, "rows do not cross warps");
  // as many blocks as are resident together; each takes its rows in turn
  int resident = 0;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kernel, 128, 0);
  if (e != cudaSuccess) return e;
  const long long rows = 128 / G, blocks = (p.rows + rows - 1) / rows;
  const long long most = (long long)(resident < 1 ? 1 : resident) * kSms;
  kernel<<<(unsigned)(blocks < most ? blocks : most), 128, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, bool kFp8, bool kWhole>
cudaError_t launch_block(const NormParams& p, cudaStream_t stream) {
  // one vector a thread for few rows (latency), two for many; four for the widest
  const int nvec = (p.D + 7) / 8;
  const int nv = nvec > 1024 ? 4 : p.rows <= kSms ? 1 : 2;
  const int G = ((nvec + nv - 1) / nv + 31) / 32 * 32;
  const unsigned grid = (unsigned)p.rows;
  const auto kernel = nv == 1   ? norm_block_kernel<T, kFp8, kWhole, 1>
                      : nv == 2 ? norm_block_kernel<T, kFp8, kWhole, 2>
                                : norm_block_kernel<T, kFp8, kWhole, 4>;
  kernel<<<grid, G, 0, stream>>>(p, G);
  return cudaGetLastError();
}

template <typename T>
int slot_of(const NormParams& p) {  // bytes of a row's tensors
  return p.D * (int)sizeof(T) * (1 + (p.residual ? 1 : 0) + (p.gate ? 1 : 0));
}
template <typename T, bool kFp8, int NV>
cudaError_t launch_ring(NormParams p, cudaStream_t stream) {
  const int slot_bytes = slot_of<T>(p);
  const int G = ((p.D / 8 + NV - 1) / NV + 31) / 32 * 32;
  // blocks of about 1024 threads an SM together, each with four slots or more; fewer where the
  // rows are too wide for that, down to one with two slots
  int blocks = 1024 / G < 2 ? 2 : 1024 / G > 8 ? 8 : 1024 / G;
  while (blocks > 1 && kRingBytes / blocks / slot_bytes < 4) --blocks;
  int slots = kRingBytes / blocks / slot_bytes;
  if (slots > 8) slots = 8;
  const auto kernel = norm_ring_kernel<T, kFp8, NV>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       slots * slot_bytes);
  if (e == cudaSuccess) e = device_error_word(&p.err);
  if (e != cudaSuccess) return e;
  const long long most = (long long)blocks * kSms;
  const unsigned grid = (unsigned)(p.rows < most ? p.rows : most);
  kernel<<<grid, G, slots * slot_bytes, stream>>>(p, G, slots, slot_bytes);
  return cudaGetLastError();
}

template <typename T, bool kFp8>
cudaError_t launch_t(const NormParams& p, cudaStream_t stream) {
  if (p.D <= 32) return launch_warp<T, kFp8, 4, 1>(p, stream);
  if (p.D <= 64) return launch_warp<T, kFp8, 8, 1>(p, stream);
  if (p.D <= 128) return launch_warp<T, kFp8, 16, 1>(p, stream);
  if (p.D <= 256) return launch_warp<T, kFp8, 32, 1>(p, stream);
  if (p.D <= 512) return launch_warp<T, kFp8, 32, 2>(p, stream);
  // the ring's copies are of whole 16-byte pieces; it pays once every block has a few rows (8192
  // rows of 5120, e4m3: 64 us a row per block, 52; 3531 of 11648 with a gate, e4m3: 72, 54)
  if (p.by == 8 && p.D <= 24 * kRingThreads && p.rows >= 8 * kSms && 2 * slot_of<T>(p) <= kRingBytes) {
    const int nv = (p.D / 8 + kRingThreads - 1) / kRingThreads;
    if (nv <= 1) return launch_ring<T, kFp8, 1>(p, stream);
    if (nv == 2) return launch_ring<T, kFp8, 2>(p, stream);
    return launch_ring<T, kFp8, 3>(p, stream);
  }
  return p.by == 8 ? launch_block<T, kFp8, true>(p, stream) : launch_block<T, kFp8, false>(p, stream);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, bool f32, bool fp8, cudaStream_t stream) {
  if (f32) return fp8 ? launch_t<float, true>(p, stream) : launch_t<float, false>(p, stream);
  return fp8 ? launch_t<__nv_bfloat16, true>(p, stream) : launch_t<__nv_bfloat16, false>(p, stream);
}

}  // namespace gdn
