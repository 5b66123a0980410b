// glr_common.cuh - what the gated linear recurrence's kernels share: channel pairs, gates,
// sequence borders, and the composition of stretches of time.
//
//   h_t = a_t h_{t-1} + s(a_t) x_t,   a = exp(L):
//   gate      L = g (log), log sigmoid(g) (sigmoid), rate sigmoid(g) (rate)
//   weight    s = 1 (none), 1 - a (linear), sqrt(1 - a^2) (sqrt)
//
// A stretch of tokens maps the state before it to A h + H.  Stretches compose, so time is cut
// everywhere: a thread has kRun tokens of two channels, a warp 64 channels, a block's warps
// follow each other in time, and so do the blocks of a cluster.
#pragma once

#include <stdlib.h>
#include <atomic>

#include "cluster.cuh"
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {

constexpr float kTiny = 1.17549435e-38f;  // 2^-126

// ---- two channels of a row ---------------------------------------------------------------
// Channels 2 lane, 2 lane + 1 of a warp's 64: in one access where rows are aligned to pairs (vec).
template <typename T>
struct Raw2;
template <>
struct Raw2<__nv_bfloat16> {
  uint32_t v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool vec, bool c0, bool c1) {
    if (vec) {
      v = c0 ? *reinterpret_cast<const uint32_t*>(p) : 0u;
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
      v = (c0 ? (uint32_t)q[0] : 0u) | (c1 ? (uint32_t)q[1] << 16 : 0u);
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, bool vec, bool c0, bool c1) const {
    if (vec) {
      if (c0) *reinterpret_cast<uint32_t*>(p) = v;
    } else {
      uint16_t* q = reinterpret_cast<uint16_t*>(p);
      if (c0) q[0] = (uint16_t)v;
      if (c1) q[1] = (uint16_t)(v >> 16);
    }
  }
  __device__ __forceinline__ f32x2 get() const {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(v << 16), "r"(v & 0xffff0000u));
    return r;
  }
  __device__ __forceinline__ void set(f32x2 x) {
    float a, b;
    unpack2(x, a, b);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(b), "f"(a));
  }
};
template <>
struct Raw2<float> {
  f32x2 v;
  __device__ __forceinline__ void load(const float* p, bool vec, bool c0, bool c1) {
    if (vec) v = c0 ? *reinterpret_cast<const f32x2*>(p) : 0ull;
    else v = pack2(c0 ? p[0] : 0.f, c1 ? p[1] : 0.f);
  }
  __device__ __forceinline__ void store(float* p, bool vec, bool c0, bool c1) const {
    if (vec) {
      if (c0) *reinterpret_cast<f32x2*>(p) = v;
    } else {
      float a, b;
      unpack2(v, a, b);
      if (c0) p[0] = a;
      if (c1) p[1] = b;
    }
  }
  __device__ __forceinline__ f32x2 get() const { return v; }
  __device__ __forceinline__ void set(f32x2 x) { v = x; }
};
__device__ __forceinline__ f32x2 load_f32(const float* p, bool vec, bool c0, bool c1) {
  Raw2<float> r;
  r.load(p, vec, c0, c1);
  return r.v;
}
__device__ __forceinline__ void store_f32(float* p, f32x2 x, bool vec, bool c0, bool c1) {
  Raw2<float> r;
  r.v = x;
  r.store(p, vec, c0, c1);
}
// A tile's pair in shared memory, tokens of 64 channels.
template <typename T>
__device__ __forceinline__ f32x2 pair_at(const T* tile, int token, int lane) {
  Raw2<T> r;
  r.load(tile + token * 64 + 2 * lane, true, true, true);
  return r.get();
}

// ---- tiles on their way into shared memory ---------------------------------------------------
// Bytes of an access: 16 and 4 are asynchronous copies, 2 plain loads (odd rows of bf16).
template <int kBytes>
__device__ __forceinline__ void copy_piece(void* to, const void* from, bool ok) {
  if constexpr (kBytes == 16) {
    cp_async16(to, from, ok);
  } else if constexpr (kBytes == 4) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(ok ? 4 : 0)
                 : "memory");
  } else {
    *static_cast<uint16_t*>(to) = ok ? *static_cast<const uint16_t*>(from) : (uint16_t)0;
  }
}
// Up to kTokens rows (`tokens`) of 64 channels, `cols` of which exist, from src; zeros for rows from
// `rows` on and for channels that do not exist.
template <int kBytes, int kTokens, int kThreads, typename T>
__device__ __forceinline__ void copy_rows(T* tile, const T* src, long long stride, int rows, int tokens, int cols) {
  constexpr int kCols = kBytes / (int)sizeof(T), kPieces = 64 / kCols;
  if (kBytes == 16 && blockDim.x == kThreads && rows >= kTokens) {  // a whole tile, by a whole block
    constexpr int kStep = kThreads / kPieces;
    const int row = threadIdx.x / kPieces, col = threadIdx.x % kPieces * kCols;
    const T* from = src + row * stride + col;
    const bool ok = col < cols;
    if (!ok) from = src;
    const long long step = ok ? kStep * stride : 0;
    tile += row * 64 + col;
#pragma unroll
    for (int i = 0; i < kTokens / kStep; ++i) {
      copy_piece<kBytes>(tile + i * kStep * 64, from, ok);
      from += step;
    }
    return;
  }
#pragma unroll 4
  for (int i = threadIdx.x; i < tokens * kPieces; i += blockDim.x) {
    const int row = i / kPieces, col = i % kPieces * kCols;
    const bool ok = col < cols && row < rows;
    copy_piece<kBytes>(tile + row * 64 + col, ok ? src + row * stride + col : src, ok);
  }
}
// By all threads of the block; rows are made of, and aligned to, pieces of so many bytes.
template <int kTokens, int kThreads, typename T>
__device__ __forceinline__ void copy_tile(T* tile, const T* src, long long stride, int rows, int tokens, int cols,
                                          int piece) {
  if (piece == 16) {
    copy_rows<16, kTokens, kThreads>(tile, src, stride, rows, tokens, cols);
  } else if (sizeof(T) == 4 || piece == 4) {
    copy_rows<4, kTokens, kThreads>(tile, src, stride, rows, tokens, cols);
  } else if constexpr (sizeof(T) == 2) {
    copy_rows<2, kTokens, kThreads>(tile, src, stride, rows, tokens, cols);
  }
}

// ---- gates -------------------------------------------------------------------------------
__device__ __forceinline__ float sqrt_ftz(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <typename F>
__device__ __forceinline__ f32x2 each(f32x2 x, F f) {
  float a, b;
  unpack2(x, a, b);
  return pack2(f(a), f(b));
}
__device__ __forceinline__ f32x2 neg2(f32x2 x) { return x ^ 0x8000000080000000ull; }

// e^u - 1 for |u| < 1/2: u times the polynomial of degree 6 with the least relative error there
// (3.0e-9, by Remez's exchange; 1.2e-7 with the roundings).
__device__ __forceinline__ f32x2 expm1_small(f32x2 u) {
  f32x2 r = dup2(0.000198411915f);
  r = fma2(r, u, dup2(0.00139973243f));
  r = fma2(r, u, dup2(0.00833363459f));
  r = fma2(r, u, dup2(0.0416653194f));
  r = fma2(r, u, dup2(0.166666627f));
  r = fma2(r, u, dup2(0.50000006f));
  r = fma2(r, u, dup2(1.f));
  return mul2(r, u);
}
__device__ __forceinline__ f32x2 rcp2(f32x2 x) {
  return each(x, [](float v) { return rcp(v); });
}
__device__ __forceinline__ f32x2 exp_neg(f32x2 g) {
  return each(mul2(g, dup2(-kLog2e)), [](float v) { return ex2(v); });
}
// sigmoid(g) and 1 - sigmoid(g), each to its last digits: with e = e^-g and q = 1 / (1 + e) they are q and
// e q, but what is nearer to 1 is 1 less the other.
__device__ __forceinline__ void sigmoid2(f32x2 g, f32x2& sig, f32x2& rest) {
  const f32x2 one = dup2(1.f), minus = dup2(-1.f), e = exp_neg(g);
  const f32x2 nq = rcp2(fma2(e, minus, minus));  // -q
  float e0, e1, q0, q1, p0, p1, l0, l1, r0, r1;
  unpack2(e, e0, e1);
  unpack2(nq, q0, q1);
  unpack2(mul2(e, nq), p0, p1);
  unpack2(fma2(e, nq, one), l0, l1);
  unpack2(add2(one, nq), r0, r1);
  sig = pack2(e0 < 1.f ? l0 : -q0, e1 < 1.f ? l1 : -q1);
  rest = pack2(e0 < 1.f ? -p0 : r0, e1 < 1.f ? -p1 : r1);
}

// The decay a and the input's weight s of a token.  Decays next to 1 come from 1 - a, which keeps its
// digits there: a then is off by one rounding, not by the error of 2^x, whose like sign over the
// thousand tokens that such a decay remembers would show in fp32 sums.
template <int kGate, int kNorm>
__device__ __forceinline__ void gate2(f32x2 g, f32x2 rate, f32x2& a, f32x2& s) {
  const f32x2 one = dup2(1.f);
  f32x2 left;  // 1 - a
  if (kGate == GLR_SIGMOID) {
    sigmoid2(g, a, left);
  } else {
    f32x2 log = g;
    if (kGate == GLR_RATE) log = mul2(rate, rcp2(add2(exp_neg(g), one)));
    const f32x2 e = each(mul2(log, dup2(kLog2e)), [](float v) { return ex2(v); }), small = expm1_small(log);
    float u0, u1, s0, s1, a0, a1, e0, e1, d0, d1;
    unpack2(log, u0, u1);
    unpack2(small, s0, s1);
    unpack2(add2(one, small), a0, a1);
    unpack2(e, e0, e1);
    unpack2(fma2(e, dup2(-1.f), one), d0, d1);
    const bool near0 = fabsf(u0) < 0.5f, near1 = fabsf(u1) < 0.5f;
    a = pack2(near0 ? a0 : e0, near1 ? a1 : e1);
    left = pack2(near0 ? -s0 : d0, near1 ? -s1 : d1);
  }
  if (kNorm == GLR_NONE) s = one;
  if (kNorm == GLR_LINEAR) s = left;
  if (kNorm == GLR_SQRT) s = each(fma2(left, a, left), [](float v) { return sqrt_ftz(v); });
}

// ---- stretches of time ---------------------------------------------------------------------
// A product of decays that underflows stays at 2^-126: an infinite state before it stays infinite,
// as it does token by token, and of finite ones nothing is left either way.  A = 0 is a border: what
// lies behind it sees nothing from before, not even infinities.
__device__ __forceinline__ f32x2 at_least_tiny(f32x2 a) {
  return each(a, [](float v) { return fmaxf(v, kTiny); });
}
template <bool kBorders>
__device__ __forceinline__ f32x2 through(f32x2 A, f32x2 H, f32x2 h) {  // A h + H
  if (!kBorders) return fma2(A, h, H);
  float a0, a1, b0, b1, r0, r1;
  unpack2(A, a0, a1);
  unpack2(H, b0, b1);
  unpack2(fma2(A, h, H), r0, r1);
  return pack2(a0 == 0.f ? b0 : r0, a1 == 0.f ? b1 : r1);
}
// (A, H) followed by (B, G)
template <bool kBorders>
__device__ __forceinline__ void follow(f32x2& A, f32x2& H, f32x2 B, f32x2 G) {
  H = through<kBorders>(B, G, H);
  const f32x2 product = at_least_tiny(mul2(A, B));
  if (!kBorders) {
    A = product;
    return;
  }
  float a0, a1, b0, b1, p0, p1;
  unpack2(A, a0, a1);
  unpack2(B, b0, b1);
  unpack2(product, p0, p1);
  A = pack2(a0 == 0.f || b0 == 0.f ? 0.f : p0, a1 == 0.f || b1 == 0.f ? 0.f : p1);
}

// ---- sequence borders of a packed row ------------------------------------------------------
// The first m in [0, N] with min(max(cu[m], 0), end) > v, N + 1 if there is none; by a warp,
// 32 places at a time.  In range whatever the table holds.
__device__ __forceinline__ int first_border_above(const int32_t* cu, int N, int end, int v) {
  const int lane = threadIdx.x & 31;
  long long lo = 0, hi = (long long)N + 1;
  while (lo < hi) {
    const long long step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool above = at >= hi || min(max(cu[at], 0), end) > v;
    const unsigned votes = __ballot_sync(0xffffffffu, above);
    const int first = votes ? __ffs(votes) - 1 : 32;
    if (first == 0) return (int)lo;
    const long long top = lo + first * step;
    lo += (first - 1) * step + 1;
    if (top < hi) hi = top;
  }
  return (int)lo;
}
// The sequence that holds token v.  (Not inlined: the loops over a thread's tokens are unrolled.)
static __device__ __noinline__ int sequence_of(const int32_t* cu, int N, int end, int v) {
  return min(max(first_border_above(cu, N, end, v) - 1, 0), N - 1);
}
// Bit i: a sequence starts at token t + i, or the last one ends before it (i <= run).
static __device__ __noinline__ unsigned borders_of(const int32_t* cu, int N, int end, int t, int run) {
  int m = first_border_above(cu, N, end, t);
  unsigned bits = m > 0 && min(max(cu[m - 1], 0), end) == t ? 1u : 0u;
  while (m <= N) {
    const int b = min(max(cu[m], 0), end);  // above t, and above the one before
    if (b - t > run) break;
    bits |= 1u << (b - t);
    if (b >= end) break;
    m = first_border_above(cu, N, end, b);
  }
  return bits;
}

// ---- launches --------------------------------------------------------------------------------
// Blocks of a cluster: they go on together through a row's `spans`, and as many clusters as there is room
// for run at once, which depends on the size (of 256 threads at two blocks an SM, 36 clusters of 8 but only
// 14 of 14 fit this GPU).  The size with the fewest rounds over all waves of clusters is taken.  The GPU is
// asked once for each kernel and size.
template <auto kKernel>
cudaError_t choose_cluster(GlrParams* p, unsigned threads, size_t smem, long long spans) {
  static std::atomic<int> room[kGlrMaxCluster + 1];
  const long long units = glr_units(*p);
  long long best = -1;
  const int force = getenv("GLR_K") ? atoi(getenv("GLR_K")) : 0;
  for (int k = 1; k <= kGlrMaxCluster && (k == 1 || k <= spans); ++k) {
    int n = room[k].load(std::memory_order_relaxed);
    if (!n) {
      cudaError_t e = allow_clusters(kKernel, k, smem);
      if (e != cudaSuccess) return e;
      const ClusterConfig c(k, threads, k, smem, nullptr);
      if (k == 1) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kKernel, threads, smem);
        n *= kSms;
      } else {
        e = cudaOccupancyMaxActiveClusters(&n, kKernel, &c.cfg);
      }
      if (e != cudaSuccess) return e;
      n = n < 1 ? -1 : n;
      room[k].store(n, std::memory_order_relaxed);
    }
    if (n < 0) continue;
    // (a wave's start costs about two rounds)
    const long long cost = ((units + n - 1) / n) * ((spans + k - 1) / k + 2);
    if (best < 0 || cost < best || k == force) best = k == force ? 0 : cost, p->cluster = k;
  }
  return best < 0 ? cudaErrorInvalidConfiguration : cudaSuccess;
}

}  // namespace gdn
