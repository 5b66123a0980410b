// glr_common.cuh - what the gated linear recurrence's kernels share: channel pairs, gates,
// sequence borders, and the composition of stretches of time.
//
//   h_t = a_t h_{t-1} + s(a_t) x_t,   a = exp(L):
//   gate      L = g (log), log sigmoid(g) (sigmoid), rate sigmoid(g) (rate)
//   weight    s = 1 (none), 1 - a (linear), sqrt(1 - a^2) (sqrt)
//
// A stretch of tokens maps the state before it to A h + H.  Stretches compose, so time is cut
// everywhere: a thread has kGlrRun tokens of two channels, a warp 64 channels, a block's warps
// follow each other in time, and so do the blocks of a cluster.
#pragma once

#include "cluster.cuh"
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {

constexpr int kGlrRun = kGlrSpan / kGlrWarps;  // tokens of a thread in a round
constexpr float kTiny = 1.17549435e-38f;       // 2^-126

// ---- two channels of a row ---------------------------------------------------------------
// Aligned rows: channels 2 lane, 2 lane + 1 of the 64 in one access; others: channels lane and
// lane + 32 in an access each (so that a warp's accesses are dense).
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
      v = (c0 ? (uint32_t)q[0] : 0u) | (c1 ? (uint32_t)q[32] << 16 : 0u);
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, bool vec, bool c0, bool c1) const {
    if (vec) {
      if (c0) *reinterpret_cast<uint32_t*>(p) = v;
    } else {
      uint16_t* q = reinterpret_cast<uint16_t*>(p);
      if (c0) q[0] = (uint16_t)v;
      if (c1) q[32] = (uint16_t)(v >> 16);
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
  __device__ __forceinline__ void zero() { v = 0u; }
};
template <>
struct Raw2<float> {
  f32x2 v;
  __device__ __forceinline__ void load(const float* p, bool vec, bool c0, bool c1) {
    if (vec) v = c0 ? *reinterpret_cast<const f32x2*>(p) : 0ull;
    else v = pack2(c0 ? p[0] : 0.f, c1 ? p[32] : 0.f);
  }
  __device__ __forceinline__ void store(float* p, bool vec, bool c0, bool c1) const {
    if (vec) {
      if (c0) *reinterpret_cast<f32x2*>(p) = v;
    } else {
      float a, b;
      unpack2(v, a, b);
      if (c0) p[0] = a;
      if (c1) p[32] = b;
    }
  }
  __device__ __forceinline__ f32x2 get() const { return v; }
  __device__ __forceinline__ void set(f32x2 x) { v = x; }
  __device__ __forceinline__ void zero() { v = 0ull; }
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

// ---- gates -------------------------------------------------------------------------------
__device__ __forceinline__ float sqrt_ftz(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
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
// 1 - e^u where e = e^u is known: the difference loses what small |u| have, the series does not.
__device__ __forceinline__ f32x2 one_less(f32x2 u, f32x2 e) {
  float s0, s1, u0, u1, d0, d1;
  unpack2(neg2(expm1_small(u)), s0, s1);
  unpack2(u, u0, u1);
  unpack2(add2(dup2(1.f), neg2(e)), d0, d1);
  return pack2(fabsf(u0) < 0.5f ? s0 : d0, fabsf(u1) < 0.5f ? s1 : d1);
}
// e^-g, at most 2^126 so that its product with sigmoid(g) = 1 / (1 + e^-g) is 1 - sigmoid(g)
// for every g
__device__ __forceinline__ f32x2 exp_neg(f32x2 g) {
  return each(mul2(g, dup2(-kLog2e)), [](float v) { return ex2(min_nan(v, 126.f)); });
}
__device__ __forceinline__ f32x2 rcp2(f32x2 x) {
  return each(x, [](float v) { return rcp(v); });
}

// The decay a and the input's weight s of a token.
template <int kGate, int kNorm>
__device__ __forceinline__ void gate2(f32x2 g, f32x2 rate, f32x2& a, f32x2& s) {
  const auto root = [](f32x2 v) { return each(v, [](float x) { return sqrt_ftz(x); }); };
  s = dup2(1.f);
  if (kGate == GLR_SIGMOID) {
    const f32x2 e = exp_neg(g);
    a = rcp2(add2(e, dup2(1.f)));
    const f32x2 left = mul2(e, a);  // 1 - a
    if (kNorm == GLR_LINEAR) s = left;
    if (kNorm == GLR_SQRT) s = root(fma2(left, a, left));
  } else {
    const f32x2 log = kGate == GLR_LOG ? g : mul2(rate, rcp2(add2(exp_neg(g), dup2(1.f))));
    a = each(mul2(log, dup2(kLog2e)), [](float v) { return ex2(v); });
    if (kNorm == GLR_LINEAR) s = one_less(log, a);
    if (kNorm == GLR_SQRT) s = root(one_less(add2(log, log), mul2(a, a)));
  }
}

// ---- stretches of time ---------------------------------------------------------------------
// A product of decays that underflows stays at 2^-126: an infinite state before it stays infinite,
// as it does token by token, and of finite ones nothing is left either way.  A = 0 is a border: what
// lies behind it sees nothing from before, not even infinities.
__device__ __forceinline__ f32x2 at_least_tiny(f32x2 a) {
  return each(a, [](float v) { return fmaxf(v, kTiny); });
}
__device__ __forceinline__ f32x2 through(f32x2 A, f32x2 H, f32x2 h) {  // A h + H
  float a0, a1, b0, b1, r0, r1;
  unpack2(A, a0, a1);
  unpack2(H, b0, b1);
  unpack2(fma2(A, h, H), r0, r1);
  return pack2(a0 == 0.f ? b0 : r0, a1 == 0.f ? b1 : r1);
}
// (A, H) followed by (B, G)
__device__ __forceinline__ void follow(f32x2& A, f32x2& H, f32x2 B, f32x2 G) {
  H = through(B, G, H);
  float a0, a1, b0, b1;
  unpack2(A, a0, a1);
  unpack2(B, b0, b1);
  A = pack2(a0 == 0.f || b0 == 0.f ? 0.f : fmaxf(a0 * b0, kTiny),
            a1 == 0.f || b1 == 0.f ? 0.f : fmaxf(a1 * b1, kTiny));
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
// The sequence that holds token v.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int N, int end, int v) {
  return min(max(first_border_above(cu, N, end, v) - 1, 0), N - 1);
}
// Bit i: a sequence starts at token t + i, or the last one ends before it (i <= kGlrRun).
__device__ __forceinline__ unsigned borders_of(const int32_t* cu, int N, int end, int t) {
  int m = first_border_above(cu, N, end, t);
  unsigned bits = m > 0 && min(max(cu[m - 1], 0), end) == t ? 1u : 0u;
  while (m <= N) {
    const int b = min(max(cu[m], 0), end);  // above t, and above the one before
    if (b - t > kGlrRun) break;
    bits |= 1u << (b - t);
    if (b >= end) break;
    m = first_border_above(cu, N, end, b);
  }
  return bits;
}

}  // namespace gdn
