// layer_common.cuh - device helpers of the layer operators around the forwards (short
// convolution, S6 scan, RMS norm): 8-element rows of bf16 or fp32, packed fp32 pairs,
// and the activations in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;

// ---- element types ---------------------------------------------------------------
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Eight consecutive elements as they are stored: 16 bytes of bf16, 32 of fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void set(const float (&o)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(o[2 * i + 1]), "f"(o[2 * i]));
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
  // the first n of 8, n a multiple of the `by` (4, 2 or 1) elements of an access; the others read
  // as zero
  __device__ __forceinline__ void load_by(const __nv_bfloat16* p, int n, int by) {
    if (by == 1) {
      load_n(p, n);
    } else if (by == 2) {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
      v = make_uint4(n > 0 ? q[0] : 0u, n > 2 ? q[1] : 0u, n > 4 ? q[2] : 0u, n > 6 ? q[3] : 0u);
    } else {
      const uint2 zero = make_uint2(0u, 0u);
      const uint2 a = n > 0 ? *reinterpret_cast<const uint2*>(p) : zero;
      const uint2 b = n > 4 ? *reinterpret_cast<const uint2*>(p + 4) : zero;
      v = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
  __device__ __forceinline__ void store_by(__nv_bfloat16* p, int n, int by) const {
    if (by == 1) {
      store_n(p, n);
    } else if (by == 2) {
      uint32_t* q = reinterpret_cast<uint32_t*>(p);
      if (n > 0) q[0] = v.x;
      if (n > 2) q[1] = v.y;
      if (n > 4) q[2] = v.z;
      if (n > 6) q[3] = v.w;
    } else {
      if (n > 0) *reinterpret_cast<uint2*>(p) = make_uint2(v.x, v.y);
      if (n > 4) *reinterpret_cast<uint2*>(p + 4) = make_uint2(v.z, v.w);
    }
  }
  // element by element, the first n of 8 (n <= 0: none); the others read as zero
  __device__ __forceinline__ void load_n(const __nv_bfloat16* p, int n) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < n ? q[2 * i] : 0u, hi = 2 * i + 1 < n ? q[2 * i + 1] : 0u;
      w[i] = lo | (hi << 16);
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store_n(__nv_bfloat16* p, int n) const {
    uint16_t* q = reinterpret_cast<uint16_t*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
  }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void get(float (&o)[8]) const {
    o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w;
    o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&o)[8]) {
    a = make_float4(o[0], o[1], o[2], o[3]);
    b = make_float4(o[4], o[5], o[6], o[7]);
  }
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void load_by(const float* p, int n, int by) {
    if (by == 1) {
      load_n(p, n);
    } else if (by == 2) {
      const float2* q = reinterpret_cast<const float2*>(p);
      const float2 zero = make_float2(0.f, 0.f);
      const float2 c = n > 0 ? q[0] : zero, d = n > 2 ? q[1] : zero;
      const float2 e = n > 4 ? q[2] : zero, f = n > 6 ? q[3] : zero;
      a = make_float4(c.x, c.y, d.x, d.y);
      b = make_float4(e.x, e.y, f.x, f.y);
    } else {
      const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
      a = n > 0 ? reinterpret_cast<const float4*>(p)[0] : zero;
      b = n > 4 ? reinterpret_cast<const float4*>(p)[1] : zero;
    }
  }
  __device__ __forceinline__ void store_by(float* p, int n, int by) const {
    if (by == 1) {
      store_n(p, n);
    } else if (by == 2) {
      float2* q = reinterpret_cast<float2*>(p);
      if (n > 0) q[0] = make_float2(a.x, a.y);
      if (n > 2) q[1] = make_float2(a.z, a.w);
      if (n > 4) q[2] = make_float2(b.x, b.y);
      if (n > 6) q[3] = make_float2(b.z, b.w);
    } else {
      if (n > 0) reinterpret_cast<float4*>(p)[0] = a;
      if (n > 4) reinterpret_cast<float4*>(p)[1] = b;
    }
  }
  __device__ __forceinline__ void load_n(const float* p, int n) {
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = i < n ? p[i] : 0.f;
    set(o);
  }
  __device__ __forceinline__ void store_n(float* p, int n) const {
    float o[8];
    get(o);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = o[i];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
};
// Four consecutive elements as they are stored: 8 bytes of bf16, 16 of fp32.
template <typename T>
struct Raw4;
template <>
struct Raw4<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void zero() { v = make_uint2(0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int n, bool vec) {
    if (vec) {
      v = *reinterpret_cast<const uint2*>(p);
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
      v.x = (n > 0 ? q[0] : 0u) | (n > 1 ? (uint32_t)q[1] << 16 : 0u);
      v.y = (n > 2 ? q[2] : 0u) | (n > 3 ? (uint32_t)q[3] << 16 : 0u);
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, int n, bool vec) const {
    if (vec) {
      *reinterpret_cast<uint2*>(p) = v;
    } else {
      uint16_t* q = reinterpret_cast<uint16_t*>(p);
      if (n > 0) q[0] = (uint16_t)v.x;
      if (n > 1) q[1] = (uint16_t)(v.x >> 16);
      if (n > 2) q[2] = (uint16_t)v.y;
      if (n > 3) q[3] = (uint16_t)(v.y >> 16);
    }
  }
  __device__ __forceinline__ float4 get() const {
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  }
  __device__ __forceinline__ void set(float a, float b, float c, float d) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.x) : "f"(b), "f"(a));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.y) : "f"(d), "f"(c));
  }
};
template <>
struct Raw4<float> {
  float4 v;
  __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p, int n, bool vec) {
    if (vec) v = *reinterpret_cast<const float4*>(p);
    else v = make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
  }
  __device__ __forceinline__ void store(float* p, int n, bool vec) const {
    if (vec) {
      *reinterpret_cast<float4*>(p) = v;
    } else {
      if (n > 0) p[0] = v.x;
      if (n > 1) p[1] = v.y;
      if (n > 2) p[2] = v.z;
      if (n > 3) p[3] = v.w;
    }
  }
  __device__ __forceinline__ float4 get() const { return v; }
  __device__ __forceinline__ void set(float a, float b, float c, float d) {
    v = make_float4(a, b, c, d);
  }
};
// Eight elements as four packed pairs, and back.
__device__ __forceinline__ void pairs_of(const Raw8<__nv_bfloat16>& r, unsigned long long (&o)[4]) {
  const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("mov.b64 %0, {%1, %2};" : "=l"(o[i]) : "r"(w[i] << 16), "r"(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void pairs_of(const Raw8<float>& r, unsigned long long (&o)[4]) {
  asm("mov.b64 %0, {%1, %2};" : "=l"(o[0]) : "f"(r.a.x), "f"(r.a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(o[1]) : "f"(r.a.z), "f"(r.a.w));
  asm("mov.b64 %0, {%1, %2};" : "=l"(o[2]) : "f"(r.b.x), "f"(r.b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(o[3]) : "f"(r.b.z), "f"(r.b.w));
}
template <typename T>
__device__ __forceinline__ Raw8<T> raw_of(const unsigned long long (&v)[4]) {
  float o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o[2 * i]), "=f"(o[2 * i + 1]) : "l"(v[i]));
  Raw8<T> r;
  r.set(o);
  return r;
}
// The first n of 8 elements at p in accesses of `by` elements (8, 4, 2 or 1): p is aligned to
// them (at most 16 bytes) and n a multiple of `by`, or larger.
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p, int n, int by) {
  Raw8<T> r;
  if (by == 8) r.load(p); else r.load_by(p, n, by);
  return r;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const Raw8<T>& r, int n, int by) {
  if (by == 8) r.store(p); else r.store_by(p, n, by);
}

// Four states of the recurrence (n of them exist): rows of Ns floats, 16-byte aligned bases.
__device__ __forceinline__ float4 load_h(const float* p, int n, int Ns) {
  if ((Ns & 3) == 0) return n > 0 ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
  return make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f,
                     n > 3 ? p[3] : 0.f);
}
__device__ __forceinline__ void store_h(float* p, float4 v, int n, int Ns) {
  if ((Ns & 3) == 0) {
    if (n > 0) *reinterpret_cast<float4*>(p) = v;
    return;
  }
  if (n > 0) p[0] = v.x;
  if (n > 1) p[1] = v.y;
  if (n > 2) p[2] = v.z;
  if (n > 3) p[3] = v.w;
}

// ---- fp32 arithmetic ---------------------------------------------------------------
__device__ __forceinline__ float ex2(float x) {  // 2^x: max 1.4e-7 relative, subnormals flushed
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// x sigmoid(x) = x / (1 + 2^(-x log2 e)); x -> -inf gives -inf * 0 = NaN as the quotient does
__device__ __forceinline__ float silu(float x) { return x * rcp(1.f + ex2(-kLog2e * x)); }

// Two fp32 values in one 64-bit register, the operand of the packed fp32 instructions.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 dup2(float x) { return pack2(x, x); }

// x sigmoid(x) of two values
__device__ __forceinline__ f32x2 silu2(f32x2 x) {
  float e0, e1;
  unpack2(mul2(x, dup2(-kLog2e)), e0, e1);
  unpack2(add2(pack2(ex2(e0), ex2(e1)), dup2(1.f)), e0, e1);
  return mul2(x, pack2(rcp(e0), rcp(e1)));
}

// softplus(x) = max(x, 0) + log1p(u), u = exp(-|x|) in (0, 1], of two values at once.
// log1p(u) = u P(u), P the polynomial of degree 8 with the least relative error on (0, 1]
// (3.0e-8, by Remez's exchange; 1.7e-7 with the roundings): a small u keeps its relative
// accuracy, which log(1 + u) does not.
__device__ __forceinline__ f32x2 softplus2(f32x2 x) {
  float x0, x1;
  unpack2(x, x0, x1);
  const f32x2 u = pack2(ex2(-kLog2e * fabsf(x0)), ex2(-kLog2e * fabsf(x1)));
  f32x2 r = dup2(0.0052326942f);
  r = fma2(r, u, dup2(-0.029505238f));
  r = fma2(r, u, dup2(0.078225952f));
  r = fma2(r, u, dup2(-0.13663246f));
  r = fma2(r, u, dup2(0.19106007f));
  r = fma2(r, u, dup2(-0.24842982f));
  r = fma2(r, u, dup2(0.33319097f));
  r = fma2(r, u, dup2(-0.49999493f));
  r = fma2(r, u, dup2(0.99999997f));
  return fma2(r, u, pack2(fmaxf(x0, 0.f), fmaxf(x1, 0.f)));
}
__device__ __forceinline__ float softplus(float x) {
  float lo, hi;
  unpack2(softplus2(dup2(x)), lo, hi);
  return lo;
}

}  // namespace gdn
