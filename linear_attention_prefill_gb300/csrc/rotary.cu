// rotary.cu - rotary positions of q and k.
//
//   pair i of a head's first R columns: (x, y) -> m (x cos - y sin, y cos + x sin),
//   angle = position turns[i] of a whole turn; backwards the turn is undone (its transpose)
//
// turns[i] is a frequency as a fraction of a turn in 64-bit fixed point, so position times turns[i]
// modulo 2^64 is the angle modulo one turn, exactly, at any position; of an fp32 angle at position
// 2^20 only 4 bits behind the point would be left.  A block takes a few tokens: it makes their
// cosines and sines once, a pair a thread, and walks all heads of q and k with them, in one launch.
// The first loads are under way meanwhile.  Every element crosses HBM once each way; loads in flight bound it
// (q and k of 4096 tokens, 16 heads of 128 in bf16: 16 us, 4.2 TB/s).  Products are fp32, rounded once.
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {
namespace {

// V elements of an access, 2 to 16 bytes.
template <int kBytes>
struct Access;
template <>
struct Access<16> { using type = uint4; };
template <>
struct Access<8> { using type = uint2; };
template <>
struct Access<4> { using type = uint32_t; };
template <>
struct Access<2> { using type = uint16_t; };
template <typename T, int V>
struct Piece {
  using Word = typename Access<V * sizeof(T)>::type;
  union {
    Word word;
    T e[V];
    uint32_t pair[V * sizeof(T) < 4 ? 1 : V * sizeof(T) / 4];
  };
  __device__ __forceinline__ Piece() {}
  __device__ __forceinline__ void load(const T* p) { word = *reinterpret_cast<const Word*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Word*>(p) = word; }
  // (pairs of bf16 as halves of a register)
  __device__ __forceinline__ void get(float (&o)[V]) const {
    if constexpr (sizeof(T) == 2 && V > 1) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        o[2 * i] = __uint_as_float(pair[i] << 16);
        o[2 * i + 1] = __uint_as_float(pair[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = to_f32(e[i]);
    }
  }
  __device__ __forceinline__ void set(const float (&o)[V]) {
    if constexpr (sizeof(T) == 2 && V > 1) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pair[i]) : "f"(o[2 * i + 1]), "f"(o[2 * i]));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) from_f32(e + i, o[i]);
    }
  }
};

// The position of a token, counted over the whole batch; false: behind the last sequence.
__device__ __forceinline__ bool position_of(const RotaryParams& p, long long token, long long* at) {
  if (p.positions) {
    *at = p.positions[token];
    return true;
  }
  long long n, first;
  if (p.cu) {  // the last sequence that starts at or before the token
    if (token >= p.cu[p.N]) return false;
    int lo = 0, hi = p.N;
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (p.cu[mid] <= token) lo = mid; else hi = mid;
    }
    n = lo;
    first = p.cu[lo];
  } else {
    n = (unsigned)token / (unsigned)p.T;  // (tokens fit 31 bits)
    first = n * p.T;
  }
  *at = token - first + (p.offsets ? p.offsets[n] : 0);
  return true;
}

// blockDim.x threads of a head: R / 2 / V of them have V pairs each, the others 2 V columns that are
// passed through.  blockDim.y is the block's tokens times some heads of each: a thread stays with its
// token, whose cosines and sines it keeps, and takes every so many of its heads, kAhead loads ahead.
constexpr int kRotaryThreads = 128, kAhead = 4;
template <typename T, int V, bool kNext>
__global__ void __launch_bounds__(V > 1 ? 256 : 512, V > 1 ? 3 : 1) rotary_kernel(const RotaryParams p) {
  extern __shared__ __align__(16) float2 s_turn[];  // [tokens of the block][R / 2]: m cos, m sin
  const int half = p.R / 2, pairs = half / V;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
  const long long token0 = (long long)blockIdx.x * p.block_tokens;
  const int here = (int)min((long long)p.block_tokens, p.tokens - token0);
  const bool rotates = (int)threadIdx.x < pairs;
  // the thread's two pieces of a head
  const int rest = p.R + ((int)threadIdx.x - pairs) * 2 * V;
  const int at0 = rotates ? (kNext ? 2 : 1) * V * (int)threadIdx.x : rest;
  const int at1 = rotates ? (kNext ? at0 + V : at0 + half) : rest + V;
  const bool two = rotates || at1 < p.D;
  const long long end = p.cu && !p.positions ? min((long long)p.cu[p.N], p.tokens) : p.tokens;
  const int mine = threadIdx.y % p.block_tokens, step = blockDim.y / p.block_tokens;
  const long long t = token0 + mine;
  const int heads = mine < here && t < end ? p.Hq + p.Hk : 0;

  const T* q = static_cast<const T*>(p.q) + t * p.q_stride;
  const T* k = static_cast<const T*>(p.k) + t * p.k_stride - (long long)p.Hq * p.D;
  T* q_out = static_cast<T*>(p.q_out) + t * p.q_out_stride;
  T* k_out = static_cast<T*>(p.k_out) + t * p.k_out_stride - (long long)p.Hq * p.D;
  // passed through in place already
  const auto moves = [&](int h) { return h < heads && (rotates || !(h < p.Hq ? p.q_same : p.k_same)); };
  Piece<T, V> a[kAhead], b[kAhead];
  const auto load = [&](int first) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = first + i * step;
      if (!moves(h)) continue;
      const T* x = (h < p.Hq ? q : k) + (long long)h * p.D;
      a[i].load(x + at0);
      if (two) b[i].load(x + at1);
    }
  };
  int h0 = threadIdx.y / p.block_tokens;
  load(h0);
  for (int i = tid; i < here * half; i += threads) {
    const int j = i / half;
    long long at = 0;
    float2 cs = make_float2(1.f, 0.f);
    if (position_of(p, token0 + j, &at)) {
      const unsigned long long turn = p.turns[i - j * half] * (unsigned long long)at + 0x80000000ull;
      float s, c;
      sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &c);  // [-1, 1) half turns
      cs = make_float2(p.magnitude * c, p.magnitude * (p.backward ? -s : s));
    }
    s_turn[i] = cs;
  }
  __syncthreads();
  float2 cs[V];
#pragma unroll
  for (int j = 0; j < V; ++j) cs[j] = rotates ? s_turn[mine * half + threadIdx.x * V + j] : make_float2(1.f, 0.f);
  while (h0 < heads) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = h0 + i * step;
      if (!moves(h)) continue;
      T* out = (h < p.Hq ? q_out : k_out) + (long long)h * p.D;
      if (rotates) {
        float x[V], y[V], u[V], v[V];
        a[i].get(x);
        b[i].get(y);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          // neighbours: x and y are 2 V columns in a row, pair j is columns 2 j, 2 j + 1 of them
          const float2 r = cs[j];
          const float e = kNext ? (2 * j < V ? x[(2 * j) % V] : y[(2 * j) % V]) : x[j];
          const float f = kNext ? (2 * j + 1 < V ? x[(2 * j + 1) % V] : y[(2 * j + 1) % V]) : y[j];
          const float g = e * r.x - f * r.y, h = f * r.x + e * r.y;
          if (kNext) {
            (2 * j < V ? u[(2 * j) % V] : v[(2 * j) % V]) = g;
            (2 * j + 1 < V ? u[(2 * j + 1) % V] : v[(2 * j + 1) % V]) = h;
          } else {
            u[j] = g;
            v[j] = h;
          }
        }
        a[i].set(u);
        b[i].set(v);
      }
      a[i].store(out + at0);
      if (two) b[i].store(out + at1);
    }
    h0 += kAhead * step;
    load(h0);
  }
}

template <typename T, int V>
cudaError_t launch(RotaryParams p, cudaStream_t stream) {
  const int half = p.R / 2, heads = p.Hq + p.Hk;
  const int x = half / V + (p.D - p.R + 2 * V - 1) / (2 * V), rows = kRotaryThreads / x > 1 ? kRotaryThreads / x : 1;
  // a thread has about kAhead heads, the block as many tokens as that leaves room for; but for fewer
  // tokens than two blocks an SM would have, a token a block with all its rows of threads
  int step = (heads + kAhead - 1) / kAhead;
  if (step > rows || p.tokens < 2 * kSms) step = rows < heads ? rows : heads;
  long long tokens = rows / step;
  if (tokens > p.tokens / (2 * kSms)) tokens = p.tokens / (2 * kSms);
  if (tokens < 1) tokens = 1;
  p.block_tokens = (int)tokens;
  const long long grid = (p.tokens + tokens - 1) / tokens;
  const size_t smem = (size_t)tokens * half * sizeof(float2);
  const dim3 block(x, (unsigned)(tokens * step));
  if (p.interleaved)
    rotary_kernel<T, V, true><<<(unsigned)grid, block, smem, stream>>>(p);
  else
    rotary_kernel<T, V, false><<<(unsigned)grid, block, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, bool f32, cudaStream_t stream) {
  if (f32)
    return p.by == 4 ? launch<float, 4>(p, stream) : p.by == 2 ? launch<float, 2>(p, stream)
                                                               : launch<float, 1>(p, stream);
  return p.by == 8   ? launch<__nv_bfloat16, 8>(p, stream)
         : p.by == 4 ? launch<__nv_bfloat16, 4>(p, stream)
         : p.by == 2 ? launch<__nv_bfloat16, 2>(p, stream)
                     : launch<__nv_bfloat16, 1>(p, stream);
}

}  // namespace gdn
