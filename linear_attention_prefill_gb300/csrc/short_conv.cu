// short_conv.cu - the short causal convolution that a linear-attention layer applies to its
// projections before the forward (q, k, v of GDN and KDA; x, B, C of the SSD scan; x of S6),
// for prompts and for single tokens.
//
// Per channel d and token t of a sequence, W taps (2 to 4):
//   y_t = act(bias + sum_j w[d, j] x_{t - W + 1 + j}),   act = identity or SiLU,
// where the W - 1 inputs before the sequence come from its state s0 (zeros without one) and
// the last W - 1 inputs become the state sT.  Sums in fp32, one rounding at the end.
//
// HBM bandwidth bounds it: 2 bytes in and 2 out per element against ~8 instructions.  A
// thread has 4 channels (8 bytes of bf16) and walks a run of tokens with the window in
// registers as packed fp32 pairs, so that each input is loaded once except for the W - 1 rows
// before a run.  Its own inputs come by cp.async through a private ring of shared memory, three
// rounds of four tokens ahead: what is in flight then costs no registers (loads ahead in
// registers, one round: 22.4 us at 4096 x 6144 where the ring takes CONV_RING).  Rows off
// 4-channel pieces are loaded element by element, one round ahead.
#include "gdn_common.cuh"
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {
namespace {

constexpr int kVec4 = 4;      // channels per thread
constexpr int kThreads = 128;
constexpr int kAhead = 4;     // tokens of a round
constexpr int kRounds = 4;    // rounds of the ring

// Four channels of a row in fp32.
struct Four {
  f32x2 lo, hi;
};
template <typename T>
__device__ __forceinline__ Four four(const Raw4<T>& r) {
  const float4 v = r.get();
  return {pack2(v.x, v.y), pack2(v.z, v.w)};
}

// The filters of channels c..c+3, tap by tap: w is [D, W] and c a multiple of 4, so the 4 W
// floats are whole 16-byte pieces.
template <int W>
__device__ __forceinline__ void load_filter(const float* w, int c, int n, Four (&f)[W]) {
  float v[kVec4 * W];
  if (n >= kVec4) {
    const float4* p = reinterpret_cast<const float4*>(w + (long long)c * W);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float4 q = p[i];
      v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec4 * W; ++i) v[i] = i / W < n ? w[(long long)c * W + i] : 0.f;
  }
#pragma unroll
  for (int j = 0; j < W; ++j) f[j] = {pack2(v[j], v[W + j]), pack2(v[2 * W + j], v[3 * W + j])};
}
__device__ __forceinline__ Four load_bias(const float* bias, int c, int n) {
  float b[kVec4];
#pragma unroll
  for (int i = 0; i < kVec4; ++i) b[i] = bias && i < n ? bias[c + i] : 0.f;
  return {pack2(b[0], b[1]), pack2(b[2], b[3])};
}
// act(bias + sum of taps), rounded
template <typename T, int W>
__device__ __forceinline__ Raw4<T> filter(const Four (&f)[W], const Four& bias, const Four (&win)[W],
                                          int act) {
  Four a = bias;
#pragma unroll
  for (int j = 0; j < W; ++j) {
    a.lo = fma2(f[j].lo, win[j].lo, a.lo);
    a.hi = fma2(f[j].hi, win[j].hi, a.hi);
  }
  if (act) {
    a.lo = silu2(a.lo);
    a.hi = silu2(a.hi);
  }
  float v0, v1, v2, v3;
  unpack2(a.lo, v0, v1);
  unpack2(a.hi, v2, v3);
  Raw4<T> o;
  o.set(v0, v1, v2, v3);
  return o;
}

// A sequence's tokens in the packed (or row-major) batch, clamped to the batch so that no
// border read from the device leads outside of it.
struct Span {
  long long begin, end;
};
__device__ __forceinline__ Span span_of(const ConvParams& p, int n) {
  if (!p.cu) return {(long long)n * p.T, (long long)(n + 1) * p.T};
  const long long b = min(max(p.cu[n], 0), p.T), e = min(max(p.cu[n + 1], 0), p.T);
  return {b, max(b, e)};
}

// Row of the window of a token of sequence n, t = an absolute row: an input, or the state.
template <typename T, int W>
__device__ __forceinline__ Raw4<T> tap(const ConvParams& p, const Span& s, int n, long long t,
                                       int c, int left, bool vec) {
  Raw4<T> r;
  if (t >= s.begin) {
    r.load(static_cast<const T*>(p.x) + t * p.x_stride + c, left, vec);
  } else if (p.s0) {
    r.load(static_cast<const T*>(p.s0) +
               ((long long)n * (W - 1) + (W - 1) + (t - s.begin)) * p.D + c,
           left, vec);
  } else {
    r.zero();
  }
  return r;
}

// State of sequence n after its tokens: the last W - 1 rows of [s0; x].
template <typename T, int W>
__device__ __forceinline__ void write_state(const ConvParams& p, int n, int c, int left, bool vec) {
  const Span s = span_of(p, n);
  Raw4<T> r[W - 1];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) r[j] = tap<T, W>(p, s, n, s.end - (W - 1) + j, c, left, vec);
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    r[j].store(static_cast<T*>(p.sT) + ((long long)n * (W - 1) + j) * p.D + c, left, vec);
}

// cp.async of one thread's four channels
__device__ __forceinline__ void copy_four(Raw4<__nv_bfloat16>* dst, const __nv_bfloat16* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_four(Raw4<float>* dst, const float* src) {
  cp_async16(dst, src, true);
}

// blockIdx.x: run of `run` tokens, then (with sT) one sequence's state each; blockIdx.y: 128
// threads of 4 channels.  kVec: whole aligned pieces.
template <typename T, int W, bool kVec>
__global__ void __launch_bounds__(kThreads) conv_kernel(const ConvParams p, int run, int runs,
                                                        long long tokens) {
  __shared__ __align__(16) unsigned char s_ring[kVec ? kRounds * kAhead * kThreads * sizeof(Raw4<T>) : 16];
  const int c = (blockIdx.y * kThreads + threadIdx.x) * kVec4;
  if (c >= p.D) return;
  const int left = p.D - c;
  constexpr bool vec = kVec;
  if ((int)blockIdx.x >= runs) {
    write_state<T, W>(p, blockIdx.x - runs, c, left, vec);
    return;
  }
  const long long t0 = (long long)blockIdx.x * run, t1 = min(t0 + run, tokens);
  const T* x = static_cast<const T*>(p.x) + t0 * p.x_stride + c;
  T* y = static_cast<T*>(p.y) + t0 * p.D + c;
  Raw4<T> ahead[kVec ? 1 : kAhead];  // the tokens of the next round
  Raw4<T>* ring = reinterpret_cast<Raw4<T>*>(s_ring) + threadIdx.x;
  const int len = (int)(t1 - t0);
  auto request = [&](int round) {  // this thread's inputs of a round, x at its first token
    if constexpr (kVec) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (round * kAhead + u < len)
          copy_four(ring + (round % kRounds * kAhead + u) * kThreads, x + u * p.x_stride);
      cp_async_commit();
    } else {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (round * kAhead + u < len) ahead[u].load(x + u * p.x_stride, left, false);
    }
    x += kAhead * p.x_stride;
  };
#pragma unroll
  for (int round = 0; round < (kVec ? kRounds - 1 : 1); ++round) request(round);

  // the sequence of token t0: the first one that ends behind it
  int n = 0;
  if (p.cu) {
    int lo = 0, hi = p.N;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (min(max(p.cu[mid + 1], 0), p.T) > t0) hi = mid; else lo = mid + 1;
    }
    n = lo;
  } else {
    n = (int)(t0 / p.T);
  }
  if (n >= p.N) return;  // behind the last sequence: left as it was
  Span s = span_of(p, n);

  Four f[W], win[W];  // the filter, and the inputs under it
  load_filter<W>(p.w, c, left, f);
  const Four bias = load_bias(p.bias, c, left);
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    win[j] = four(tap<T, W>(p, s, n, max(t0, s.begin) - (W - 1) + j, c, left, vec));

  int round = 0;
  for (long long t = t0; t < t1; t += kAhead, ++round) {
    Raw4<T> raw[kAhead];
    if constexpr (kVec) {
      request(round + kRounds - 1);
      cp_async_wait<kRounds - 1>();
#pragma unroll
      for (int u = 0; u < kAhead; ++u) raw[u] = ring[(round % kRounds * kAhead + u) * kThreads];
    } else {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) raw[u] = ahead[u];
      request(round + 1);
    }
    if (t >= s.begin && t + kAhead <= min(t1, s.end)) {  // one sequence's tokens
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        win[W - 1] = four(raw[u]);
        filter<T, W>(f, bias, win, p.silu).store(y + (long long)u * p.D, left, vec);
#pragma unroll
        for (int j = 0; j + 1 < W; ++j) win[j] = win[j + 1];
      }
    } else {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const long long tt = t + u;
        if (tt >= t1) return;
        if (tt >= s.end) {  // the next sequence that has tokens begins
          do {
            if (++n >= p.N) return;
            s = span_of(p, n);
          } while (tt >= s.end);
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
            win[j] = four(tap<T, W>(p, s, n, max(tt, s.begin) - (W - 1) + j, c, left, vec));
        }
        if (tt < s.begin) continue;
        win[W - 1] = four(raw[u]);
        filter<T, W>(f, bias, win, p.silu).store(y + (long long)u * p.D, left, vec);
#pragma unroll
        for (int j = 0; j + 1 < W; ++j) win[j] = win[j + 1];
      }
    }
    y += kAhead * (long long)p.D;
  }
}

// The states alone, after conv_kernel: for a state that is updated in place (another block
// of conv_kernel may still read it), or a batch without tokens.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_state_kernel(const ConvParams p) {
  const int c = (blockIdx.y * kThreads + threadIdx.x) * kVec4;
  if (c < p.D) write_state<T, W>(p, blockIdx.x, c, p.D - c, p.vec);
}

// One token per sequence: a thread holds the windows of 4 channels of kSeqs sequences and
// shifts their states in place.  kSeqs > 1 shares the filter, which is as many bytes as the
// window and the output of one sequence.
template <typename T, int W, int kSeqs>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const ConvParams p, int per_row) {
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long first = id / per_row * kSeqs;
  if (first >= p.N) return;
  const int c = (int)(id % per_row) * kVec4;
  const int left = p.D - c;
  const bool vec = p.vec;
  Raw4<T> r[kSeqs][W];
#pragma unroll
  for (int i = 0; i < kSeqs; ++i) {
    if (first + i >= p.N) break;
    const T* s = static_cast<const T*>(p.sT) + (first + i) * (W - 1) * p.D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[i][j].load(s + (long long)j * p.D, left, vec);
    r[i][W - 1].load(static_cast<const T*>(p.x) + (first + i) * p.x_stride + c, left, vec);
  }
  Four f[W];
  load_filter<W>(p.w, c, left, f);
  const Four bias = load_bias(p.bias, c, left);
#pragma unroll
  for (int i = 0; i < kSeqs; ++i) {
    if (first + i >= p.N) break;
    Four win[W];
#pragma unroll
    for (int j = 0; j < W; ++j) win[j] = four(r[i][j]);
    filter<T, W>(f, bias, win, p.silu)
        .store(static_cast<T*>(p.y) + (first + i) * p.D + c, left, vec);
    T* s = static_cast<T*>(p.sT) + (first + i) * (W - 1) * p.D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[i][j + 1].store(s + (long long)j * p.D, left, vec);
  }
}

template <typename T, int W>
cudaError_t launch_w(const ConvParams& p, cudaStream_t stream) {
  const long long tokens = p.cu ? (long long)p.T : (long long)p.N * p.T;
  const int per_row = (p.D + kVec4 - 1) / kVec4;
  const unsigned by = (per_row + kThreads - 1) / kThreads;
  // long runs repeat fewer rows (W - 1 each), short ones fill the GPU: 8 blocks per SM
  int run = 64;
  while (run > kAhead && (tokens + run - 1) / run * by < 8 * kSms) run /= 2;
  const long long runs = (tokens + run - 1) / run;
  // sT == s0: the states wait for every block that reads them
  const bool apart = p.sT && (p.s0 == p.sT || tokens == 0);
  const long long bx = runs + (p.sT && !apart ? p.N : 0);
  if (tokens > 0) {
    const dim3 grid((unsigned)bx, by);
    if (p.vec) conv_kernel<T, W, true><<<grid, kThreads, 0, stream>>>(p, run, (int)runs, tokens);
    else conv_kernel<T, W, false><<<grid, kThreads, 0, stream>>>(p, run, (int)runs, tokens);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (apart)
    conv_state_kernel<T, W><<<dim3((unsigned)p.N, by), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const ConvParams& p, cudaStream_t stream) {
  if (p.W == 4) return launch_w<T, 4>(p, stream);
  if (p.W == 3) return launch_w<T, 3>(p, stream);
  return launch_w<T, 2>(p, stream);
}

template <typename T, int W>
cudaError_t launch_step_w(const ConvParams& p, cudaStream_t stream) {
  const int per_row = (p.D + kVec4 - 1) / kVec4;
  const auto blocks = [&](int seqs) {
    return (unsigned)(((long long)((p.N + seqs - 1) / seqs) * per_row + kThreads - 1) / kThreads);
  };
  // two sequences a thread once that still leaves 8 blocks per SM
  if (blocks(2) >= 8 * kSms)
    conv_step_kernel<T, W, 2><<<blocks(2), kThreads, 0, stream>>>(p, per_row);
  else
    conv_step_kernel<T, W, 1><<<blocks(1), kThreads, 0, stream>>>(p, per_row);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_step_t(const ConvParams& p, cudaStream_t stream) {
  if (p.W == 4) return launch_step_w<T, 4>(p, stream);
  if (p.W == 3) return launch_step_w<T, 3>(p, stream);
  return launch_step_w<T, 2>(p, stream);
}

}  // namespace

cudaError_t launch_conv(const ConvParams& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_t<float>(p, stream) : launch_t<__nv_bfloat16>(p, stream);
}
cudaError_t launch_conv_step(const ConvParams& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_step_t<float>(p, stream) : launch_step_t<__nv_bfloat16>(p, stream);
}

}  // namespace gdn
