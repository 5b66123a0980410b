// short_conv.cu - the short causal convolution that a linear-attention layer applies to its
// projections before the forward (q, k, v of GDN and KDA; x, B, C of the SSD scan; x of S6),
// for prompts and for single tokens.
//
// Per channel d and token t of a sequence, W taps (2 to 4):
//   y_t = act(bias + sum_j w[d, j] x_{t - W + 1 + j}),   act = identity or SiLU,
// where the W - 1 inputs before the sequence come from its state s0 (zeros without one) and
// the last W - 1 inputs become the state sT.  Sums in fp32, one rounding at the end.
//
// HBM bandwidth bounds it: 2 bytes in and 2 out per element against ~12 instructions.  A
// thread keeps 8 channels (one 16-byte access) and walks a run of tokens with the window in
// registers, so that each input is loaded once except for the W - 1 rows before a run.
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {
namespace {

constexpr int kVec = 8;       // channels per thread
constexpr int kThreads = 128;
constexpr int kUnroll = 4;    // tokens whose loads are in flight together

// The filters of channels c..c+7: w is [D, W] and c a multiple of 8, so the 8 W floats are
// whole 16-byte pieces.
template <int W>
__device__ __forceinline__ void load_filter(const float* w, int c, int n, float (&f)[kVec][W]) {
  if (n >= kVec) {
    const float4* p = reinterpret_cast<const float4*>(w + (long long)c * W);
    float* o = &f[0][0];
#pragma unroll
    for (int i = 0; i < kVec * W / 4; ++i) {
      const float4 v = p[i];
      o[4 * i] = v.x, o[4 * i + 1] = v.y, o[4 * i + 2] = v.z, o[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j) f[i][j] = i < n ? w[(long long)(c + i) * W + j] : 0.f;
  }
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

// Row of the window of token t (of the sequence `s`), j tokens back: an input, or the state.
template <typename T, int W>
__device__ __forceinline__ Raw8<T> tap(const ConvParams& p, const Span& s, int n, long long t,
                                       int c, int left, bool vec) {
  if (t >= s.begin) return load8(static_cast<const T*>(p.x) + t * p.x_stride + c, left, vec);
  Raw8<T> r;
  r.zero();
  if (p.s0)
    r = load8(static_cast<const T*>(p.s0) +
                  ((long long)n * (W - 1) + (W - 1) + (t - s.begin)) * p.D + c,
              left, vec);
  return r;
}

// State of sequence n after its tokens: the last W - 1 rows of [s0; x].
template <typename T, int W>
__device__ __forceinline__ void write_state(const ConvParams& p, int n, int c, int left, bool vec) {
  const Span s = span_of(p, n);
  Raw8<T> r[W - 1];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) r[j] = tap<T, W>(p, s, n, s.end - (W - 1) + j, c, left, vec);
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    store8(static_cast<T*>(p.sT) + ((long long)n * (W - 1) + j) * p.D + c, r[j], left, vec);
}

// blockIdx.x: run of `run` tokens, then (with `states`) one sequence's state each;
// blockIdx.y: 128 threads of 8 channels.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_kernel(const ConvParams p, int run, int runs,
                                                        long long tokens) {
  const int c = (blockIdx.y * kThreads + threadIdx.x) * kVec;
  if (c >= p.D) return;
  const int left = p.D - c;
  const bool vec = p.vec;
  if ((int)blockIdx.x >= runs) {
    write_state<T, W>(p, blockIdx.x - runs, c, left, vec);
    return;
  }
  const long long t0 = (long long)blockIdx.x * run, t1 = min(t0 + run, tokens);
  const T* x = static_cast<const T*>(p.x) + c;
  T* y = static_cast<T*>(p.y) + c;

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

  float f[kVec][W], bias[kVec], win[W - 1][kVec];
  load_filter<W>(p.w, c, left, f);
#pragma unroll
  for (int i = 0; i < kVec; ++i) bias[i] = p.bias && i < left ? p.bias[c + i] : 0.f;
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    tap<T, W>(p, s, n, max(t0, s.begin) - (W - 1) + j, c, left, vec).get(win[j]);

  for (long long t = t0; t < t1; t += kUnroll) {
    Raw8<T> raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (t + u < t1) raw[u] = load8(x + (t + u) * p.x_stride, left, vec);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long tt = t + u;
      if (tt >= t1) return;
      if (tt >= s.end) {  // the next sequence that has tokens begins
        do {
          if (++n >= p.N) return;
          s = span_of(p, n);
        } while (tt >= s.end);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
          tap<T, W>(p, s, n, max(tt, s.begin) - (W - 1) + j, c, left, vec).get(win[j]);
      }
      if (tt < s.begin) continue;
      float in[kVec], out[kVec];
      raw[u].get(in);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        float a = bias[i];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) a = fmaf(f[i][j], win[j][i], a);
        out[i] = fmaf(f[i][W - 1], in[i], a);
      }
      if (p.silu) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) out[i] = silu(out[i]);
      }
      Raw8<T> o;
      o.set(out);
      store8(y + tt * p.D, o, left, vec);
#pragma unroll
      for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < kVec; ++i) win[j][i] = win[j + 1][i];
#pragma unroll
      for (int i = 0; i < kVec; ++i) win[W - 2][i] = in[i];
    }
  }
}

// The states alone, after conv_kernel: for a state that is updated in place (another block
// of conv_kernel may still read it), or a batch without tokens.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_state_kernel(const ConvParams p) {
  const int c = (blockIdx.y * kThreads + threadIdx.x) * kVec;
  if (c < p.D) write_state<T, W>(p, blockIdx.x, c, p.D - c, p.vec);
}

// One token per sequence: a thread holds the window of 8 channels, s is shifted in place.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const ConvParams p, int per_row) {
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long n = id / per_row;
  if (n >= p.N) return;
  const int c = (int)(id % per_row) * kVec;
  const int left = p.D - c;
  const bool vec = p.vec;
  T* s = static_cast<T*>(p.sT) + n * (W - 1) * p.D + c;
  Raw8<T> r[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) r[j] = load8(s + (long long)j * p.D, left, vec);
  r[W - 1] = load8(static_cast<const T*>(p.x) + n * p.x_stride + c, left, vec);
  float f[kVec][W], out[kVec];
  load_filter<W>(p.w, c, left, f);
#pragma unroll
  for (int i = 0; i < kVec; ++i) out[i] = p.bias && i < left ? p.bias[c + i] : 0.f;
#pragma unroll
  for (int j = 0; j < W; ++j) {
    float in[kVec];
    r[j].get(in);
#pragma unroll
    for (int i = 0; i < kVec; ++i) out[i] = fmaf(f[i][j], in[i], out[i]);
  }
  if (p.silu) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) out[i] = silu(out[i]);
  }
  Raw8<T> o;
  o.set(out);
  store8(static_cast<T*>(p.y) + n * p.D + c, o, left, vec);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store8(s + (long long)j * p.D, r[j + 1], left, vec);
}

template <typename T, int W>
cudaError_t launch_w(const ConvParams& p, cudaStream_t stream) {
  const long long tokens = p.cu ? (long long)p.T : (long long)p.N * p.T;
  const int per_row = (p.D + kVec - 1) / kVec;
  const unsigned by = (per_row + kThreads - 1) / kThreads;
  const int run = 32;
  const long long runs = (tokens + run - 1) / run;
  // sT == s0: the states wait for every block that reads them
  const bool apart = p.sT && (p.s0 == p.sT || tokens == 0);
  const long long bx = runs + (p.sT && !apart ? p.N : 0);
  if (tokens > 0) {
    conv_kernel<T, W><<<dim3((unsigned)bx, by), kThreads, 0, stream>>>(p, run, (int)runs, tokens);
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

template <typename T>
cudaError_t launch_step_t(const ConvParams& p, cudaStream_t stream) {
  const int per_row = (p.D + kVec - 1) / kVec;
  const unsigned blocks = (unsigned)(((long long)p.N * per_row + kThreads - 1) / kThreads);
  if (p.W == 4) conv_step_kernel<T, 4><<<blocks, kThreads, 0, stream>>>(p, per_row);
  else if (p.W == 3) conv_step_kernel<T, 3><<<blocks, kThreads, 0, stream>>>(p, per_row);
  else conv_step_kernel<T, 2><<<blocks, kThreads, 0, stream>>>(p, per_row);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_conv(const ConvParams& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_t<float>(p, stream) : launch_t<__nv_bfloat16>(p, stream);
}
cudaError_t launch_conv_step(const ConvParams& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_step_t<float>(p, stream) : launch_step_t<__nv_bfloat16>(p, stream);
}

}  // namespace gdn
