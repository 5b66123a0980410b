// short_conv.cu - the short causal convolution that a linear-attention layer applies to its
// projections before the forward (q, k, v of GDN and KDA; x, B, C of the SSD scan; x of S6),
// for prompts and for single tokens.
//
// Per channel d and token t of a sequence, W taps (2 to 4):
//   y_t = act(bias + sum_j w[d, j] x_{t - W + 1 + j}),   act = identity or SiLU,
// where the W - 1 inputs before the sequence come from its state s0 (zeros without one) and
// the last W - 1 inputs become the state sT.  Sums in fp32, one rounding at the end.
//
// HBM bandwidth bounds it: 2 bytes in and 2 out per element against ~13 instructions.  A
// thread has 4 channels (8 bytes of bf16) and walks a run of tokens with the window in
// registers as packed fp32 pairs, so that each input is loaded once except for the W - 1 rows
// before a run.  Its own inputs come by cp.async through a private ring of shared memory, two
// rounds of four tokens ahead: what is in flight then costs no registers.  At 4096 x 6144 (bf16,
// 101 MB): 39 us with 8 channels a thread and loads as they are needed, 26.6 us with 4 and one
// round ahead in registers, 19.7 us with the ring (5.1 TB/s; 10007 x 5376 36.8 us, 5.9 TB/s), both
// in a graph; one round more or less ahead 20.0 and 21.2.  Eight channels a thread on the ring
// take a quarter fewer instructions but 124 registers: no faster.  Rows off 4-channel pieces are
// loaded element by element.
#include "gdn_common.cuh"
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 64;
constexpr int kStepThreads = 128;
constexpr int kAhead = 4;     // tokens of a round
constexpr int kRounds = 3;    // rounds of the ring

constexpr int kChans = 4;          // channels per thread

// kChans neighbouring channels of a row, as stored and as fp32 pairs.
template <typename T>
struct Piece {
  Raw4<T> r;
  __device__ __forceinline__ void zero() { r.zero(); }
  __device__ __forceinline__ void load(const T* p, int n, bool vec) { r.load(p, n, vec); }
  __device__ __forceinline__ void store(T* p, int n, bool vec) const { r.store(p, n, vec); }
  __device__ __forceinline__ void get(f32x2 (&o)[kChans / 2]) const {
    const float4 v = r.get();
    o[0] = pack2(v.x, v.y);
    o[1] = pack2(v.z, v.w);
  }
  __device__ __forceinline__ void set(const f32x2 (&v)[kChans / 2]) {
    float a, b, c, d;
    unpack2(v[0], a, b);
    unpack2(v[1], c, d);
    r.set(a, b, c, d);
  }
};

// The filters of channels c..c+kChans-1, tap by tap: w is [D, W] and c a multiple of kChans, so the kChans W
// floats are whole 16-byte pieces.
template <int W>
__device__ __forceinline__ void load_filter(const float* w, int c, int n, f32x2 (&f)[W][kChans / 2]) {
  float v[kChans * W];
  if (n >= kChans) {
    const float4* p = reinterpret_cast<const float4*>(w + (long long)c * W);
#pragma unroll
    for (int i = 0; i < kChans * W / 4; ++i) {
      const float4 q = p[i];
      v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kChans * W; ++i) v[i] = i / W < n ? w[(long long)c * W + i] : 0.f;
  }
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int i = 0; i < kChans / 2; ++i) f[j][i] = pack2(v[2 * i * W + j], v[(2 * i + 1) * W + j]);
}
__device__ __forceinline__ void load_bias(const float* bias, int c, int n, f32x2 (&b)[kChans / 2]) {
#pragma unroll
  for (int i = 0; i < kChans / 2; ++i)
    b[i] = pack2(bias && 2 * i < n ? bias[c + 2 * i] : 0.f,
                 bias && 2 * i + 1 < n ? bias[c + 2 * i + 1] : 0.f);
}
// act(bias + sum of taps), rounded
template <typename T, int W>
__device__ __forceinline__ Piece<T> filter(const f32x2 (&f)[W][kChans / 2], const f32x2 (&bias)[kChans / 2],
                                              const f32x2 (&win)[W][kChans / 2], int act) {
  f32x2 a[kChans / 2];
#pragma unroll
  for (int i = 0; i < kChans / 2; ++i) {
    a[i] = bias[i];
#pragma unroll
    for (int j = 0; j < W; ++j) a[i] = fma2(f[j][i], win[j][i], a[i]);
  }
  if (act) {
#pragma unroll
    for (int i = 0; i < kChans / 2; ++i) a[i] = silu2(a[i]);
  }
  Piece<T> o;
  o.set(a);
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

// The first sequence of a packed batch, from number lo on, that ends behind row t (N: none does).
__device__ __forceinline__ int ends_behind(const ConvParams& p, int lo, long long t) {
  int hi = p.N;
  while (lo < hi) {
    const int mid = lo + ((hi - lo) >> 1);  // (lo + hi may pass 31 bits)
    if (min(max(p.cu[mid + 1], 0), p.T) > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Row of the window of a token of sequence n, t = an absolute row: an input, or the state.
template <typename T, int W>
__device__ __forceinline__ Piece<T> tap(const ConvParams& p, const Span& s, int n, long long t,
                                           int c, int left, bool vec) {
  Piece<T> r;
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
  Piece<T> r[W - 1];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) r[j] = tap<T, W>(p, s, n, s.end - (W - 1) + j, c, left, vec);
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    r[j].store(static_cast<T*>(p.sT) + ((long long)n * (W - 1) + j) * p.D + c, left, vec);
}

// cp.async of one thread's piece
template <int kBytes>
__device__ __forceinline__ void copy_piece(void* dst, const void* src) {
  if constexpr (kBytes == 16)
    cp_async16(dst, src, true);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// blockIdx.x: run of `run` tokens, then (with sT) one sequence's state each; blockIdx.y: 64
// threads of kChans channels.  kVec: whole aligned pieces.
template <typename T, int W, bool kVec>
__global__ void __launch_bounds__(kThreads) conv_kernel(const ConvParams p, int run, int runs,
                                                        long long tokens) {
  using P = Piece<T>;
  __shared__ __align__(16) unsigned char s_ring[kVec ? kRounds * kAhead * kThreads * sizeof(P) : 16];
  const int c = (blockIdx.y * kThreads + threadIdx.x) * kChans;
  if (c >= p.D) return;
  const int left = p.D - c;
  if ((int)blockIdx.x >= runs) {
    write_state<T, W>(p, blockIdx.x - runs, c, left, kVec);
    return;
  }
  const long long t0 = (long long)blockIdx.x * run, t1 = min(t0 + run, tokens);
  const T* x = static_cast<const T*>(p.x) + t0 * p.x_stride + c;
  T* y = static_cast<T*>(p.y) + t0 * p.D + c;
  P ahead[kVec ? 1 : kAhead];  // the tokens of the next round
  P* ring = reinterpret_cast<P*>(s_ring) + threadIdx.x;
  const int len = (int)(t1 - t0);
  int wanted = len, to = 0;  // tokens not yet requested; the ring's place for the next round
  auto request = [&]() {     // this thread's inputs of the next round, x at its first token
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (u < wanted) {
        if constexpr (kVec) copy_piece<sizeof(P)>(ring + (to * kAhead + u) * kThreads, x);
        else ahead[u].load(x, left, false);
      }
      x += p.x_stride;
    }
    if constexpr (kVec) cp_async_commit();
    wanted -= kAhead;
    if (++to == kRounds) to = 0;
  };
#pragma unroll
  for (int round = 0; round < (kVec ? kRounds - 1 : 1); ++round) request();

  // the sequence of token t0: the first one that ends behind it
  int n = p.cu ? ends_behind(p, 0, t0) : (int)(t0 / p.T);
  if (n >= p.N) {  // behind the last sequence: left as it was
    if constexpr (kVec) cp_async_wait<0>();  // (no thread leaves while its copies are in flight)
    return;
  }
  Span s = span_of(p, n);

  f32x2 f[W][kChans / 2], win[W][kChans / 2], bias[kChans / 2];  // the filter, and the inputs under it
  load_filter<W>(p.w, c, left, f);
  load_bias(p.bias, c, left, bias);
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    tap<T, W>(p, s, n, max(t0, s.begin) - (W - 1) + j, c, left, kVec).get(win[j]);
  auto next = [&](const P& in, T* to) {  // one token
    in.get(win[W - 1]);
    filter<T, W>(f, bias, win, p.silu).store(to, left, kVec);
#pragma unroll
    for (int j = 0; j + 1 < W; ++j)
#pragma unroll
      for (int i = 0; i < kChans / 2; ++i) win[j][i] = win[j + 1][i];
  };

  // the sequence's tokens, counted from t0
  int begin = (int)max(s.begin - t0, 0ll), end = (int)min(s.end - t0, (long long)len);
  for (int t = 0, from = 0; t < len; t += kAhead) {
    P raw[kAhead];
    if constexpr (kVec) {
      request();
      cp_async_wait<kRounds - 1>();
#pragma unroll
      for (int u = 0; u < kAhead; ++u) raw[u] = ring[(from * kAhead + u) * kThreads];
      if (++from == kRounds) from = 0;
    } else {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) raw[u] = ahead[u];
      request();
    }
    if (t >= begin && t + kAhead <= end) {  // one sequence's tokens
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        next(raw[u], y);
        y += p.D;
      }
    } else {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int tt = t + u;
        if (tt >= len) return;
        if (tt >= end) {  // the next sequence that has tokens begins
          if (++n < p.N) s = span_of(p, n);
          if (n < p.N && t0 + tt >= s.end) {  // an empty one: past all of them
            n = ends_behind(p, n + 1, t0 + tt);
            if (n < p.N) s = span_of(p, n);
          }
          if (n >= p.N) {
            if constexpr (kVec) cp_async_wait<0>();
            return;
          }
          begin = (int)max(s.begin - t0, 0ll);
          end = (int)min(s.end - t0, (long long)len);
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
            tap<T, W>(p, s, n, max(t0 + tt, s.begin) - (W - 1) + j, c, left, kVec).get(win[j]);
        }
        if (tt >= begin) next(raw[u], y);
        y += p.D;
      }
    }
  }
}

// The states alone, after conv_kernel: for a state that is updated in place (another block
// of conv_kernel may still read it), or a batch without tokens.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_state_kernel(const ConvParams p) {
  const int c = (blockIdx.y * kThreads + threadIdx.x) * kChans;
  if (c < p.D) write_state<T, W>(p, blockIdx.x, c, p.D - c, p.vec);
}

// One token per sequence: a thread holds the windows of 4 channels of kSeqs sequences and
// shifts their states in place.  kSeqs > 1 shares the filter, which is as many bytes as the
// window and the output of one sequence.  256 x 8192 (bf16, 34 MB): 7.0 us in a graph (4.8 TB/s), 1
// x 8192 1.6.  The 1 in the bounds lets the compiler take the registers to have every load in
// flight at once (70; 56 by itself, 8.9 us).
template <typename T, int W, int kSeqs, bool kVec>
__global__ void __launch_bounds__(kStepThreads, 1) conv_step_kernel(const ConvParams p, int per_row) {
  const long long id = (long long)blockIdx.x * kStepThreads + threadIdx.x;
  const long long first = id / per_row * kSeqs;
  if (first >= p.N) return;
  const int c = (int)(id % per_row) * kChans;
  const int left = kVec ? kChans : p.D - c;
  Piece<T> r[kSeqs][W];
#pragma unroll
  for (int i = 0; i < kSeqs; ++i) {
    if (first + i >= p.N) break;
    const T* s = static_cast<const T*>(p.sT) + (first + i) * (W - 1) * p.D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[i][j].load(s + (long long)j * p.D, left, kVec);
    r[i][W - 1].load(static_cast<const T*>(p.x) + (first + i) * p.x_stride + c, left, kVec);
  }
  f32x2 f[W][kChans / 2], bias[kChans / 2];
  load_filter<W>(p.w, c, left, f);
  load_bias(p.bias, c, left, bias);
#pragma unroll
  for (int i = 0; i < kSeqs; ++i) {
    if (first + i >= p.N) break;
    f32x2 win[W][kChans / 2];
#pragma unroll
    for (int j = 0; j < W; ++j) r[i][j].get(win[j]);
    filter<T, W>(f, bias, win, p.silu)
        .store(static_cast<T*>(p.y) + (first + i) * p.D + c, left, kVec);
    T* s = static_cast<T*>(p.sT) + (first + i) * (W - 1) * p.D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[i][j + 1].store(s + (long long)j * p.D, left, kVec);
  }
}

template <typename T, int W, bool kVec>
cudaError_t launch_v(const ConvParams& p, bool states, cudaStream_t stream) {
  const long long tokens = p.cu ? (long long)p.T : (long long)p.N * p.T;
  const unsigned by = ((p.D + kChans - 1) / kChans + kThreads - 1) / kThreads;
  // long runs repeat fewer rows (W - 1 each), short ones fill the GPU: 16 blocks per SM (runs of
  // 64: 22.0 us at 4096 x 6144 and 26.3 at 16384 x 2048; of 32: 21.1 and 26.4; of 16: 23.2, 28.3)
  int run = 32;
  while (run > kAhead && (tokens + run - 1) / run * by < 16 * kSms) run /= 2;
  const long long runs = (tokens + run - 1) / run;
  const dim3 grid((unsigned)(runs + (states ? p.N : 0)), by);
  conv_kernel<T, W, kVec><<<grid, kThreads, 0, stream>>>(p, run, (int)runs, tokens);
  return cudaGetLastError();
}

template <typename T, int W>
cudaError_t launch_w(const ConvParams& p, cudaStream_t stream) {
  const bool none = p.T == 0;
  // sT == s0: the states wait for every block that reads them
  const bool apart = p.sT && (p.s0 == p.sT || none), states = p.sT && !apart;
  cudaError_t e = cudaSuccess;
  if (none) {
  } else if (p.vec) {
    e = launch_v<T, W, true>(p, states, stream);
  } else {
    e = launch_v<T, W, false>(p, states, stream);
  }
  if (e != cudaSuccess || !apart) return e;
  const unsigned by = ((p.D + kChans - 1) / kChans + kThreads - 1) / kThreads;
  conv_state_kernel<T, W><<<dim3((unsigned)p.N, by), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const ConvParams& p, cudaStream_t stream) {
  if (p.W == 4) return launch_w<T, 4>(p, stream);
  if (p.W == 3) return launch_w<T, 3>(p, stream);
  return launch_w<T, 2>(p, stream);
}

template <typename T, int W, bool kVec>
cudaError_t launch_step_v(const ConvParams& p, cudaStream_t stream) {
  const int per_row = (p.D + kChans - 1) / kChans;
  const auto blocks = [&](int seqs) {
    return (unsigned)(((long long)((p.N + seqs - 1) / seqs) * per_row + kStepThreads - 1) /
                      kStepThreads);
  };
  // two sequences a thread once that still leaves 8 blocks per SM
  if (blocks(2) >= 8 * kSms)
    conv_step_kernel<T, W, 2, kVec><<<blocks(2), kStepThreads, 0, stream>>>(p, per_row);
  else
    conv_step_kernel<T, W, 1, kVec><<<blocks(1), kStepThreads, 0, stream>>>(p, per_row);
  return cudaGetLastError();
}
template <typename T, int W>
cudaError_t launch_step_w(const ConvParams& p, cudaStream_t stream) {
  return p.vec ? launch_step_v<T, W, true>(p, stream) : launch_step_v<T, W, false>(p, stream);
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
