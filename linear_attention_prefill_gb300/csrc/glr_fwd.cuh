// glr_fwd.cuh - the gated linear recurrence over a prompt, and for one token.
//
//   h_t = a_t h_{t-1} + s(a_t) x_t,   y_t = h_t   (glr_common.cuh: gates and weights)
//
// One pass: a token's x and gate are read once, its decay and weighted input stay in registers
// until the state before them is known.  In a round the blocks of a cluster take 64 tokens each of
// the same 64 channels: every thread reduces its 16 tokens to (A, H), the warps exchange these through
// shared memory and the blocks through each other's, and a second walk over the 16 tokens, now
// from the right state, writes y.  Tiles arrive by asynchronous copies, two rounds ahead.
//
// State, products and sums are fp32; y is rounded once.
#pragma once

#include "glr_common.cuh"

namespace gdn {
namespace {

constexpr int kStages = 3;

template <typename T, int kGate, int kNorm, bool kPacked>
__global__ void __launch_bounds__(32 * kGlrWarps, sizeof(T) == 2 ? 4 : 2) glr_fwd_kernel(const GlrParams p) {
  extern __shared__ __align__(16) unsigned char s_tiles[];  // [stages][x, g][64 tokens][64 channels]
  __shared__ ulonglong2 s_warp[2][kGlrWarps][32];
  __shared__ ulonglong2 s_rank[2][kGlrMaxCluster][32];
  __shared__ uint64_t s_bar[2];
  __shared__ int s_dead;
  volatile int* const dead = &s_dead;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // (known to be the warp's)
  const unsigned K = p.cluster, rank = K > 1 ? cluster_rank() : 0;
  if (K > 1) {
    if (threadIdx.x == 0) {
      mbar_init(&s_bar[0], 1);
      mbar_init(&s_bar[1], 1);
      mbar_fence_init();
      s_dead = 0;
    }
    __syncwarp();
    cluster_arrive();
  }
  const unsigned unit = blockIdx.x / K;
  const long long row = unit / p.tiles;
  const int tile = (int)(unit - (unsigned)row * p.tiles);
  const bool vec = p.vec;
  const long long c = (long long)tile * 64 + 2 * lane;
  const bool c0 = c < p.D, c1 = c + 1 < p.D;
  const unsigned end = kPacked ? min(max(p.cu[p.N], 0), p.T) : p.T;
  const unsigned span = warps * kGlrRun, round = K * span;
  const unsigned rounds = end ? (end - 1) / round + 1 : 0;
  const f32x2 rate = kGate == GLR_RATE ? load_f32(p.rate + c, vec, c0, c1) : 0ull;
  f32x2 carry = !kPacked && p.h0 ? load_f32(p.h0 + row * p.D + c, vec, c0, c1) : 0ull;

  T* tiles = reinterpret_cast<T*>(s_tiles);
  const int cols = (int)min(64ll, p.D - (long long)tile * 64);
  const auto fetch = [&](unsigned r) {  // round r into its stage
    if (r < rounds) {
      const unsigned first = r * round + rank * span;
      const int left = first < end ? (int)min(end - first, 64u) : 0;  // rows that exist
      const long long at = row * p.T + first;
      T* to = tiles + r % kStages * (2 * 64 * 64);
      copy_tile(to, static_cast<const T*>(p.x) + at * p.x_stride + tile * 64ll, p.x_stride, left, span, cols, p.piece);
      copy_tile(to + 64 * 64, static_cast<const T*>(p.g) + at * p.g_stride + tile * 64ll, p.g_stride, left, span, cols, p.piece);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int r = 0; r < kStages - 1; ++r) fetch(r);
  unsigned t = rank * span + warp * kGlrRun;  // this thread's first token
  T* y = static_cast<T*>(p.y) + (row * p.T + t) * p.D + c;
  if (K > 1) cluster_wait();
  for (unsigned r = 0; r < rounds; ++r, t += round) {
    const int turn = r & 1;
    // (a block that has given up a wait neither expects nor sends: its neighbours give up, too)
    if (K > 1 && threadIdx.x == 0 && !*dead) mbar_expect_tx(&s_bar[turn], K * 32 * 16);
    cp_async_wait<kStages - 2>();
    __syncthreads();
    fetch(r + kStages - 1);
    const T* xs = tiles + r % kStages * (2 * 64 * 64) + warp * kGlrRun * 64;
    const T* gs = xs + 64 * 64;
    const int n = t < end ? (int)min(end - t, (unsigned)kGlrRun) : 0;  // tokens that exist
    const unsigned borders = kPacked && n ? borders_of(p.cu, p.N, (int)end, (int)t) : 0u;
    f32x2 a[kGlrRun], b[kGlrRun];
    f32x2 A = dup2(1.f), H = 0ull;
    bool cut = false;
#pragma unroll
    for (int i = 0; i < kGlrRun; ++i) {
      f32x2 s;
      gate2<kGate, kNorm>(pair_at(gs, i, lane), rate, a[i], s);
      b[i] = pair_at(xs, i, lane);
      if (kNorm != GLR_NONE) b[i] = mul2(s, b[i]);
      if (kPacked && borders >> i & 1) {
        if (p.h0 && i < n) {
          const long long q = sequence_of(p.cu, p.N, (int)end, (int)t + i);
          b[i] = fma2(a[i], load_f32(p.h0 + q * p.D + c, vec, c0, c1), b[i]);
        }
        H = b[i];
        cut = true;
      } else {
        H = fma2(a[i], H, b[i]);
        A = mul2(A, a[i]);
      }
    }
    // (behind the last token nothing is read from h: what zeros make of the gates there does not matter)
    A = kPacked && cut ? 0ull : at_least_tiny(A);
    s_warp[turn][warp][lane] = make_ulonglong2(A, H);
    __syncthreads();
    // all the warps' stretches in order; (A, H) becomes what lies before this warp's
    f32x2 sA = dup2(1.f), sH = 0ull;
#pragma unroll 4
    for (int w = 0; w < warps; ++w) {
      if (w == warp) A = sA, H = sH;
      const ulonglong2 v = s_warp[turn][w][lane];
      follow<kPacked>(sA, sH, v.x, v.y);
    }
    f32x2 h = carry;
    if (K > 1) {
      if (!*dead) {
        for (unsigned k = warp; k < K; k += warps) send_to_rank(&s_rank[turn][rank][lane], &s_bar[turn], k, sA, sH);
      }
      wait_for_ranks(&s_bar[turn], r >> 1 & 1, p.err, dead);
      f32x2 now = carry;
      for (unsigned k = 0; k < K; ++k) {
        if (k == rank) h = now;
        const ulonglong2 v = s_rank[turn][k][lane];
        now = through<kPacked>(v.x, v.y, now);
      }
      carry = now;
    } else {
      carry = through<kPacked>(sA, sH, carry);
    }
    if (p.states && warp == 0 && n)
      store_f32(p.states + (row * p.chunks + t / kGlrSpan) * p.D + c, h, vec, c0, c1);
    h = through<kPacked>(A, H, h);
    const int last = t + n == end ? n : 0;  // (1 and on: the row's last token is among these)
#pragma unroll
    for (int i = 0; i < kGlrRun; ++i) {
      h = kPacked && borders >> i & 1 ? b[i] : fma2(a[i], h, b[i]);
      if (i < n) {
        Raw2<T> o;
        o.set(h);
        o.store(y + i * (long long)p.D, vec, c0, c1);
      }
      if (kPacked ? i < n && borders >> (i + 1) & 1 : i + 1 == last) {
        if (p.hT) {
          const long long q = kPacked ? sequence_of(p.cu, p.N, (int)end, (int)t + i) : row;
          store_f32(p.hT + q * p.D + c, h, vec, c0, c1);
        }
      }
    }
    y += (long long)round * p.D;
  }
  cp_async_wait<0>();
  if (K > 1) cluster_sync();  // no block leaves before its neighbours have sent what they send
  if (!p.hT || p.hT == p.h0) return;
  if (!kPacked) {  // no token at all
    if (rounds == 0 && rank == 0 && warp == 0) store_f32(p.hT + row * p.D + c, carry, vec, c0, c1);
    return;
  }
  for (long long q = rank * warps + warp; q < p.N; q += K * warps) {  // sequences without tokens
    if (min(max(p.cu[q + 1], 0), (int)end) > min(max(p.cu[q], 0), (int)end)) continue;
    const f32x2 h = p.h0 ? load_f32(p.h0 + q * p.D + c, vec, c0, c1) : 0ull;
    store_f32(p.hT + q * p.D + c, h, vec, c0, c1);
  }
}

// One token a sequence: a warp has 64 channels of one.
template <typename T, int kGate, int kNorm>
__global__ void __launch_bounds__(128) glr_step_kernel(const GlrParams p) {
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5), row = unit / p.tiles;
  if (row >= p.N) return;
  const bool vec = p.vec;
  const long long c = (unit - row * p.tiles) * 64 + 2 * lane;
  const bool c0 = c < p.D, c1 = c + 1 < p.D;
  Raw2<T> x, g, o;
  x.load(static_cast<const T*>(p.x) + row * p.x_stride + c, vec, c0, c1);
  g.load(static_cast<const T*>(p.g) + row * p.g_stride + c, vec, c0, c1);
  f32x2 h = load_f32(p.h0 + row * p.D + c, vec, c0, c1), a, s;
  gate2<kGate, kNorm>(g.get(), kGate == GLR_RATE ? load_f32(p.rate + c, vec, c0, c1) : 0ull, a, s);
  h = fma2(a, h, kNorm == GLR_NONE ? x.get() : mul2(s, x.get()));
  o.set(h);
  o.store(static_cast<T*>(p.y) + row * p.D + c, vec, c0, c1);
  store_f32(p.hT + row * p.D + c, h, vec, c0, c1);
}

template <typename T, int kGate, int kNorm>
cudaError_t launch(const GlrParams& p, bool step, cudaStream_t stream) {
  if (step) {
    glr_step_kernel<T, kGate, kNorm><<<(unsigned)(((long long)p.N * p.tiles + 3) / 4), 128, 0, stream>>>(p);
    return cudaGetLastError();
  }
  const auto kernel = p.cu ? glr_fwd_kernel<T, kGate, kNorm, true> : glr_fwd_kernel<T, kGate, kNorm, false>;
  return launch_clusters(kernel, glr_grid(p), 32 * p.warps, p.cluster, p, stream, kStages * 2 * 64 * 64 * sizeof(T));
}
template <typename T, int kGate>
cudaError_t launch_gate(const GlrParams& p, bool step, cudaStream_t stream) {
  return p.norm == GLR_NONE     ? launch<T, kGate, GLR_NONE>(p, step, stream)
         : p.norm == GLR_LINEAR ? launch<T, kGate, GLR_LINEAR>(p, step, stream)
                                : launch<T, kGate, GLR_SQRT>(p, step, stream);
}
template <typename T>
cudaError_t launch_type(const GlrParams& p, bool step, cudaStream_t stream) {
  return p.gate == GLR_LOG       ? launch_gate<T, GLR_LOG>(p, step, stream)
         : p.gate == GLR_SIGMOID ? launch_gate<T, GLR_SIGMOID>(p, step, stream)
                                 : launch_gate<T, GLR_RATE>(p, step, stream);
}

}  // namespace
}  // namespace gdn
