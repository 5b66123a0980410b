// glr_fwd.cu - the gated linear recurrence over a prompt, and for one token.
//
//   h_t = a_t h_{t-1} + s(a_t) x_t,   y_t = h_t   (glr_common.cuh: gates and weights)
//
// One pass: a token's x and gate are read once, its decay and weighted input stay in registers
// until the state before them is known.  In a round the blocks of a cluster take 64 tokens each of
// the same 64 channels: every thread reduces its 8 tokens to (A, H), the warps exchange these through
// shared memory and the blocks through each other's, and a second walk over the 8 tokens, now
// from the right state, writes y.  The next round's loads are under way meanwhile.  HBM bandwidth
// bounds long prompts, the rounds' exchanges short ones.
//
// State, products and sums are fp32; y is rounded once.
#include "glr_common.cuh"

namespace gdn {
namespace {

template <typename T, int kGate, int kNorm>
__global__ void __launch_bounds__(32 * kGlrWarps) glr_fwd_kernel(const GlrParams p) {
  __shared__ ulonglong2 s_warp[2][kGlrWarps][32];
  __shared__ ulonglong2 s_rank[2][kGlrMaxCluster][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const unsigned K = p.cluster, rank = K > 1 ? cluster_rank() : 0;
  if (K > 1) cluster_arrive();
  const unsigned unit = blockIdx.x / K;
  const long long row = unit / p.tiles;
  const int tile = (int)(unit - (unsigned)row * p.tiles);
  const bool vec = p.vec;
  const long long c = (long long)tile * 64 + (vec ? 2 * lane : lane);
  const bool c0 = c < p.D, c1 = vec ? c0 : c + 32 < p.D;
  const int end = p.cu ? min(max(p.cu[p.N], 0), p.T) : p.T;
  const unsigned span = warps * kGlrRun, round = K * span;
  const unsigned rounds = end ? ((unsigned)end - 1) / round + 1 : 0;
  const f32x2 rate = kGate == GLR_RATE ? load_f32(p.rate + c, vec, c0, c1) : 0ull;
  f32x2 carry = p.h0 && !p.cu ? load_f32(p.h0 + row * p.D + c, vec, c0, c1) : 0ull;

  Raw2<T> x[kGlrRun], g[kGlrRun];
  unsigned t = rank * span + warp * kGlrRun;  // this thread's first token
  const T* xp = static_cast<const T*>(p.x) + (row * p.T + t) * p.x_stride + c;
  const T* gp = static_cast<const T*>(p.g) + (row * p.T + t) * p.g_stride + c;
  T* y = static_cast<T*>(p.y) + (row * p.T + t) * p.D + c;
  auto load = [&](unsigned first) {
#pragma unroll
    for (int i = 0; i < kGlrRun; ++i) {
      x[i].zero(), g[i].zero();
      if (first + i < (unsigned)end) {
        x[i].load(xp + i * p.x_stride, vec, c0, c1);
        g[i].load(gp + i * p.g_stride, vec, c0, c1);
      }
    }
    xp += round * p.x_stride;
    gp += round * p.g_stride;
  };
  load(t);
  if (K > 1) cluster_wait();
  for (unsigned r = 0; r < rounds; ++r, t += round) {
    const int turn = r & 1;
    const unsigned borders = p.cu && t < (unsigned)end ? borders_of(p.cu, p.N, end, (int)t) : 0u;
    f32x2 a[kGlrRun], b[kGlrRun];
    f32x2 A = dup2(1.f), H = 0ull;
    bool cut = false;
#pragma unroll
    for (int i = 0; i < kGlrRun; ++i) {
      if (t + i >= (unsigned)end) {  // (warp-uniform) behind the last token nothing is read from h
        a[i] = dup2(1.f), b[i] = 0ull;
        continue;
      }
      f32x2 s;
      gate2<kGate, kNorm>(g[i].get(), rate, a[i], s);
      b[i] = kNorm == GLR_NONE ? x[i].get() : mul2(s, x[i].get());
      if (borders >> i & 1) {
        if (p.h0) {
          const long long n = sequence_of(p.cu, p.N, end, (int)t + i);
          b[i] = fma2(a[i], load_f32(p.h0 + n * p.D + c, vec, c0, c1), b[i]);
        }
        H = b[i];
        cut = true;
      } else {
        H = fma2(a[i], H, b[i]);
        A = mul2(A, a[i]);
      }
    }
    A = cut ? 0ull : at_least_tiny(A);
    if (r + 1 < rounds) load(t + round);
    s_warp[turn][warp][lane] = make_ulonglong2(A, H);
    __syncthreads();
    // all the warps' stretches in order; (A, H) becomes what lies before this warp's
    f32x2 sA = dup2(1.f), sH = 0ull;
    for (int w = 0; w < warps; ++w) {
      if (w == warp) A = sA, H = sH;
      const ulonglong2 v = s_warp[turn][w][lane];
      follow(sA, sH, v.x, v.y);
    }
    f32x2 h = carry;
    if (K > 1) {
      if (warp < (int)K) store_to_rank(&s_rank[turn][rank][lane], warp, sA, sH);
      cluster_sync();
      f32x2 now = carry;
      for (unsigned k = 0; k < K; ++k) {
        if (k == rank) h = now;
        const ulonglong2 v = s_rank[turn][k][lane];
        now = through(v.x, v.y, now);
      }
      carry = now;
    } else {
      carry = through(sA, sH, carry);
    }
    if (p.states && warp == 0 && t < (unsigned)end)
      store_f32(p.states + (row * p.chunks + t / kGlrSpan) * p.D + c, h, vec, c0, c1);
    h = through(A, H, h);
#pragma unroll
    for (int i = 0; i < kGlrRun; ++i) {
      if (t + i >= (unsigned)end) break;
      h = borders >> i & 1 ? b[i] : fma2(a[i], h, b[i]);
      Raw2<T> o;
      o.set(h);
      o.store(y + i * (long long)p.D, vec, c0, c1);
      if (p.hT && (p.cu ? (borders >> (i + 1) & 1) != 0 : t + i + 1 == (unsigned)end)) {
        const long long n = p.cu ? sequence_of(p.cu, p.N, end, (int)t + i) : row;
        store_f32(p.hT + n * p.D + c, h, vec, c0, c1);
      }
    }
    y += (long long)round * p.D;
  }
  if (!p.hT || p.hT == p.h0) return;
  if (!p.cu) {  // no token at all
    if (rounds == 0 && rank == 0 && warp == 0) store_f32(p.hT + row * p.D + c, carry, vec, c0, c1);
    return;
  }
  for (long long n = rank * warps + warp; n < p.N; n += K * warps) {  // sequences without tokens
    if (min(max(p.cu[n + 1], 0), end) > min(max(p.cu[n], 0), end)) continue;
    const f32x2 h = p.h0 ? load_f32(p.h0 + n * p.D + c, vec, c0, c1) : 0ull;
    store_f32(p.hT + n * p.D + c, h, vec, c0, c1);
  }
}

// One token a sequence: a warp has 64 channels of one.
template <typename T, int kGate, int kNorm>
__global__ void __launch_bounds__(128) glr_step_kernel(const GlrParams p) {
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5), row = unit / p.tiles;
  if (row >= p.N) return;
  const bool vec = p.vec;
  const long long c = (unit - row * p.tiles) * 64 + (vec ? 2 * lane : lane);
  const bool c0 = c < p.D, c1 = vec ? c0 : c + 32 < p.D;
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
  return launch_clusters(glr_fwd_kernel<T, kGate, kNorm>, glr_grid(p), 32 * p.warps, p.cluster, p, stream);
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

cudaError_t launch_glr(const GlrParams& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_type<float>(p, false, stream) : launch_type<__nv_bfloat16>(p, false, stream);
}
cudaError_t launch_glr_step(const GlrParams& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_type<float>(p, true, stream) : launch_type<__nv_bfloat16>(p, true, stream);
}

}  // namespace gdn
