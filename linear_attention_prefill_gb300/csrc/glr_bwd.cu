// glr_bwd.cu - the gradient of the gated linear recurrence over a prompt.
//
// With lambda_t the gradient that reaches h_t and m_t = a_t lambda_t what it passes on:
//
//   lambda_t = dy_t + m_{t+1} (a sequence's last token: dhT),   dx_t = s_t lambda_t,
//   dL_t = lambda_t (a_t h_{t-1} + (ds/dL) x_t),   ds/dL = 0, -a or -a^2 / s,
//   dg_t = dL_t (log), dL_t (1 - a_t) (sigmoid), dL_t rate sig (1 - sig) (rate),
//   drate = sum of dL_t sig,   dh0 = m of the sequence's first token.
//
// One pass from the last tokens to the first, laid out as the forward is (glr_fwd.cu): m runs
// backwards over the same stretches, m_t = a_t (dy_t + m_{t+1}), and is exchanged the same way.
// h_{t-1} comes forwards again from the fp32 state that the forward left before the block's 64 tokens,
// so that no rounded y enters the gates' gradient and y itself is not read.  x, g and dy are
// read once, dx and dg written once: HBM bandwidth bounds it.  Where s = 0 (a = 1 exactly) the weight
// has no derivative; its share is left out.
//
// drate is summed by threads over their tokens, then over warps, blocks and rows in a fixed order.
#include "glr_common.cuh"

namespace gdn {
namespace {

template <typename T, int kGate, int kNorm>
__global__ void __launch_bounds__(32 * kGlrWarps, sizeof(T) == 2 ? 2 : 1) glr_bwd_kernel(const GlrParams p) {
  __shared__ ulonglong2 s_ahead[2][kGlrWarps][32], s_back[2][kGlrWarps][32];
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
  f32x2 carry = p.dhT && !p.cu ? load_f32(p.dhT + row * p.D + c, vec, c0, c1) : 0ull;
  f32x2 drate = 0ull;

  Raw2<T> x[kGlrRun], g[kGlrRun], dy[kGlrRun];
  f32x2 before = 0ull;  // the state before the block's tokens
  auto load = [&](unsigned t) {
    const long long at = row * p.T + t;
    const T* xp = static_cast<const T*>(p.x) + at * p.x_stride + c;
    const T* gp = static_cast<const T*>(p.g) + at * p.g_stride + c;
    const T* dp = static_cast<const T*>(p.dy) + at * p.dy_stride + c;
#pragma unroll
    for (int i = 0; i < kGlrRun; ++i) {
      x[i].zero(), g[i].zero(), dy[i].zero();
      if (t + i < (unsigned)end) {
        x[i].load(xp + i * p.x_stride, vec, c0, c1);
        g[i].load(gp + i * p.g_stride, vec, c0, c1);
        dy[i].load(dp + i * p.dy_stride, vec, c0, c1);
      }
    }
    const unsigned first = t - warp * kGlrRun;
    if (first < (unsigned)end)
      before = load_f32(p.kept + (row * p.chunks + first / kGlrSpan) * p.D + c, vec, c0, c1);
  };
  unsigned t = (rounds - 1) * round + rank * span + warp * kGlrRun;  // this thread's first token
  if (rounds) load(t);
  if (K > 1) cluster_wait();
  for (unsigned r = 0; r < rounds; ++r, t -= round) {
    const int turn = r & 1;
    const unsigned borders = p.cu && t < (unsigned)end ? borders_of(p.cu, p.N, end, (int)t) : 0u;
    f32x2 a[kGlrRun], s[kGlrRun];
    f32x2 A = dup2(1.f), H = 0ull;
    bool cut = false;
#pragma unroll
    for (int i = 0; i < kGlrRun; ++i) {
      if (t + i >= (unsigned)end) {  // (warp-uniform)
        a[i] = dup2(1.f), s[i] = 0ull;
        continue;
      }
      gate2<kGate, kNorm>(g[i].get(), rate, a[i], s[i]);
      const f32x2 b = kNorm == GLR_NONE ? x[i].get() : mul2(s[i], x[i].get());
      if (borders >> i & 1) {
        f32x2 h = 0ull;
        if (p.h0) h = load_f32(p.h0 + (long long)sequence_of(p.cu, p.N, end, (int)t + i) * p.D + c, vec, c0, c1);
        H = fma2(a[i], h, b);
        cut = true;
      } else {
        H = fma2(a[i], H, b);
        A = mul2(A, a[i]);
      }
    }
    s_ahead[turn][warp][lane] = make_ulonglong2(cut ? 0ull : at_least_tiny(A), H);
    // backwards: m before these tokens from m behind them
    A = dup2(1.f);
    f32x2 M = 0ull;
    cut = false;
#pragma unroll
    for (int i = kGlrRun - 1; i >= 0; --i) {
      if (t + i >= (unsigned)end) continue;
      f32x2 lam = dy[i].get();
      if (p.cu && borders >> (i + 1) & 1) {
        if (p.dhT)
          lam = add2(lam, load_f32(p.dhT + (long long)sequence_of(p.cu, p.N, end, (int)t + i) * p.D + c, vec,
                                   c0, c1));
        cut = true;
        M = mul2(a[i], lam);
      } else {
        M = mul2(a[i], add2(lam, M));
        A = mul2(A, a[i]);
      }
    }
    A = cut ? 0ull : at_least_tiny(A);
    s_back[turn][warp][lane] = make_ulonglong2(A, M);
    __syncthreads();
    f32x2 h = before;
    for (int w = 0; w < warp; ++w) {
      const ulonglong2 v = s_ahead[turn][w][lane];
      h = through(v.x, v.y, h);
    }
    f32x2 sA = dup2(1.f), sM = 0ull;
    for (int w = warps - 1; w >= 0; --w) {
      if (w == warp) A = sA, M = sM;
      const ulonglong2 v = s_back[turn][w][lane];
      follow(sA, sM, v.x, v.y);
    }
    f32x2 m = carry;
    if (K > 1) {
      if (warp < (int)K) store_to_rank(&s_rank[turn][rank][lane], warp, sA, sM);
      cluster_sync();
      f32x2 now = carry;
      for (int k = (int)K - 1; k >= 0; --k) {
        if (k == (int)rank) m = now;
        const ulonglong2 v = s_rank[turn][k][lane];
        now = through(v.x, v.y, now);
      }
      carry = now;
    } else {
      carry = through(sA, sM, carry);
    }
    m = through(A, M, m);
    f32x2 hp[kGlrRun];  // the state before each token
#pragma unroll
    for (int i = 0; i < kGlrRun; ++i) {
      if (t + i >= (unsigned)end) break;
      if (borders >> i & 1) {
        h = 0ull;
        if (p.h0) h = load_f32(p.h0 + (long long)sequence_of(p.cu, p.N, end, (int)t + i) * p.D + c, vec, c0, c1);
      }
      hp[i] = h;
      h = fma2(a[i], h, kNorm == GLR_NONE ? x[i].get() : mul2(s[i], x[i].get()));
    }
    T* dx = static_cast<T*>(p.dx) + (row * p.T + t) * p.D + c;
    T* dg = static_cast<T*>(p.dg) + (row * p.T + t) * p.D + c;
#pragma unroll
    for (int i = kGlrRun - 1; i >= 0; --i) {
      if (t + i >= (unsigned)end) continue;
      f32x2 lam = dy[i].get();
      if (p.cu && borders >> (i + 1) & 1) {
        if (p.dhT)
          lam = add2(lam, load_f32(p.dhT + (long long)sequence_of(p.cu, p.N, end, (int)t + i) * p.D + c, vec,
                                   c0, c1));
      } else {
        lam = add2(lam, m);
      }
      Raw2<T> o;
      o.set(kNorm == GLR_NONE ? lam : mul2(s[i], lam));
      o.store(dx + i * (long long)p.D, vec, c0, c1);
      // dL / (a lambda): h_{t-1} and the weight's share
      f32x2 slope = hp[i];
      if (kNorm == GLR_LINEAR) slope = add2(slope, neg2(x[i].get()));
      if (kNorm == GLR_SQRT) {
        const f32x2 inv = each(s[i], [](float v) { return v > 0.f ? rcp(v) : 0.f; });
        slope = fma2(neg2(mul2(a[i], inv)), x[i].get(), slope);
      }
      m = mul2(a[i], lam);
      f32x2 d = mul2(m, slope);
      if (kGate == GLR_SIGMOID) {
        d = mul2(d, kNorm == GLR_LINEAR ? s[i] : mul2(exp_neg(g[i].get()), a[i]));
      } else if (kGate == GLR_RATE) {
        const f32x2 e = exp_neg(g[i].get()), sig = rcp2(add2(e, dup2(1.f)));
        d = mul2(d, sig);
        drate = add2(drate, d);
        d = mul2(mul2(d, rate), mul2(e, sig));
      }
      o.set(d);
      o.store(dg + i * (long long)p.D, vec, c0, c1);
      if (p.dh0 && (p.cu ? (borders >> i & 1) != 0 : t + i == 0)) {
        const long long n = p.cu ? sequence_of(p.cu, p.N, end, (int)t + i) : row;
        store_f32(p.dh0 + n * p.D + c, m, vec, c0, c1);
      }
    }
    if (r + 1 < rounds) load(t - round);
  }
  if (kGate == GLR_RATE) {  // the block's sum, its warps in order
    __syncthreads();
    f32x2* sum = reinterpret_cast<f32x2*>(&s_ahead[0][0][0]);
    sum[warp * 32 + lane] = drate;
    __syncthreads();
    if (warp == 0) {
      for (int w = 1; w < warps; ++w) drate = add2(drate, sum[w * 32 + lane]);
      store_f32(p.partial + (row * K + rank) * p.D + c, drate, vec, c0, c1);
    }
  }
  if (!p.dh0) return;
  if (!p.cu) {
    if (rounds == 0 && rank == 0 && warp == 0) store_f32(p.dh0 + row * p.D + c, carry, vec, c0, c1);
    return;
  }
  for (long long n = rank * warps + warp; n < p.N; n += K * warps) {  // sequences without tokens
    if (min(max(p.cu[n + 1], 0), end) > min(max(p.cu[n], 0), end)) continue;
    const f32x2 d = p.dhT ? load_f32(p.dhT + n * p.D + c, vec, c0, c1) : 0ull;
    store_f32(p.dh0 + n * p.D + c, d, vec, c0, c1);
  }
}

template <typename T, int kGate>
cudaError_t launch_gate(const GlrParams& p, cudaStream_t stream) {
  const auto kernel = p.norm == GLR_NONE     ? glr_bwd_kernel<T, kGate, GLR_NONE>
                      : p.norm == GLR_LINEAR ? glr_bwd_kernel<T, kGate, GLR_LINEAR>
                                             : glr_bwd_kernel<T, kGate, GLR_SQRT>;
  return launch_clusters(kernel, glr_grid(p), 32 * p.warps, p.cluster, p, stream);
}
template <typename T>
cudaError_t launch_type(const GlrParams& p, cudaStream_t stream) {
  return p.gate == GLR_LOG       ? launch_gate<T, GLR_LOG>(p, stream)
         : p.gate == GLR_SIGMOID ? launch_gate<T, GLR_SIGMOID>(p, stream)
                                 : launch_gate<T, GLR_RATE>(p, stream);
}

}  // namespace

cudaError_t launch_glr_bwd(const GlrParams& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_type<float>(p, stream) : launch_type<__nv_bfloat16>(p, stream);
}

}  // namespace gdn
