// glr_bwd.cuh - the gradient of the gated linear recurrence over a prompt.
//
// With lambda_t the gradient that reaches h_t and m_t = a_t lambda_t what it passes on:
//
//   lambda_t = dy_t + m_{t+1} (a sequence's last token: dhT),   dx_t = s_t lambda_t,
//   dL_t = lambda_t (a_t h_{t-1} + (ds/dL) x_t),   ds/dL = 0, -a or -a^2 / s,
//   dg_t = dL_t (log), dL_t (1 - a_t) (sigmoid), dL_t rate sig (1 - sig) (rate),
//   drate = sum of dL_t sig,   dh0 = m of the sequence's first token.
//
// One pass from the last tokens to the first, laid out as the forward is (glr_fwd.cuh): m runs
// backwards over the same stretches, m_t = a_t (dy_t + m_{t+1}), and is exchanged the same way.
// h_{t-1} comes forwards again from the fp32 state that the forward left before the block's 64 tokens,
// so that no rounded y enters the gates' gradient and y itself is not read.  x, g and dy are
// read once, dx and dg written once.  Where s = 0 (a = 1 exactly) the weight has no derivative; its
// share is left out.
//
// 8 x 2048 x 2560 in bf16 with rate and sqrt takes 146 us, 2.9 TB/s, bound by instruction issue (64 % of its slots)
// at 12 warps an SM: 168 registers hold 16 tokens' decays, weights and states.
//
// A product that goes on into a sum is written as one operation: the compiler joins packed ones of its own, in
// one kernel and not in another, and the same call on other alignments would have other last bits.
//
// drate is summed by threads over their tokens, then over warps, blocks and rows in a fixed order.
#pragma once

#include "glr_common.cuh"

namespace gdn {
namespace {

// Two rounds' tiles: three would leave two blocks an SM instead of three.
constexpr int kMinBlocks = kGlrBwdBlocks, kStages = 2, kRun = kGlrBwdRun, kWarps = kGlrBwdWarps;
template <typename T, bool kNarrow>
constexpr int kTileOf = kRun * kWarps * kPitch<T, kNarrow>;  // of a tensor's tokens in shared memory

// lambda of a sequence's last token without what comes from behind: dy + dhT
__device__ __forceinline__ f32x2 with_last(const GlrParams& p, const int32_t* cu, f32x2 dy, int end, int t, long long c, bool c0,
                                           bool c1) {
  if (!p.dhT) return dy;
  return add2(dy, load_f32(p.dhT + (long long)sequence_of(cu, p.N, end, t) * p.D + c, p.vec, c0, c1));
}

// kGeneral: borders between tokens (packed rows); kNarrow: rows that are not aligned to pairs
template <typename T, int kGate, int kNorm, bool kGeneral, bool kNarrow>
__global__ void __launch_bounds__(32 * kWarps, sizeof(T) == 2 ? kMinBlocks : 1) glr_bwd_kernel(const GlrParams p) {
  constexpr int kTile = kTileOf<T, kNarrow>;
  extern __shared__ __align__(16) unsigned char s_tiles[];  // [stages][x, g, dy][tokens][64 channels and padding]
  __shared__ ulonglong2 s_ahead[2][kWarps][32], s_back[2][kWarps][32];
  __shared__ ulonglong2 s_state[32];
  __shared__ uint64_t s_bar[2];
  __shared__ int s_dead;
  volatile int* const dead = &s_dead;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // (known to be the warp's)
  const unsigned K = p.cluster, rank = K > 1 ? cluster_rank() : 0;
  const unsigned unit = blockIdx.x / K;
  const long long row = unit / p.tiles;
  const int tile = (int)(unit - (unsigned)row * p.tiles);
  const bool vec = !kNarrow || p.vec;
  const long long c = (long long)tile * 64 + 2 * lane;
  const bool c0 = c < p.D, c1 = c + 1 < p.D;
  const Places at = places<kNarrow>(vec, c0, c1);
  __shared__ int32_t s_cu[kGeneral ? kBorders : 1];
  const bool packed = kGeneral && p.cu;
  const int32_t* cu = kGeneral ? take_borders(p, s_cu) : nullptr;
  const unsigned end = packed ? min(max(p.cu[p.N], 0), p.T) : p.T;
  const unsigned span = warps * kRun, round = K * span;
  const unsigned rounds = end ? (end - 1) / round + 1 : 0;
  const f32x2 rate = kGate == GLR_RATE ? load_f32(p.rate + c, vec, c0, c1) : 0ull;
  f32x2 carry = !packed && p.dhT ? load_f32(p.dhT + row * p.D + c, vec, c0, c1) : 0ull;
  f32x2 drate = 0ull;

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
  T* tiles = reinterpret_cast<T*>(s_tiles);
  // behind them, of a cluster: [2][K blocks][32]
  ulonglong2* const s_rank = reinterpret_cast<ulonglong2*>(tiles + kStages * 3 * kTile);
  const bool odd = kNarrow && sizeof(T) == 2 && p.piece == 2;
  const int cols = (int)min(64ll, p.D - (long long)tile * 64);
  const long long tokens = packed ? p.T : (long long)p.N * p.T;
  const auto fetch = [&](unsigned r) {  // round r, counted from the last tokens, into its stage
    if (r < rounds) {
      const unsigned first = (rounds - 1 - r) * round + rank * span;
      const int left = first < end ? (int)min(end - first, (unsigned)(kRun * kWarps)) : 0;  // rows that exist
      T* to = tiles + r % kStages * (3 * kTile);
#pragma unroll 1
      for (int k = 0; k < 3; ++k, to += kTile) {
        const void* from = k == 0 ? p.x : k == 1 ? p.g : p.dy;
        const long long stride = k == 0 ? p.x_stride : k == 1 ? p.g_stride : p.dy_stride;
        copy_tile<kNarrow>(to, static_cast<const T*>(from) + (row * p.T + first) * stride + tile * 64ll, stride, left, span,
                             cols, p.piece, from, (tokens - 1) * stride + p.D);
      }
    }
    cp_async_commit();
  };
  unsigned t = (rounds - 1) * round + rank * span + warp * kRun;  // this thread's first token
  // the state before the chunk of 64 tokens that t lies in, of this round and the next; the chunk's warps
  // before this one lead on from it
  static_assert(kRun * kWarps % kGlrChunk == 0, "blocks of whole chunks");
  const auto state_before = [&](unsigned t) {
    return t < end ? load_f32(p.kept + (row * p.chunks + t / kGlrChunk) * p.D + c, vec, c0, c1) : 0ull;
  };
  f32x2 before = rounds ? state_before(t) : 0ull;
  constexpr int kChunkWarps = kGlrChunk / kRun;
  if (K > 1) cluster_wait();
  fetch(0);
  static_assert(kStages == 2, "a round's tiles are on their way while the one before is worked on");
  for (unsigned r = 0; r < rounds; ++r, t -= round) {
    const int turn = r & 1;
    // (a block that has given up a wait neither expects nor sends: its neighbours give up, too)
    if (K > 1 && threadIdx.x == 0 && !*dead) mbar_expect_tx(&s_bar[turn], K * 32 * 16);
    cp_async_wait<0>();
    __syncthreads();
    fetch(r + 1);
    const T* xs = tiles + r % kStages * (3 * kTile) + warp * kRun * kPitch<T, kNarrow>;
    const T *gs = xs + kTile, *ds = gs + kTile;
    const int n = t < end ? (int)min(end - t, (unsigned)kRun) : 0;  // tokens that exist
    const unsigned xsodd = odd && n ? odd_rows(static_cast<const T*>(p.x) + (row * p.T + t) * p.x_stride + tile * 64ll, p.x_stride) : 0u;
    const unsigned gsodd = odd && n ? odd_rows(static_cast<const T*>(p.g) + (row * p.T + t) * p.g_stride + tile * 64ll, p.g_stride) : 0u;
    const unsigned dsodd = odd && n ? odd_rows(static_cast<const T*>(p.dy) + (row * p.T + t) * p.dy_stride + tile * 64ll, p.dy_stride) : 0u;
    const unsigned borders = packed && n ? borders_of(cu, p.N, (int)end, (int)t, kRun) : 0u;
    f32x2 h = before;
    if (r + 1 < rounds) before = state_before(t - round);
    // One border among the run's tokens, and fewer tokens than a run has, are dealt with by selects, as
    // forwards: with the state that the border's sequence starts from, and the gradient that the one
    // before it ends with.
    const int border = kGeneral && borders ? __ffs(borders) - 1 : 2 * kRun;
    const bool many = kGeneral && (borders & (borders - 1)) != 0;
    const bool full = n == kRun && !borders;
    f32x2 start = 0ull, finish = 0ull;
    if (kGeneral && border < n && p.h0)
      start = load_f32(p.h0 + (long long)sequence_of(cu, p.N, (int)end, (int)t + border) * p.D + c, vec, c0, c1);
    if (kGeneral && border > 0 && border <= n && p.dhT)
      finish = load_f32(p.dhT + (long long)sequence_of(cu, p.N, (int)end, (int)t + border - 1) * p.D + c, vec, c0, c1);
    f32x2 a[kRun], s[kRun];
    f32x2 P = dup2(kWhole), H = 0ull, M = 0ull, lam = 0ull;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      gate2<kGate, kNorm>(pair_at<kNarrow>(gs, i, lane, gsodd), rate, a[i], s[i]);
      const f32x2 x = pair_at<kNarrow>(xs, i, lane, xsodd);
      H = fma2(a[i], kGeneral ? pick(i == border, start, H) : H, kNorm == GLR_NONE ? x : mul2(s[i], x));
      if (!full) a[i] = pick(i < n, a[i], dup2(1.f));  // (tokens that do not exist pass m on)
      P = mul2(P, a[i]);
    }
    // a border among the tokens, or behind them, cuts what goes on from them; many of them both ways
    const bool apart = kGeneral && border < kRun, apart_back = kGeneral && (many || (border > 0 && border <= kRun));
    P = at_least(P);
    if (!(kGeneral && many)) {
      // backwards: m before these tokens from m behind them
#pragma unroll
      for (int i = kRun - 1; i >= 0; --i) {
        const f32x2 dy = pair_at<kNarrow>(ds, i, lane, dsodd);
        const bool ends = kGeneral && i + 1 == border;
        if (i + 1 == kRun) lam = kGeneral ? add2(dy, pick(ends, finish, 0ull)) : dy;
        else lam = fma2(kGeneral ? pick(ends, dup2(1.f), a[(i + 1) % kRun]) : a[(i + 1) % kRun],
                        kGeneral ? pick(ends, finish, lam) : lam, dy);
      }
      M = mul2(a[0], lam);
    } else {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const f32x2 x = pair_at<kNarrow>(xs, i, lane, xsodd);
        f32x2 from = H;
        if (borders >> i & 1)
          from = p.h0 && i < n ? load_f32(p.h0 + (long long)sequence_of(cu, p.N, (int)end, (int)t + i) * p.D + c, vec,
                                          c0, c1)
                               : 0ull;
        H = fma2(a[i], from, kNorm == GLR_NONE ? x : mul2(s[i], x));
      }
#pragma unroll
      for (int i = kRun - 1; i >= 0; --i) {
        const f32x2 dy = pair_at<kNarrow>(ds, i, lane, dsodd);
        lam = i + 1 < kRun ? fma2(a[(i + 1) % kRun], lam, dy) : dy;
        if (i < n && borders >> (i + 1) & 1) lam = with_last(p, cu, dy, (int)end, (int)t + i, c, c0, c1);
      }
      M = mul2(a[0], lam);
    }
    s_ahead[turn][warp][lane] = make_ulonglong2(apart ? 0ull : P, H);
    s_back[turn][warp][lane] = make_ulonglong2(apart_back ? 0ull : P, M);
    __syncthreads();
    for (int w = warp / kChunkWarps * kChunkWarps; w < warp; ++w) {
      const ulonglong2 v = s_ahead[turn][w][lane];
      h = through<kGeneral>(v.x, v.y, h);
    }
    // the warps behind this one, last to first; (P, M) becomes what lies behind this warp's
    f32x2 sP = dup2(kWhole), sM = 0ull;
    ulonglong2 runs[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) runs[w] = w < warps ? s_back[turn][w][lane] : make_ulonglong2(dup2(kWhole), 0ull);
#pragma unroll
    for (int w = kWarps - 1; w >= 0; --w) {
      if (w == warp) P = sP, M = sM;
      follow<kGeneral>(sP, sM, runs[w].x, runs[w].y);
    }
    f32x2 m = carry;
    if (K > 1) {
      const f32x2 sent = to_send<kGeneral>(sP);
      if (!*dead) {
        for (unsigned k = warp; k < K; k += warps) send_to_rank(&s_rank[(turn * K + rank) * 32 + lane], &s_bar[turn], k, sent, sM);
      }
      if (warp == 0) {  // (one warp for all, the last block first)
        wait_for_ranks(&s_bar[turn], r >> 1 & 1, p.err, dead);
        s_state[lane] = pass_blocks<kGeneral>(carry, s_rank + (turn * K + K - 1) * 32 + lane, -32, (int)(K - 1 - rank), (int)K);
      }
      __syncthreads();
      m = s_state[lane].x, carry = s_state[lane].y;
    } else {
      carry = through<kGeneral>(sP, sM, carry);
    }
    m = through<kGeneral>(P, M, m);
    T* dx = static_cast<T*>(p.dx) + (row * p.T + t + kRun) * p.D + c;
    T* dg = static_cast<T*>(p.dg) + (row * p.T + t + kRun) * p.D + c;
    f32x2 hp[kRun];  // the state before each token
    const auto token = [&](int i, f32x2 x, bool some) {
      if (some) store_out<kNarrow>(dx, kNorm == GLR_NONE ? lam : mul2(s[i], lam), at);
      // dL / (a lambda): h_{t-1} and the weight's share
      f32x2 slope = hp[i];
      if (kNorm == GLR_LINEAR) slope = fma2(x, dup2(-1.f), slope);
      if (kNorm == GLR_SQRT) {
        const f32x2 inv = each(s[i], [](float v) { return v > 0.f ? -rcp(v) : 0.f; });
        slope = fma2(mul2(a[i], inv), x, slope);
      }
      m = mul2(a[i], lam);
      f32x2 d = mul2(m, slope);
      if (kGate != GLR_LOG) {
        float g0, g1, sig0, sig1, rest0, rest1;
        unpack2(s[i], rest0, rest1);
        if (kGate == GLR_RATE || kNorm != GLR_LINEAR) {
          unpack2(pair_at<kNarrow>(gs, i, lane, gsodd), g0, g1);
          sigmoid_of(g0, sig0, rest0);
          sigmoid_of(g1, sig1, rest1);
        }
        if (kGate == GLR_RATE) {
          drate = fma2(some ? d : 0ull, pack2(sig0, sig1), drate);
          d = mul2(mul2(d, pack2(sig0, sig1)), rate);
        }
        d = mul2(d, pack2(rest0, rest1));
      }
      if (some) store_out<kNarrow>(dg, d, at);
    };
    if (!(kGeneral && many)) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        hp[i] = kGeneral ? pick(i == border, start, h) : h;
        const f32x2 x = pair_at<kNarrow>(xs, i, lane, xsodd);
        h = fma2(a[i], hp[i], kNorm == GLR_NONE ? x : mul2(s[i], x));
      }
      // the gradient of the state that a sequence starts from
      const int first = packed ? border : t == 0 ? 0 : 2 * kRun;
      f32x2 of_start = 0ull;
      if (full) {
#pragma unroll
        for (int i = kRun - 1; i >= 0; --i) {
          dx -= p.D, dg -= p.D;
          const f32x2 dy = pair_at<kNarrow>(ds, i, lane, dsodd);
          lam = i + 1 == kRun ? add2(dy, m) : fma2(a[(i + 1) % kRun], lam, dy);
          token(i, pair_at<kNarrow>(xs, i, lane, xsodd), true);
        }
        of_start = m;
      } else {
        const f32x2 behind = m;
        m = 0ull;
        lam = 0ull;
#pragma unroll
        for (int i = kRun - 1; i >= 0; --i) {
          dx -= p.D, dg -= p.D;
          const f32x2 dy = pair_at<kNarrow>(ds, i, lane, dsodd);
          // what comes from the next token: nothing but `finish` at a border, m from behind the run's last
          const bool ends = kGeneral && i + 1 == border, last = i + 1 == n;
          const f32x2 by = i + 1 < kRun ? pick(ends || last, dup2(1.f), a[(i + 1) % kRun]) : dup2(1.f);
          lam = fma2(by, pick(ends, finish, pick(last, behind, lam)), dy);
          token(i, pair_at<kNarrow>(xs, i, lane, xsodd), i < n);
          of_start = pick(i == first, m, of_start);
        }
      }
      if (p.dh0 && first < n) {
        const long long q = packed ? sequence_of(cu, p.N, (int)end, (int)t + first) : row;
        store_f32(p.dh0 + q * p.D + c, of_start, vec, c0, c1);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        if (borders >> i & 1) {
          h = 0ull;
          if (p.h0 && i < n)
            h = load_f32(p.h0 + (long long)sequence_of(cu, p.N, (int)end, (int)t + i) * p.D + c, vec, c0, c1);
        }
        hp[i] = h;
        const f32x2 x = pair_at<kNarrow>(xs, i, lane, xsodd);
        h = fma2(a[i], h, kNorm == GLR_NONE ? x : mul2(s[i], x));
      }
#pragma unroll
      for (int i = kRun - 1; i >= 0; --i) {
        dx -= p.D, dg -= p.D;
        if (i >= n) continue;
        const f32x2 dy = pair_at<kNarrow>(ds, i, lane, dsodd);
        lam = borders >> (i + 1) & 1 ? with_last(p, cu, dy, (int)end, (int)t + i, c, c0, c1)
              : i + 1 == n           ? add2(dy, m)
                                     : fma2(a[(i + 1) % kRun], lam, dy);
        token(i, pair_at<kNarrow>(xs, i, lane, xsodd), true);
        if (p.dh0 && borders >> i & 1)
          store_f32(p.dh0 + (long long)sequence_of(cu, p.N, (int)end, (int)t + i) * p.D + c, m, vec, c0, c1);
      }
    }
  }
  cp_async_wait<0>();
  if (K > 1) leave_ranks(dead);
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
  if (!packed) {
    if (rounds == 0 && rank == 0 && warp == 0) store_f32(p.dh0 + row * p.D + c, carry, vec, c0, c1);
    return;
  }
  for (long long q = rank * warps + warp; q < p.N; q += K * warps) {  // sequences without tokens
    if (min(max(p.cu[q + 1], 0), (int)end) > min(max(p.cu[q], 0), (int)end)) continue;
    const f32x2 d = p.dhT ? load_f32(p.dhT + q * p.D + c, vec, c0, c1) : 0ull;
    store_f32(p.dh0 + q * p.D + c, d, vec, c0, c1);
  }
}

template <auto kKernel, typename T, bool kNarrow>
cudaError_t launch_prompt(GlrParams p, cudaStream_t stream) {
  const size_t smem = kStages * 3 * kTileOf<T, kNarrow> * sizeof(T);
  const int warps = p.T > kRun * (kWarps - 1) ? kWarps : p.T > kRun ? (p.T - 1) / kRun + 1 : 1;
  cudaError_t e = choose_cluster<kKernel, 32 * kWarps>(&p, smem, ((long long)p.T + kRun * kWarps - 1) / (kRun * kWarps));
  if (e == cudaSuccess && p.cluster > 1) e = device_error_word(&p.err);
  if (e == cudaSuccess) e = launch_clusters(kKernel, glr_grid(p), 32 * warps, p.cluster, p, stream,
                         glr_smem(smem, p.cluster), glr_smem(smem, kGlrMaxCluster));
  if (e != cudaSuccess || !p.drate) return e;
  return launch_column_sums(p.partial, p.drate, nullptr, (p.cu ? 1 : p.N) * p.cluster, p.D, stream);
}
template <typename T, int kGate, int kNorm>
cudaError_t launch(const GlrParams& p, cudaStream_t stream) {
  // each has the borders' arithmetic or the odd rows' only where it needs it (packed rows of pairs, 2560 x 16384
  // bf16 backwards with rate and sqrt: 226 us, 278 with the arithmetic of odd rows)
  if (!p.vec || p.piece == 2) return launch_prompt<glr_bwd_kernel<T, kGate, kNorm, true, true>, T, true>(p, stream);
  return p.cu ? launch_prompt<glr_bwd_kernel<T, kGate, kNorm, true, false>, T, false>(p, stream)
              : launch_prompt<glr_bwd_kernel<T, kGate, kNorm, false, false>, T, false>(p, stream);
}
template <typename T, int kGate>
cudaError_t launch_gate(const GlrParams& p, cudaStream_t stream) {
  return p.norm == GLR_NONE     ? launch<T, kGate, GLR_NONE>(p, stream)
         : p.norm == GLR_LINEAR ? launch<T, kGate, GLR_LINEAR>(p, stream)
                                : launch<T, kGate, GLR_SQRT>(p, stream);
}
template <typename T>
cudaError_t launch_type(const GlrParams& p, cudaStream_t stream) {
  return p.gate == GLR_LOG       ? launch_gate<T, GLR_LOG>(p, stream)
         : p.gate == GLR_SIGMOID ? launch_gate<T, GLR_SIGMOID>(p, stream)
                                 : launch_gate<T, GLR_RATE>(p, stream);
}

}  // namespace
}  // namespace gdn
