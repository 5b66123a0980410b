// glr_fwd.cuh - the gated linear recurrence over a prompt, and for one token.
//
//   h_t = a_t h_{t-1} + s(a_t) x_t,   y_t = h_t   (glr_common.cuh: gates and weights)
//
// One pass: a token's x and gate are read once, its decay and weighted input stay in registers
// until the state before them is known.  In a round the blocks of a cluster take 64 tokens each of
// the same 64 channels: every thread reduces its 16 tokens to (A, H), the warps exchange these through
// shared memory and the blocks through each other's, and a second walk over the 16 tokens, now
// from the right state, writes y.  Tiles arrive by asynchronous copies, one round ahead.
//
// State, products and sums are fp32; y is rounded once.
//
// 65536 x 2560 in bf16 takes 256 us, 3.9 TB/s: instruction issue bounds it (60 % of its slots) at 14 warps an SM,
// which cannot hide all of the exchange.  16 tokens a thread is what 128 registers hold, and four
// blocks of four warps an SM; with 8 tokens the rounds were twice as many and the time longer.
#pragma once

#include "glr_common.cuh"

namespace gdn {
namespace {

constexpr int kMinBlocks = kGlrFwdBlocks, kStages = 2, kRun = kGlrFwdRun, kWarps = kGlrFwdWarps;
template <typename T, bool kNarrow>
constexpr int kTileOf = kRun * kWarps * kPitch<T, kNarrow>;  // of a tensor's tokens in shared memory

// kGeneral: borders between tokens (packed rows); kNarrow: rows that are not aligned to pairs
template <typename T, int kGate, int kNorm, bool kGeneral, bool kNarrow>
__global__ void __launch_bounds__(32 * kWarps, sizeof(T) == 2 ? kMinBlocks : 1) glr_fwd_kernel(const GlrParams p) {
  constexpr int kTile = kTileOf<T, kNarrow>;
  extern __shared__ __align__(16) unsigned char s_tiles[];  // [stages][x, g][tokens][64 channels and padding]
  __shared__ ulonglong2 s_warp[2][kWarps][32];
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
  f32x2 carry = !packed && p.h0 ? load_f32(p.h0 + row * p.D + c, vec, c0, c1) : 0ull;

  // (the state is read before the others hear of this block: the last token's block may write it in place)
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
  ulonglong2* const s_rank = reinterpret_cast<ulonglong2*>(tiles + kStages * 2 * kTile);
  const bool odd = kNarrow && sizeof(T) == 2 && p.piece == 2;
  const int cols = (int)min(64ll, p.D - (long long)tile * 64);
  const long long tokens = packed ? p.T : (long long)p.N * p.T;
  const auto fetch = [&](unsigned r) {  // round r into its stage
    if (r < rounds) {
      const unsigned first = r * round + rank * span;
      const int left = first < end ? (int)min(end - first, (unsigned)(kRun * kWarps)) : 0;  // rows that exist
      T* to = tiles + r % kStages * (2 * kTile);
#pragma unroll 1
      for (int k = 0; k < 2; ++k, to += kTile) {
        const void* from = k ? p.g : p.x;
        const long long stride = k ? p.g_stride : p.x_stride;
        copy_tile<kNarrow>(to, static_cast<const T*>(from) + (row * p.T + first) * stride + tile * 64ll, stride, left, span,
                             cols, p.piece, from, (tokens - 1) * stride + p.D);
      }
    }
    cp_async_commit();
  };
  unsigned t = rank * span + warp * kRun;  // this thread's first token
  T* y = static_cast<T*>(p.y) + (row * p.T + t) * p.D + c;
  if (K > 1) cluster_wait();
  fetch(0);
  static_assert(kStages == 2, "a round's tiles are on their way while the one before is worked on");
  for (unsigned r = 0; r < rounds; ++r, t += round) {
    const int turn = r & 1;
    // (a block that has given up a wait neither expects nor sends: its neighbours give up, too)
    if (K > 1 && threadIdx.x == 0 && !*dead) mbar_expect_tx(&s_bar[turn], K * 32 * 16);
    cp_async_wait<0>();
    __syncthreads();
    fetch(r + 1);
    const T* xs = tiles + r % kStages * (2 * kTile) + warp * kRun * kPitch<T, kNarrow>;
    const T* gs = xs + kTile;
    const int n = t < end ? (int)min(end - t, (unsigned)kRun) : 0;  // tokens that exist
    const unsigned xsodd = odd && n ? odd_rows(static_cast<const T*>(p.x) + (row * p.T + t) * p.x_stride + tile * 64ll, p.x_stride) : 0u;
    const unsigned gsodd = odd && n ? odd_rows(static_cast<const T*>(p.g) + (row * p.T + t) * p.g_stride + tile * 64ll, p.g_stride) : 0u;
    const unsigned borders = packed && n ? borders_of(cu, p.N, (int)end, (int)t, kRun) : 0u;
    // The first border among the run's tokens (a sequence starts there, or the last one ended before it), and
    // the state that it starts from.  One border, and fewer tokens than a run has, are dealt with by
    // selects: branches between the tokens would keep their arithmetic apart (the gradient of 8 x 2048 x 2560
    // took 172 us so, 146 now).  Runs with more borders are rare.
    const int border = kGeneral && borders ? __ffs(borders) - 1 : 2 * kRun;
    const bool many = kGeneral && (borders & (borders - 1)) != 0;
    f32x2 start = 0ull;
    if (kGeneral && border < n && p.h0)
      start = load_f32(p.h0 + (long long)sequence_of(cu, p.N, (int)end, (int)t + border) * p.D + c, vec, c0, c1);
    f32x2 a[kRun], b[kRun];
    f32x2 P = dup2(kWhole), H = 0ull;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      f32x2 s;
      gate2<kGate, kNorm>(pair_at<kNarrow>(gs, i, lane, gsodd), rate, a[i], s);
      b[i] = pair_at<kNarrow>(xs, i, lane, xsodd);
      if (kNorm != GLR_NONE) b[i] = mul2(s, b[i]);
      H = fma2(a[i], kGeneral ? pick(i == border, start, H) : H, b[i]);
      P = mul2(P, a[i]);
    }
    if (kGeneral && many) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        if (borders >> i & 1) {
          f32x2 first = 0ull;
          if (p.h0 && i < n)
            first = load_f32(p.h0 + (long long)sequence_of(cu, p.N, (int)end, (int)t + i) * p.D + c, vec, c0, c1);
          b[i] = fma2(a[i], first, b[i]);
          H = b[i];
        } else {
          H = fma2(a[i], H, b[i]);
        }
      }
    }
    // (behind the last token nothing is read from h: what zeros make of the gates there does not matter)
    s_warp[turn][warp][lane] = make_ulonglong2(kGeneral && border < kRun ? 0ull : at_least(P), H);
    __syncthreads();
    // all the warps' stretches in order; (P, H) becomes what lies before this warp's
    f32x2 sP = dup2(kWhole), sH = 0ull;
    ulonglong2 runs[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) runs[w] = w < warps ? s_warp[turn][w][lane] : make_ulonglong2(dup2(kWhole), 0ull);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) P = sP, H = sH;
      follow<kGeneral>(sP, sH, runs[w].x, runs[w].y);
    }
    f32x2 h = carry;
    if (K > 1) {
      const f32x2 sent = to_send<kGeneral>(sP);
      if (!*dead) {
        for (unsigned k = warp; k < K; k += warps) send_to_rank(&s_rank[(turn * K + rank) * 32 + lane], &s_bar[turn], k, sent, sH);
      }
      // One warp for all: fewer instructions.  In graphs 65536 x 2560 takes 254 us, 265 by every warp, the gradient of
      // 10007 x 1111 108 and 110.
      if (warp == 0) {
        wait_for_ranks(&s_bar[turn], r >> 1 & 1, p.err, dead);
        s_state[lane] = pass_blocks<kGeneral>(carry, s_rank + turn * K * 32 + lane, 32, (int)rank, (int)K);
      }
      __syncthreads();
      h = s_state[lane].x, carry = s_state[lane].y;
    } else {
      carry = through<kGeneral>(sP, sH, carry);
    }
    h = through<kGeneral>(P, H, h);
    if (p.states && t % kGlrChunk == 0 && n)
      store_f32(p.states + (row * p.chunks + t / kGlrChunk) * p.D + c, h, vec, c0, c1);
    T* to = y;
    if (n == kRun && !borders) {
#pragma unroll
      for (int i = 0; i < kRun; ++i, to += p.D) {
        h = fma2(a[i], h, b[i]);
        store_out<kNarrow>(to, h, at);
      }
      if (p.hT && t + kRun == end) store_f32(p.hT + row * p.D + c, h, vec, c0, c1);
    } else if (!many) {
      const int last = packed ? border : t + n == end ? n : 0;  // (the token before it ends its sequence)
      f32x2 final = 0ull;
#pragma unroll
      for (int i = 0; i < kRun; ++i, to += p.D) {
        h = fma2(a[i], kGeneral ? pick(i == border, start, h) : h, b[i]);
        if (i < n) store_out<kNarrow>(to, h, at);
        final = pick(i + 1 == last, h, final);
      }
      if (p.hT && last > 0 && last <= n) {
        const long long q = packed ? sequence_of(cu, p.N, (int)end, (int)t + last - 1) : row;
        store_f32(p.hT + q * p.D + c, final, vec, c0, c1);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRun; ++i, to += p.D) {
        if (i >= n) break;
        h = borders >> i & 1 ? b[i] : fma2(a[i], h, b[i]);
        store_out<kNarrow>(to, h, at);
        if (p.hT && borders >> (i + 1) & 1)
          store_f32(p.hT + (long long)sequence_of(cu, p.N, (int)end, (int)t + i) * p.D + c, h, vec, c0, c1);
      }
    }
    y += (long long)round * p.D;
  }
  cp_async_wait<0>();
  if (K > 1) leave_ranks(dead);
  if (!p.hT || p.hT == p.h0) return;
  if (!packed) {  // no token at all
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

template <auto kKernel, typename T, bool kNarrow>
cudaError_t launch_prompt(GlrParams p, cudaStream_t stream) {
  const size_t smem = kStages * 2 * kTileOf<T, kNarrow> * sizeof(T);
  const int warps = p.T > kRun * (kWarps - 1) ? kWarps : p.T > kRun ? (p.T - 1) / kRun + 1 : 1;
  cudaError_t e = choose_cluster<kKernel, 32 * kWarps>(&p, smem, ((long long)p.T + kRun * kWarps - 1) / (kRun * kWarps));
  if (e == cudaSuccess && p.cluster > 1) e = device_error_word(&p.err);
  if (e != cudaSuccess) return e;
  return launch_clusters(kKernel, glr_grid(p), 32 * warps, p.cluster, p, stream,
                         glr_smem(smem, p.cluster), glr_smem(smem, kGlrMaxCluster));
}
template <typename T, int kGate, int kNorm>
cudaError_t launch(const GlrParams& p, bool step, cudaStream_t stream) {
  if (step) {
    glr_step_kernel<T, kGate, kNorm><<<(unsigned)(((long long)p.N * p.tiles + 3) / 4), 128, 0, stream>>>(p);
    return cudaGetLastError();
  }
  // each has the borders' arithmetic or the odd rows' only where it needs it (packed rows of pairs, 2560 x 32768
  // bf16 forwards, log gate and 1 - a: 180 us, 200 with the arithmetic of odd rows)
  if (!p.vec || p.piece == 2) return launch_prompt<glr_fwd_kernel<T, kGate, kNorm, true, true>, T, true>(p, stream);
  return p.cu ? launch_prompt<glr_fwd_kernel<T, kGate, kNorm, true, false>, T, false>(p, stream)
              : launch_prompt<glr_fwd_kernel<T, kGate, kNorm, false, false>, T, false>(p, stream);
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
