// glr_common.cuh - what the gated linear recurrence's kernels share: channel pairs, gates,
// sequence borders, and the composition of stretches of time.
//
//   h_t = a_t h_{t-1} + s(a_t) x_t,   a = exp(L):
//   gate      L = g (log), log sigmoid(g) (sigmoid), rate sigmoid(g) (rate)
//   weight    s = 1 (none), 1 - a (linear), sqrt(1 - a^2) (sqrt)
//
// A stretch of tokens maps the state before it to A h + H.  Stretches compose, so time is cut
// everywhere: a thread has kRun tokens of two channels, a warp 64 channels, a block's warps
// follow each other in time, and so do the blocks of a cluster.
#pragma once

#include <atomic>
#include <type_traits>

#include "cluster.cuh"
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {

// ---- two channels of a row ---------------------------------------------------------------
// Channels 2 lane, 2 lane + 1 of a warp's 64: in one access where rows are aligned to pairs (vec).
template <typename T>
struct Raw2;
template <>
struct Raw2<__nv_bfloat16> {
  uint32_t v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool vec, bool c0, bool c1) {
    if (vec) {
      v = c0 ? *reinterpret_cast<const uint32_t*>(p) : 0u;
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
      v = (c0 ? (uint32_t)q[0] : 0u) | (c1 ? (uint32_t)q[1] << 16 : 0u);
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, bool vec, bool c0, bool c1) const {
    if (vec) {
      if (c0) *reinterpret_cast<uint32_t*>(p) = v;
    } else {
      uint16_t* q = reinterpret_cast<uint16_t*>(p);
      if (c0) q[0] = (uint16_t)v;
      if (c1) q[1] = (uint16_t)(v >> 16);
    }
  }
  __device__ __forceinline__ f32x2 get() const {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(v << 16), "r"(v & 0xffff0000u));
    return r;
  }
  __device__ __forceinline__ void set(f32x2 x) {
    float a, b;
    unpack2(x, a, b);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(b), "f"(a));
  }
};
template <>
struct Raw2<float> {
  f32x2 v;
  __device__ __forceinline__ void load(const float* p, bool vec, bool c0, bool c1) {
    if (vec) v = c0 ? *reinterpret_cast<const f32x2*>(p) : 0ull;
    else v = pack2(c0 ? p[0] : 0.f, c1 ? p[1] : 0.f);
  }
  __device__ __forceinline__ void store(float* p, bool vec, bool c0, bool c1) const {
    if (vec) {
      if (c0) *reinterpret_cast<f32x2*>(p) = v;
    } else {
      float a, b;
      unpack2(v, a, b);
      if (c0) p[0] = a;
      if (c1) p[1] = b;
    }
  }
  __device__ __forceinline__ f32x2 get() const { return v; }
  __device__ __forceinline__ void set(f32x2 x) { v = x; }
};
__device__ __forceinline__ f32x2 load_f32(const float* p, bool vec, bool c0, bool c1) {
  Raw2<float> r;
  r.load(p, vec, c0, c1);
  return r.v;
}
__device__ __forceinline__ void store_f32(float* p, f32x2 x, bool vec, bool c0, bool c1) {
  Raw2<float> r;
  r.v = x;
  r.store(p, vec, c0, c1);
}
// The pair of an output: a kernel of narrow rows stores in one of two ways, each under its own condition
// (a branch would keep the tokens' arithmetic apart).
struct Places {
  bool pair, first, second;
};
template <bool kNarrow>
__device__ __forceinline__ Places places(bool vec, bool c0, bool c1) {
  return {c0 && (!kNarrow || vec), c0 && !vec, c1 && !vec};
}
template <bool kNarrow, typename T>
__device__ __forceinline__ void store_out(T* p, f32x2 x, const Places& at) {
  Raw2<T> o;
  o.set(x);
  if (at.pair) o.store(p, true, true, true);
  if (kNarrow) {
    if (at.first) o.store(p, false, true, false);
    if (at.second) o.store(p, false, false, true);
  }
}
// Tiles lie in shared memory as tokens of 64 channels, `pitch` elements apart.  Rows of bf16 that are not
// aligned to pairs (odd rows) lie one element further on: bit i of their mask is token i's.
template <typename T, bool kNarrow>
constexpr int kPitch = kNarrow && sizeof(T) == 2 ? 72 : 64;
template <bool kNarrow, typename T>
__device__ __forceinline__ f32x2 pair_at(const T* tile, int token, int lane, unsigned odd) {
  const T* q = tile + token * kPitch<T, kNarrow> + 2 * lane;
  Raw2<T> r;
  r.load(q, true, true, true);
  if constexpr (kNarrow && sizeof(T) == 2) {
    Raw2<T> next;
    next.load(q + 2, true, true, true);
    r.v = __funnelshift_r(r.v, next.v, odd >> token & 1 ? 16 : 0);
  }
  return r.get();
}
// The mask for the tokens from `row` (the first one's address) on.
__device__ __forceinline__ unsigned odd_rows(const void* row, long long stride) {
  const unsigned first = (unsigned)(reinterpret_cast<uintptr_t>(row) >> 1) & 1u;
  return stride & 1 ? (first ? 0x55555555u : 0xaaaaaaaau) : 0u - first;
}

// ---- tiles on their way into shared memory ---------------------------------------------------
// A tile of `tokens` rows of 64 channels from src, `cols` of which exist: zeros for rows from `rows` on and for
// channels that do not exist.
//
// 16 bytes an asynchronous copy where rows are made of, and aligned to, them.  The others are apart from
// the kernels' loop, and not inlined: they are rare, and the loop is to stay in the instruction cache.
template <int kPitch, typename T>
__device__ __forceinline__ void copy_wide(T* tile, const T* src, long long stride, int rows, int tokens, int cols) {
  constexpr int kCols = 16 / (int)sizeof(T), kPieces = 64 / kCols;
  const int row0 = threadIdx.x / kPieces, col = threadIdx.x % kPieces * kCols, step = blockDim.x / kPieces;
  const T* from = src + row0 * stride + col;
  const long long by = step * stride;
  tile += row0 * kPitch + col;
#pragma unroll 4
  for (int row = row0; row < tokens; row += step) {
    const bool ok = col < cols && row < rows;
    cp_async16(tile, ok ? from : src, ok);
    from += by;
    tile += step * kPitch;
  }
}
__device__ __forceinline__ void cp_async4(void* to, const void* from, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(bytes) : "memory");
}
template <int kPitch, typename T>
__device__ __forceinline__ void clear_rows(T* tile, int from, int to) {
  unsigned* words = reinterpret_cast<unsigned*>(tile);
  constexpr int kWords = kPitch * (int)sizeof(T) / 4;
  for (int i = from * kWords + threadIdx.x; i < to * kWords; i += blockDim.x) words[i] = 0u;
}
// 4 bytes an asynchronous copy, a row a warp, nothing but pointers that move on in the loop over the rows
// that exist: a block has few warps, so what counts is the length of the chain of instructions.
template <int kPitch, typename T>
__device__ __noinline__ void copy_words(T* tile, const T* src, long long stride, int rows, int tokens, int cols) {
  constexpr int kCols = 4 / (int)sizeof(T);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  const int col = lane * kCols, have = min(rows, tokens);
  const int some = col < cols ? 4 : 0, more = col + 32 < cols ? 4 : 0;
  const T* from = src + warp * stride + (some ? col : 0);
  T* to = tile + warp * kPitch + col;
  const long long by = warps * stride;
#pragma unroll 8
  for (int row = warp; row < have; row += warps, from += by, to += warps * kPitch) {
    cp_async4(to, from, some);
    if (kCols == 1) cp_async4(to + 32, more ? from + 32 : from, more);
  }
  clear_rows<kPitch>(tile, have, tokens);
}
// Odd rows of bf16 so, 4 aligned bytes a copy: those of a row that begins between two words lie one element
// further on.  A word that the row shares with a neighbour is copied whole, what is not the row's is not
// stored from the tile; the operand's first and last row (from `begin` to `end`), whose words may reach out of
// it, go by elements.  Every other row of a warp begins alike.
template <int kPitch>
__device__ __noinline__ void copy_odd(uint16_t* tile, const uint16_t* src, long long stride, int rows, int tokens,
                                      int cols, const uint16_t* begin, const uint16_t* end) {
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  const int have = min(rows, tokens);
  const unsigned odd = odd_rows(src, stride);
  const auto shift_of = [&](int row) { return (int)(odd >> (row & 31) & 1u); };
  const int lo = src == begin ? 1 : 0;
  const int hi = have > 0 && src + (have - 1) * stride + cols >= end ? have - 1 : have;
  const long long by = 2 * warps * stride;
#pragma unroll 1
  for (int j = 0; j < 2; ++j) {
    int row = warp + j * warps;
    const int shift = shift_of(row), some = 2 * lane - shift < cols ? 4 : 0;
    const uint16_t* from = src + row * stride + (some ? 2 * lane - shift : shift);
    uint16_t* to = tile + row * kPitch + 2 * lane;
    if (row < lo) row += 2 * warps, from += by, to += 2 * warps * kPitch;
#pragma unroll 8
    for (; row < hi; row += 2 * warps, from += by, to += 2 * warps * kPitch) cp_async4(to, from, some);
  }
  if (cols == 64)  // the 33rd words
    for (int row = lo + threadIdx.x; row < hi; row += blockDim.x)
      if (shift_of(row)) cp_async4(tile + row * kPitch + 64, src + row * stride + 63, 4);
  const auto by_elements = [&](int row) {
    for (int col = threadIdx.x; col < cols; col += blockDim.x)
      tile[row * kPitch + shift_of(row) + col] = src[row * stride + col];
  };
  if (lo > 0 && have > 0) by_elements(0);
  if (hi < have && hi >= lo) by_elements(hi);
  clear_rows<kPitch>(tile, have, tokens);
}
// piece: bytes that rows are made of and aligned to; begin, end: the operand
template <bool kNarrow, typename T>
__device__ __forceinline__ void copy_tile(T* tile, const T* src, long long stride, int rows, int tokens, int cols,
                                          int piece, const void* begin, long long length) {
  constexpr int kP = kPitch<T, kNarrow>;
  if (piece == 16) {
    copy_wide<kP>(tile, src, stride, rows, tokens, cols);
  } else if (!kNarrow || sizeof(T) == 4 || piece == 4) {
    copy_words<kP>(tile, src, stride, rows, tokens, cols);
  } else {
    const uint16_t* first = static_cast<const uint16_t*>(begin);
    copy_odd<kP>(reinterpret_cast<uint16_t*>(tile), reinterpret_cast<const uint16_t*>(src), stride, rows, tokens, cols,
                 first, first + length);
  }
}

// ---- gates -------------------------------------------------------------------------------
__device__ __forceinline__ float sqrt_ftz(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <typename F>
__device__ __forceinline__ f32x2 each(f32x2 x, F f) {
  float a, b;
  unpack2(x, a, b);
  return pack2(f(a), f(b));
}

// The gates are computed channel by channel: their constants are operands of scalar instructions.
//
// Every rounding is written out (the compiler may join others in one kernel and not in another: a token's
// gate is to have the same bits in all of them).

// (e^u - 1) / u for |u| < 1/2: the polynomial of degree 6 with the least relative error there (3.0e-9, by
// Remez's exchange; 1.2e-7 with the roundings).
__device__ __forceinline__ float expm1_over(float u) {
  float r = 0.000198411915f;
  r = fmaf(r, u, 0.00139973243f);
  r = fmaf(r, u, 0.00833363459f);
  r = fmaf(r, u, 0.0416653194f);
  r = fmaf(r, u, 0.166666627f);
  r = fmaf(r, u, 0.50000006f);
  return fmaf(r, u, 1.f);
}
__device__ __forceinline__ float exp_of(float x) { return ex2(__fmul_rn(kLog2e, x)); }
// sigmoid(g) and 1 - sigmoid(g), each to its last digits: with e = e^-g and q = 1 / (1 + e) they are q and
// e q, but what is nearer to 1 is 1 less the other.
__device__ __forceinline__ void sigmoid_of(float g, float& sig, float& rest) {
  const float e = exp_of(-g), q = rcp(__fadd_rn(1.f, e));
  const float less = e < 1.f ? __fmul_rn(e, q) : q, more = __fsub_rn(1.f, less);
  sig = e < 1.f ? more : less;
  rest = e < 1.f ? less : more;
}
// The decay a and the input's weight s of a token.  Decays next to 1 come from 1 - a, which keeps its
// digits there: a then is off by one rounding, not by the error of 2^x, whose like sign over the
// thousand tokens that such a decay remembers would show in fp32 sums.
template <int kGate, int kNorm>
__device__ __forceinline__ void gate_of(float g, float rate, float& a, float& s) {
  float left;  // 1 - a
  if (kGate == GLR_SIGMOID) {
    sigmoid_of(g, a, left);
  } else {
    const float log = kGate == GLR_LOG ? g : __fmul_rn(rate, rcp(__fadd_rn(1.f, exp_of(-g))));
    const float e = exp_of(log), over = expm1_over(log);
    const bool near = fabsf(log) < 0.5f;
    a = near ? fmaf(over, log, 1.f) : e;
    if (kNorm != GLR_NONE) left = near ? -__fmul_rn(over, log) : __fsub_rn(1.f, e);
  }
  s = kNorm == GLR_NONE ? 1.f : kNorm == GLR_LINEAR ? left : sqrt_ftz(fmaf(left, a, left));
}
template <int kGate, int kNorm>
__device__ __forceinline__ void gate2(f32x2 g, f32x2 rate, f32x2& a, f32x2& s) {
  float g0, g1, r0, r1, a0, a1, s0, s1;
  unpack2(g, g0, g1);
  unpack2(rate, r0, r1);
  gate_of<kGate, kNorm>(g0, r0, a0, s0);
  gate_of<kGate, kNorm>(g1, r1, a1, s1);
  a = pack2(a0, a1);
  s = pack2(s0, s1);
}

// a where `take`, else b
__device__ __forceinline__ f32x2 pick(bool take, f32x2 a, f32x2 b) {
  float a0, a1, b0, b1;
  unpack2(a, a0, a1);
  unpack2(b, b0, b1);
  return pack2(take ? a0 : b0, take ? a1 : b1);
}

// ---- stretches of time ---------------------------------------------------------------------
// A stretch maps the state h before it to A h + H.  Its product of decays A is held 2^108 times as large (P): by
// itself it underflows within a few tokens of closed gates, and a state near fp32's largest would come out of it
// wrong by up to 4.  P keeps all its digits down to A = 2^-234, and what its roundings below that make of any finite
// state is less than 2^-129, below fp32's normal numbers.  P stays at 2^-149 or above: an infinite state stays
// infinite, as it does token by token, and of finite ones less than 2^-128 is left.  P = 0 (A = 0) is a border: what
// lies behind it sees nothing from before, not even infinities.  (Decays, at most 1; a product above 2^20 would
// overflow.)
constexpr float kWhole = 0x1p108f, kLeast = 0x1p-149f;  // P of no tokens; of an underflown product
__device__ __forceinline__ f32x2 at_least(f32x2 P) {
  return each(P, [](float v) { return fmaxf(v, kLeast); });
}
// H behind a border (P or A = 0), else r
__device__ __forceinline__ f32x2 unless_border(f32x2 P, f32x2 H, f32x2 r) {
  float p0, p1, b0, b1, r0, r1;
  unpack2(P, p0, p1);
  unpack2(H, b0, b1);
  unpack2(r, r0, r1);
  return pack2(p0 == 0.f ? b0 : r0, p1 == 0.f ? b1 : r1);
}
// A x is (f x) k with f = min(P, 1), k = max(P, 1) / 2^108.  One of them is a power of two, 1 for P from 1 on (the
// same bits as of A), and neither step underflows before the result does.
struct Factors {
  f32x2 f, k;
};
__device__ __forceinline__ Factors factors(f32x2 P) {
  return {each(P, [](float v) { return fminf(v, 1.f); }),
          mul2(each(P, [](float v) { return fmaxf(v, 1.f); }), dup2(1.f / kWhole))};
}
template <bool kBorders>
__device__ __forceinline__ f32x2 through(f32x2 P, f32x2 H, f32x2 h) {  // A h + H
  const Factors a = factors(P);
  const f32x2 r = fma2(mul2(a.f, h), a.k, H);
  return kBorders ? unless_border(P, H, r) : r;
}
// (P, H) followed by (Q, G)
template <bool kBorders>
__device__ __forceinline__ void follow(f32x2& P, f32x2& H, f32x2 Q, f32x2 G) {
  const Factors b = factors(Q);
  H = through<kBorders>(Q, G, H);
  const f32x2 product = at_least(mul2(mul2(b.f, P), b.k));
  P = kBorders ? unless_border(P, 0ull, unless_border(Q, 0ull, product)) : product;
}

// What a block of a cluster sends of its stretch: A, or -P of a lane's two channels if one of them is deep, P < 1,
// which 64 tokens rarely are.  The receivers go through all as if none were, and again if a sign says so (the
// factors of all for all made 65536 x 2560 7 % slower).
template <bool kBorders>
__device__ __forceinline__ f32x2 to_send(f32x2 P) {
  float p0, p1;
  unpack2(P, p0, p1);
  const bool deep = fminf(p0, p1) < 1.f && !(kBorders && P == 0ull);
  return mul2(P, dup2(deep ? -1.f : 1.f / kWhole));
}
// The states before the block after `first` others of the cluster's, and behind all of them, from h before them.
template <bool kBorders>
__device__ __forceinline__ ulonglong2 pass_blocks(f32x2 h, const ulonglong2* sent, int step, int first, int blocks) {
  const f32x2 h0 = h;
  unsigned signs = 0u;
  const auto some = [&](int from, int to) {
#pragma unroll 4
    for (int k = from; k < to; ++k) {
      const ulonglong2 v = sent[k * step];
      signs |= (unsigned)(v.x >> 32);
      const f32x2 r = fma2(v.x, h, v.y);
      h = kBorders ? unless_border(v.x, v.y, r) : r;
    }
  };
  some(0, first);
  f32x2 before = h;
  some(first, blocks);
  if ((int)signs < 0) {
    h = h0;
#pragma unroll 1
    for (int k = 0; k < blocks; ++k, sent += step) {
      const ulonglong2 v = *sent;
      before = pick(k == first, h, before);
      h = through<kBorders>(mul2(v.x, dup2((long long)v.x < 0 ? -1.f : kWhole)), v.y, h);
    }
  }
  return make_ulonglong2(before, h);
}

// ---- sequence borders of a packed row ------------------------------------------------------
// The first m in [0, N] with min(max(cu[m], 0), end) > v, N + 1 if there is none; by a warp,
// 32 places at a time.  In range whatever the table holds.
__device__ __forceinline__ int first_border_above(const int32_t* cu, int N, int end, int v) {
  const int lane = threadIdx.x & 31;
  long long lo = 0, hi = (long long)N + 1;
  while (lo < hi) {
    const long long step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool above = at >= hi || min(max(cu[at], 0), end) > v;
    const unsigned votes = __ballot_sync(0xffffffffu, above);
    const int first = votes ? __ffs(votes) - 1 : 32;
    if (first == 0) return (int)lo;
    const long long top = lo + first * step;
    lo += (first - 1) * step + 1;
    if (top < hi) hi = top;
  }
  return (int)lo;
}
// The table, in shared memory where it fits: a search takes three reads, one after the other.
constexpr int kBorders = 512;
__device__ __forceinline__ const int32_t* take_borders(const GlrParams& p, int32_t* table) {
  if (!p.cu || p.N >= kBorders) return p.cu;
  for (int i = threadIdx.x; i <= p.N; i += blockDim.x) table[i] = p.cu[i];
  return table;  // (complete after the block's next barrier)
}
// The sequence that holds token v.  (Not inlined: the loops over a thread's tokens are unrolled.)
static __device__ __noinline__ int sequence_of(const int32_t* cu, int N, int end, int v) {
  return min(max(first_border_above(cu, N, end, v) - 1, 0), N - 1);
}
// Bit i: a sequence starts at token t + i, or the last one ends before it (i <= run).
static __device__ __noinline__ unsigned borders_of(const int32_t* cu, int N, int end, int t, int run) {
  int m = first_border_above(cu, N, end, t);
  unsigned bits = m > 0 && min(max(cu[m - 1], 0), end) == t ? 1u : 0u;
  while (m <= N) {
    const int b = min(max(cu[m], 0), end);  // above t, and above the one before
    if (b - t > run) break;
    bits |= 1u << (b - t);
    if (b >= end) break;
    m = first_border_above(cu, N, end, b);
  }
  return bits;
}

// ---- launches --------------------------------------------------------------------------------
// Blocks of a cluster: they go on together through a row's `spans`, and as many clusters as there is room
// for run at once, which depends on the size (bf16 forwards 74 clusters of 8 and 35 of 14, the gradient in fp32 36
// and 7).  The size with the fewest rounds over all waves of clusters is taken.  The GPU is
// asked once for each kernel and size: rows of more than one span have blocks of kThreads threads, the others one
// block of however many.
inline size_t glr_smem(size_t tiles, int blocks) { return tiles + (blocks > 1 ? blocks * 1024 : 0); }
template <auto kKernel, unsigned kThreads>
cudaError_t choose_cluster(GlrParams* p, size_t tiles, long long spans) {
  static std::atomic<int> room[kGlrMaxCluster + 1];
  const long long units = glr_units(*p);
  long long best = -1;
  p->cluster = 1;
  if (spans <= 1) return cudaSuccess;
  for (int k = 1; k <= kGlrMaxCluster && k <= spans; ++k) {
    const size_t smem = glr_smem(tiles, k);
    int n = room[k].load(std::memory_order_relaxed);
    if (!n) {
      cudaError_t e = allow_clusters(kKernel, k, glr_smem(tiles, kGlrMaxCluster));
      if (e != cudaSuccess) return e;
      const ClusterConfig c(k, kThreads, k, smem, nullptr);
      if (k == 1) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kKernel, kThreads, smem);
        n *= kSms;
      } else {
        e = cudaOccupancyMaxActiveClusters(&n, kKernel, &c.cfg);
      }
      if (e != cudaSuccess) return e;
      n = n < 1 ? -1 : n;
      room[k].store(n, std::memory_order_relaxed);
    }
    if (n < 0) continue;
    // (a wave's start costs about two rounds)
    const long long cost = ((units + n - 1) / n) * ((spans + k - 1) / k + 2);
    if (best < 0 || cost < best) best = cost, p->cluster = k;
  }
  return best < 0 ? cudaErrorInvalidConfiguration : cudaSuccess;
}

}  // namespace gdn
