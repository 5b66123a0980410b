// s6_scan.cuh - the selective state space scan with a diagonal A (S6, the Mamba-1 member of
// the linear-attention family), for prompts.
//
// Per sequence, channel d and state n, tokens in order, D_t = softplus(dt_t + dt_bias) (or
// dt_t + dt_bias):
//
//   h_t[n] = exp(D_t A[n]) h_{t-1}[n] + D_t x_t B_t[n],
//   y_t    = (sum_n C_t[n] h_t[n] + Dskip x_t) silu(z_t).
//
// Every (token, channel, state) has a decay of its own, so there is no matrix product to
// form: per state one exponential (the special-function unit, 32 a clock and SM here) and
// four multiplies or multiply-adds (128 a clock and SM), which take about the same time.
// Multiply-adds are in packed fp32 pairs where both operands are pairs already, which halves
// the instructions issued, not the pipe's time.
//
// Layout.  LPC = Ns / 4 lanes share a channel pair (or a channel, below) and a lane keeps four
// states of it in registers; a CTA has 32 channels and walks its tokens in tiles.  The
// recurrence of one warp per scheduler cannot hide a load or a quotient, so the warps are of
// two kinds: the computing threads do nothing but the recurrence, out of shared memory, and
// the helper threads beside them prepare the next tile and finish the last one.  Per tile the
// helpers form (D_t, D_t x_t) once per token and channel, and B and C as fp32; add the lanes'
// partial sums over n, the skip and the gate into y; and keep the copies of the coming tiles in
// flight (cp.async, a ring of four).  One barrier a tile.
//
// What it works against is the path between the schedulers and the special-function units and shared
// memory: a lane takes 4 bytes a clock and SM from shared memory, whatever lanes share, so the
// bytes per (channel, state) count.  A lane with four states of two channels reads 6 (D and Dx
// 16 bytes, B and C 32, for 8 products); one with a single channel 10, or 6 where it takes bf16 B
// and C as they are.  Cycles an SM takes for a token of 32 channels (Ns = 16, 1.92 GHz, 16384
// tokens of 4864 channels a sequence): bf16 58 with one CTA an SM (one channel a lane), 54 with
// two, 46 with four; fp32 62, 55 and 51.  The exponentials alone are 16, the multiply-adds 16,
// the reads 24 or more.  4096 tokens of 5120 channels take 145 us; their bytes alone would take
// 25.  Whole sequences, one CTA an SM, keep neither the issue slots (57 %) nor the shared-memory path
// (57 %) full: the barrier of every tile, where the two kinds of warps wait for one another, is
// their first stall.
//
// Splitting over time.  A CTA per 32 channels leaves SMs idle when there are few of them.
// Channels beyond the whole-sequence ones are split over time: a first launch computes the
// state that each chunk of tokens ends in from a zero state, and the sum of its steps (the
// decay over the chunk is exp(A sum D_t)); the scan then starts each chunk from the chunks
// before it.  That computes the exponentials twice; s6_split says where it pays.
#pragma once

#include "gdn_common.cuh"
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {
namespace {

constexpr int kCh = 32;   // channels per CTA
constexpr int kRing = 4;  // tiles of raw inputs in shared memory
constexpr int kPairs = kCh / 2;

// How a channel's states fill its LPC lanes, four each: all of them (Ns = 4 LPC), some of them (Ns a
// multiple of 4), or with fewer than four in a lane.
enum class Fill { kAll, kSome, kPart };

// A variant: T inputs, LPC lanes per channel or channel pair, kWidth channels a lane, tiles of
// kTokens.  Sizes of shared memory are in pieces of 16 bytes.
template <typename T_, int LPC_, int kWidth_, int kTokens, Fill kFill, bool kSummary_>
struct Cfg {
  using T = T_;
  static constexpr int LPC = LPC_, kWidth = kWidth_, kTile = kTokens;
  static constexpr bool kPad = kFill == Fill::kPart, kEmpty = kFill == Fill::kSome;
  static constexpr bool kSummary = kSummary_;
  static constexpr int kUnits = kCh / kWidth;  // channel pairs, or channels
  static constexpr int kCompute = kUnits * LPC < 32 ? 32 : kUnits * LPC;
  static constexpr int kHelpers = kPairs * kTile / 4;  // one has 2 channels x 4 tokens of a tile
  // Alone on its SM a CTA waits for the helpers' chains: one set of them prepares tiles, another
  // finishes them (x for the skip then comes from a longer ring).
  static constexpr bool kApart = kWidth == 1;
  static constexpr int kThreads = kCompute + kHelpers * (kApart ? 2 : 1);
  // two computing warps and two helpers: one of each kind of warp a scheduler
  static constexpr bool kPlace = kCompute == 64 && kThreads == 128;
  // a raw row: 32 channels and 16 bytes more, so that rows 4 apart meet other banks
  static constexpr int kRowPieces = kCh * (int)sizeof(T) / 16, kPitch = kRowPieces + 1;
  static constexpr int kRawTile = kTile * kPitch;
  static constexpr int kCopies = kTile * kRowPieces / kHelpers;  // per helper, tensor and tile
  static constexpr int kDuTile = kPairs * (kTile + 1);  // (D0, D0 x0, D1, D1 x1) a pair and token
  // four states' B and C of a token: one piece in bf16, two in fp32.  They are read where they
  // arrive, except that lanes with two channels have bf16 widened for them by the helpers, into
  // two further tiles: there instructions count more than bytes (51 cycles against 55 where the
  // lanes widen their own), with one channel a lane the bytes do (the recurrence alone: 52 cycles
  // packed, 58 widened).
  static constexpr bool kWiden = sizeof(T) == 2 && kWidth > 1, kPacked = sizeof(T) == 2 && !kWiden;
  static constexpr int kFours = kTile * LPC, kPerHelper = (kFours + kHelpers - 1) / kHelpers;
  static constexpr int kBcPieces = (int)sizeof(T) / 2, kBcTile = kFours * kBcPieces;
  static constexpr int kWideTile = kFours * 2;
  // partial sums of y: kParts rows a pair (8 or 16 lanes add up to 4 by shuffles first) of
  // kTile / 2 pieces, each two tokens of one channel and of the other.  Rows of kTile / 2 + 2
  // pieces, moved on by one every pair: with 4 lanes the writes (8 lanes: 2 pairs x 4 rows)
  // and the reads (8 pairs) both spread over the banks.
  static constexpr int kParts = LPC < 4 ? LPC : 4, kLanes = LPC / kParts;
  static constexpr int kPartRow = kTile / 2 + 2, kPartPair = kParts * kPartRow + 1;
  static constexpr int kPartTile = kSummary ? 0 : kPairs * kPartPair;
  static constexpr int kRingX = kApart ? 2 * kRing : kRing;
  static constexpr int kX = 0, kDt = kX + kRingX * kRawTile, kZ = kDt + kRing * kRawTile;
  static constexpr int kDu = kZ + (kSummary ? 0 : kRing * kRawTile);
  static constexpr int kBc = kDu + 2 * kDuTile;
  static constexpr int kWide = kBc + kRing * kBcTile;
  static constexpr int kPart = kWide + (kWiden ? 2 * kWideTile : 0);
  static constexpr int kPieces = kPart + (kSummary ? kTile / 4 * kCh / 4 : 2 * kPartTile);
  static constexpr int kBytes = kPieces * 16;
  // The one-channel variant is for one CTA an SM: more than half of the shared memory, so that
  // no SM takes two while others have none.
  static constexpr int kAsked = kWidth == 1 && kBytes < 116 * 1024 ? 116 * 1024 : kBytes;
  // CTAs per SM: by shared memory, and by registers with at least 112 a thread, or 128 with 8
  // lanes, which spill with less (4 x 1024 tokens of 2432 channels, 32 states: 129 us against 119)
  static constexpr int kRegs = LPC == 8 ? 128 : 112;
  static constexpr int kBySmem = 227 * 1024 / (kAsked + 1024), kByRegs = 65536 / kRegs / kThreads;
  static constexpr int kBlocks = kBySmem < kByRegs ? kBySmem : kByRegs < 1 ? 1 : kByRegs;
};

// Two neighbouring channels of a raw row in shared memory.
template <typename T>
struct Raw2;
template <>
struct Raw2<__nv_bfloat16> {
  uint32_t v;
  __device__ __forceinline__ void load(const float4* row, int pair) {
    v = reinterpret_cast<const uint32_t*>(row)[pair];
  }
  __device__ __forceinline__ f32x2 get() const {
    return pack2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
};
template <>
struct Raw2<float> {
  f32x2 v;
  __device__ __forceinline__ void load(const float4* row, int pair) {
    v = reinterpret_cast<const f32x2*>(row)[pair];
  }
  __device__ __forceinline__ f32x2 get() const { return v; }
};
__device__ __forceinline__ void store2(__nv_bfloat16* p, f32x2 v, int n, bool vec) {
  float a, b;
  unpack2(v, a, b);
  if (vec) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(a, b);
  } else {
    if (n > 0) p[0] = __float2bfloat16_rn(a);
    if (n > 1) p[1] = __float2bfloat16_rn(b);
  }
}
__device__ __forceinline__ void store2(float* p, f32x2 v, int n, bool vec) {
  float a, b;
  unpack2(v, a, b);
  if (vec) {
    *reinterpret_cast<float2*>(p) = make_float2(a, b);
  } else {
    if (n > 0) p[0] = a;
    if (n > 1) p[1] = b;
  }
}
// Four bf16 in two words, as fp32.
__device__ __forceinline__ float4 wide4(float lo, float hi) {
  const uint32_t x = __float_as_uint(lo), y = __float_as_uint(hi);
  return make_float4(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u),
                     __uint_as_float(y << 16), __uint_as_float(y & 0xffff0000u));
}
// cp.async of 8 bytes (16: cp_async16), zeros where !ok
__device__ __forceinline__ void cp_async8(void* dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(smem_u32(dst)), "l"(src),
               "r"(ok ? 8 : 0)
               : "memory");
}
// cp.async of 4 bytes; zeros where !ok, and then nothing is read at src
__device__ __forceinline__ void cp_async4(void* dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(smem_u32(dst)), "l"(src),
               "r"(ok ? 4 : 0)
               : "memory");
}

// What a CTA works on: tokens [t0, t1) of sequence n (rows of the whole batch), 32 channels
// from ch0 on.
struct Task {
  int n, c;            // sequence, chunk of it (0: also a whole sequence)
  int ch0;
  long long t0, t1;
  bool last;           // the sequence ends here
  bool split;          // one of several chunks: there are summaries
};
// Borders read from the device are clamped to the batch.
__device__ __forceinline__ int border(const S6Params& p, int i) { return min(max(p.cu[i], 0), p.T); }
// Chunk c of sequence n lives in slot floor(cu[n] / chunk) + n + c (fixed-length rows:
// n ceil(T / chunk) + c); the slots of different sequences never meet.
__device__ __forceinline__ long long first_slot(const S6Params& p, int n) {
  if (p.cu) return (long long)(border(p, n) / p.chunk) + n;
  return (long long)n * ((p.T + p.chunk - 1) / p.chunk);
}
// Block -> task; false for a slot that no chunk uses.
__device__ __forceinline__ bool find_task(const S6Params& p, bool summary, int tiles, Task* k) {
  int b = blockIdx.x;
  const int whole = summary ? 0 : p.N * p.whole;
  k->c = 0;
  k->split = b >= whole;
  if (!k->split) {
    k->n = b / p.whole;
    k->ch0 = b % p.whole * kCh;
  } else {
    b -= whole;
    const int parts = tiles - p.whole, slot = b / parts;
    k->ch0 = (p.whole + b % parts) * kCh;
    if (!p.cu) {
      const int per = (p.T + p.chunk - 1) / p.chunk;
      k->n = slot / per;
      k->c = slot % per;
    } else {
      // the last sequence that begins at the slot or before it: 32 of them tried at once
      int lo = 0, hi = p.N - 1;
      while (lo < hi) {
        const int step = (hi - lo + 31) / 32, i = lo + ((int)(threadIdx.x & 31) + 1) * step;
        const bool before = i <= hi && border(p, i) / p.chunk + i <= slot;
        lo += __popc(__ballot_sync(0xffffffffu, before)) * step;
        hi = min(hi, lo + step - 1);
      }
      k->n = lo;
      k->c = slot - (border(p, lo) / p.chunk + lo);
      if (k->c < 0) return false;
    }
  }
  long long begin, end;
  if (p.cu) {
    begin = border(p, k->n);
    end = max((long long)border(p, k->n + 1), begin);
  } else {
    begin = (long long)k->n * p.T;
    end = begin + p.T;
  }
  k->t0 = begin;
  k->t1 = end;
  k->last = true;
  if (k->split) {
    k->t0 = begin + (long long)k->c * p.chunk;
    if (k->t0 >= end && k->c > 0) return false;
    if (k->t0 + p.chunk < end) {
      k->t1 = k->t0 + p.chunk;
      k->last = false;
    }
  }
  return true;
}

// The computing threads' part: the recurrence over the tiles.
template <class C>
__device__ __forceinline__ void s6_compute(const S6Params& p, const Task& k, float4* smem, int nt,
                                           int tid) {
  constexpr int kTile = C::kTile, LPC = C::LPC, kWidth = C::kWidth;
  constexpr bool kSummary = C::kSummary;
  const int unit = tid / LPC, ln = tid % LPC;  // LPC = 1: only 16 of the 32 lanes have a pair
  const bool idle = C::kUnits * LPC < 32 && unit >= C::kUnits;
  const int ch = k.ch0 + unit * kWidth, n0 = ln * 4;
  const int chs = idle ? 0 : max(0, min(kWidth, p.dim - ch));  // channels that exist
  const int nst = chs > 0 ? max(0, min(4, p.Ns - n0)) : 0;     // and states of them
  const long long hsize = (long long)p.dim * p.Ns;
  // the workspace holds the split channels only
  const int off = p.whole * kCh, wdim = p.dim - off;
  const long long wsize = (long long)wdim * p.Ns;

  f32x2 a[kWidth][2], h[kWidth][2];
  const bool kept = k.split && p.ws_h0;  // hT == h0: the scan reads the copy
  if (!kSummary && (k.c > 0 || kept)) griddep_wait();
#pragma unroll
  for (int j = 0; j < kWidth; ++j) {
    const int n = j < chs ? nst : 0;
    const long long hrow = (long long)(ch + j) * p.Ns + n0, wrow = hrow - (long long)off * p.Ns;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n > 0) v = load_h(p.A + hrow, n, p.Ns);
    a[j][0] = pack2(v.x * kLog2e, v.y * kLog2e);
    a[j][1] = pack2(v.z * kLog2e, v.w * kLog2e);
    h[j][0] = h[j][1] = pack2(0.f, 0.f);
    if (n > 0 && k.c == 0) {
      if (p.h0) {
        v = !kSummary && kept ? load_h(p.ws_h0 + k.n * wsize + wrow, n, p.Ns)
                              : load_h(p.h0 + k.n * hsize + hrow, n, p.Ns);
        h[j][0] = pack2(v.x, v.y);
        h[j][1] = pack2(v.z, v.w);
        if (kSummary && kept) store_h(p.ws_h0 + k.n * wsize + wrow, v, n, p.Ns);
      }
    } else if (n > 0 && !kSummary) {  // the state before this chunk, from the chunks before it
      const long long s0 = first_slot(p, k.n);
#pragma unroll 4
      for (int i = 0; i < k.c; ++i) {
        v = load_h(p.ws_h + (s0 + i) * wsize + wrow, n, p.Ns);
        const f32x2 s = dup2(p.ws_sum[(s0 + i) * wdim + ch + j - off]);
        float e0, e1, e2, e3;
        unpack2(mul2(a[j][0], s), e0, e1);
        unpack2(mul2(a[j][1], s), e2, e3);
        // a decay that would be 0 over the chunk, though no token's is, is 2^-126: an infinite state
        // stays infinite (0 times infinity is NaN).  What a finite state keeps of it is below any
        // rounding; where a sum is infinite or NaN, so is the chunk's own state.
        h[j][0] = fma2(pack2(ex2(fmaxf(e0, -126.f)), ex2(fmaxf(e1, -126.f))), h[j][0], pack2(v.x, v.y));
        h[j][1] = fma2(pack2(ex2(fmaxf(e2, -126.f)), ex2(fmaxf(e3, -126.f))), h[j][1], pack2(v.z, v.w));
      }
    }
  }

  struct In {  // a step's operands as they lie in shared memory
    float d[kWidth], u[kWidth];
    float4 b, c;
  };
  struct Ready {  // what the recurrence of a step needs: decays, inputs, C
    f32x2 a[kWidth][2], u[kWidth][2], c01, c23;
  };
  const int pair = idle ? 0 : unit * kWidth / 2, sub = kWidth == 1 ? unit & 1 : 0;
  for (int i = -1; i <= nt; ++i) {
    if (i >= 0 && i < nt) {
      const float4* du = smem + C::kDu + (i & 1) * C::kDuTile + pair * (kTile + 1);
      constexpr int kFour = C::kPacked ? 1 : 2;  // pieces of a token's four states
      const float4* bc = (C::kWiden ? smem + C::kWide + (i & 1) * C::kWideTile
                                    : smem + C::kBc + (i & (kRing - 1)) * C::kBcTile) + kFour * ln;
      float4* part = smem + C::kPart + (i & 1) * C::kPartTile + pair * C::kPartPair +
                     ln / C::kLanes * C::kPartRow;
      struct Two {
        float y[kWidth][2];
      };
      auto put = [&](int t, Two v) {  // the sums of tokens t and t + 1
        // A lane without states has A, B and C of zero, but an infinite step or input makes its
        // sums NaN (0 times infinity): they do not count.  (Kernels apart: 4096 tokens of 5120
        // channels, 24 states, bf16 238 us without the selects, 246 with; 12 states 148, 150.)
        if (C::kEmpty) {
#pragma unroll
          for (int j = 0; j < kWidth; ++j)
            v.y[j][0] = nst ? v.y[j][0] : 0.f, v.y[j][1] = nst ? v.y[j][1] : 0.f;
        }
#pragma unroll
        for (int o = 1; o < C::kLanes; o *= 2)
#pragma unroll
          for (int j = 0; j < kWidth; ++j) {
            v.y[j][0] += __shfl_xor_sync(0xffffffffu, v.y[j][0], o);
            v.y[j][1] += __shfl_xor_sync(0xffffffffu, v.y[j][1], o);
          }
        // (no branch where every lane writes: it would keep the steps apart)
        if ((C::kLanes == 1 || ln % C::kLanes == 0) && !idle) {
          if constexpr (kWidth == 2)
            part[t / 2] = make_float4(v.y[0][0], v.y[0][1], v.y[1][0], v.y[1][1]);
          else
            reinterpret_cast<float2*>(part + t / 2)[sub] = make_float2(v.y[0][0], v.y[0][1]);
        }
      };
      auto fetch = [&](int t) {
        In r;
        if constexpr (kWidth == 2) {
          const float4 v = du[t];
          r.d[0] = v.x, r.u[0] = v.y, r.d[1] = v.z, r.u[1] = v.w;
        } else {
          const float2 v = reinterpret_cast<const float2*>(du + t)[sub];
          r.d[0] = v.x, r.u[0] = v.y;
        }
        r.b = bc[t * LPC * kFour];
        if (!kSummary && !C::kPacked) r.c = bc[t * LPC * kFour + 1];
        return r;
      };
      auto ready = [&](const In& in) {
        Ready r;
        const float4 b = C::kPacked ? wide4(in.b.x, in.b.y) : in.b;
        const float4 c = C::kPacked ? wide4(in.b.z, in.b.w) : in.c;
#pragma unroll
        for (int j = 0; j < kWidth; ++j) {
          const f32x2 d = dup2(in.d[j]), u = dup2(in.u[j]);
          float e0, e1, e2, e3;
          unpack2(mul2(a[j][0], d), e0, e1);
          unpack2(mul2(a[j][1], d), e2, e3);
          r.a[j][0] = pack2(ex2(e0), ex2(e1));
          r.a[j][1] = pack2(ex2(e2), ex2(e3));
          r.u[j][0] = mul2(pack2(b.x, b.y), u);
          r.u[j][1] = mul2(pack2(b.z, b.w), u);
        }
        if (!kSummary) r.c01 = pack2(c.x, c.y), r.c23 = pack2(c.z, c.w);
        return r;
      };
      auto step = [&](const Ready& r, int j) -> float {
        h[j][0] = fma2(r.a[j][0], h[j][0], r.u[j][0]);
        h[j][1] = fma2(r.a[j][1], h[j][1], r.u[j][1]);
        if (C::kPad) {  // states that do not exist stay zero whatever the step
          float v0, v1, v2, v3;
          unpack2(h[j][0], v0, v1);
          unpack2(h[j][1], v2, v3);
          h[j][0] = pack2(nst > 0 ? v0 : 0.f, nst > 1 ? v1 : 0.f);
          h[j][1] = pack2(nst > 2 ? v2 : 0.f, nst > 3 ? v3 : 0.f);
        }
        if (kSummary) return 0.f;
        float y0, y1;
        unpack2(fma2(r.c01, h[j][0], mul2(r.c23, h[j][1])), y0, y1);
        return y0 + y1;
      };
      const long long left = k.t1 - (k.t0 + (long long)i * kTile);
      if (left >= kTile) {
        // in flight at once: the operands of step t + 2 are read, the decays of t + 1 formed,
        // and the recurrence takes t
        In in = fetch(0);
        Ready now = ready(in);
        in = fetch(1);
        Two out[2];  // sums wait two steps, so that their store waits for nothing
#pragma unroll
        for (int t = 0; t < kTile; ++t) {
          In later;
          Ready next;
          if (t + 2 < kTile) later = fetch(t + 2);
          if (!kSummary && t >= 2 && t % 2 == 0) put(t - 2, out[t / 2 % 2 ^ 1]);
          if (t + 1 < kTile) next = ready(in);
#pragma unroll
          for (int j = 0; j < kWidth; ++j) out[t / 2 % 2].y[j][t % 2] = step(now, j);
          if (t + 1 < kTile) now = next;
          if (t + 2 < kTile) in = later;
        }
        if (!kSummary) put(kTile - 2, out[(kTile / 2 - 1) % 2]);
      } else {
        Two out = {};
        for (int t = 0; t < (int)left; ++t) {
          const Ready r = ready(fetch(t));
#pragma unroll
          for (int j = 0; j < kWidth; ++j) {
            const float y = step(r, j);
            if (t % 2 == 0) out.y[j][0] = y; else out.y[j][1] = y;
          }
          if (!kSummary && (t % 2 == 1 || t + 1 == (int)left)) put(t, out);
        }
      }
    }
    named_sync(2, C::kThreads);
  }

#pragma unroll
  for (int j = 0; j < kWidth; ++j) {
    const int n = j < chs ? nst : 0;
    const long long hrow = (long long)(ch + j) * p.Ns + n0, wrow = hrow - (long long)off * p.Ns;
    float4 v;
    unpack2(h[j][0], v.x, v.y);
    unpack2(h[j][1], v.z, v.w);
    if (n <= 0) continue;
    if (kSummary) store_h(p.ws_h + (first_slot(p, k.n) + k.c) * wsize + wrow, v, n, p.Ns);
    else if (k.last && p.hT) store_h(p.hT + k.n * hsize + hrow, v, n, p.Ns);
  }
}

// The helper threads' part.  In iteration i the computing threads are at tile i; the helpers
// start the copies of tiles to come (x and dt of tile i + 4, B and C of i + 4 or i + 3, z of
// i + 2: the ring's places are free then), stage tile i + 1 (kStage) and write y of tile i - 1 (kFinish).
template <class C, bool kStage, bool kFinish>
__device__ __forceinline__ void s6_help(const S6Params& p, const Task& k, float4* smem, int nt,
                                        int tid) {
  using T = typename C::T;
  constexpr int kTile = C::kTile, LPC = C::LPC;
  constexpr bool kSummary = C::kSummary;
  const int pair = tid % kPairs, quad = tid / kPairs;
  const int c = k.ch0 + 2 * pair, left = p.dim - c;
  const f32x2 bias = pack2(p.dt_bias && left > 0 ? p.dt_bias[c] : 0.f,
                           p.dt_bias && left > 1 ? p.dt_bias[c + 1] : 0.f);
  const f32x2 skip = pack2(kFinish && p.D && left > 0 ? p.D[c] : 0.f,
                           kFinish && p.D && left > 1 ? p.D[c + 1] : 0.f);

  // One tile of x (0), dt (1) or z (2) into the ring; rows and channels that do not exist: 0.
  // Rows on 4-byte boundaries only are copied by words, bf16 rows off those through registers,
  // loaded at the start of an iteration and stored at its end.
  constexpr int kEach = 16 / (int)sizeof(T), kWord = 4 / (int)sizeof(T);
  constexpr int kRowStep = C::kHelpers / C::kRowPieces;  // rows between a thread's copies
  const int row0 = tid / C::kRowPieces, piece = tid % C::kRowPieces;
  const int ch = k.ch0 + piece * kEach;
  const int some = max(0, p.dim - ch);  // channels of the piece that exist
  const int len = (int)(k.t1 - k.t0);
  const T* src[3] = {static_cast<const T*>(p.x) + (some ? (k.t0 + row0) * p.x_stride + ch : 0),
                     static_cast<const T*>(p.dt) + (some ? (k.t0 + row0) * p.dt_stride + ch : 0),
                     static_cast<const T*>(p.z) + (some ? (k.t0 + row0) * p.z_stride + ch : 0)};
  constexpr bool kHalves = sizeof(T) == 2;
  Raw8<__nv_bfloat16> late[kHalves ? 3 * C::kCopies : 1];
  auto place = [&](int tensor, int i, int j) {
    const int tile = tensor == 0   ? C::kX + (i & (C::kRingX - 1)) * C::kRawTile
                     : tensor == 1 ? C::kDt + (i & (kRing - 1)) * C::kRawTile
                                   : C::kZ + (i & (kRing - 1)) * C::kRawTile;
    return smem + tile + (row0 + j * kRowStep) * C::kPitch + piece;
  };
  auto copy = [&](int tensor, long long stride, int i) {
    if (i >= nt) return;
    const int rows = len - i * kTile - row0;  // from this thread's first one on
#pragma unroll
    for (int j = 0; j < C::kCopies; ++j) {
      const bool ok = j * kRowStep < rows && some;
      const T* s = ok ? src[tensor] + j * kRowStep * stride : src[tensor];
      float4* dst = place(tensor, i, j);
      if (p.copy == 16) {
        cp_async16(dst, s, ok);
      } else if (p.copy == 4) {
#pragma unroll
        for (int w = 0; w < 4; ++w)
          cp_async4(reinterpret_cast<uint32_t*>(dst) + w, s + w * kWord, w * kWord < (ok ? some : 0));
      } else if constexpr (kHalves) {
        late[tensor * C::kCopies + j].load_n(s, ok ? some : 0);
      }
    }
    if (rows > kTile) src[tensor] += kTile * stride;  // stays inside the tensor
  };
  auto copy_late = [&](int tensor, int i) {
    if constexpr (kHalves) {
      if (p.copy == 2 && i < nt) {
#pragma unroll
        for (int j = 0; j < C::kCopies; ++j)
          *reinterpret_cast<uint4*>(place(tensor, i, j)) = late[tensor * C::kCopies + j].v;
      }
    }
  };
  // B and C of a tile, four states of a token at a time, into their ring
  static_assert(C::kPerHelper == 1 || C::kHelpers % LPC == 0, "a thread's fours: the same states");
  const int brow = tid / LPC, n0 = tid % LPC * 4;
  const int nst = max(0, p.Ns - n0);
  const T* bs = static_cast<const T*>(p.B) + (nst ? (k.t0 + brow) * p.b_stride + n0 : 0);
  const T* cs = static_cast<const T*>(p.C) + (nst ? (k.t0 + brow) * p.c_stride + n0 : 0);
  // Copies are complete three iterations after the one that starts them.  Widened, B and C are
  // read while their tile is staged, with x and dt; as they are, one iteration later.
  constexpr int kBcAhead = C::kWiden ? 4 : 3;
  auto copy_bc = [&](int i) {
    if (i >= nt) return;
    const int rows = len - i * kTile - brow;
#pragma unroll
    for (int j = 0; j < C::kPerHelper; ++j) {
      const int id = tid + j * C::kHelpers, r = j * (C::kHelpers / LPC);
      if (id >= C::kFours) break;
      float4* dst = smem + C::kBc + (i & (kRing - 1)) * C::kBcTile + id * C::kBcPieces;
      T* dst_c = reinterpret_cast<T*>(dst) + 4;
      const bool ok = r < rows && nst;
      const T *sb = ok ? bs + r * p.b_stride : bs, *sc = ok ? cs + r * p.c_stride : cs;
      if (p.copy_bc == 16) {
        cp_async16(dst, sb, ok);
        if (!kSummary) cp_async16(dst_c, sc, ok);
      } else if (p.copy_bc == 8) {
        cp_async8(dst, sb, ok);
        if (!kSummary) cp_async8(dst_c, sc, ok);
      } else if (p.copy_bc == 4) {
#pragma unroll
        for (int w = 0; w < (int)sizeof(T); ++w) {
          const bool in = w * kWord < (ok ? nst : 0);
          cp_async4(reinterpret_cast<uint32_t*>(dst) + w, sb + w * kWord, in);
          if (!kSummary) cp_async4(reinterpret_cast<uint32_t*>(dst_c) + w, sc + w * kWord, in);
        }
      } else {
        Raw4<T> b, c;
        b.load(sb, ok ? nst : 0, false);
        c.load(sc, ok ? nst : 0, false);
        *reinterpret_cast<Raw4<T>*>(dst) = b;
        *reinterpret_cast<Raw4<T>*>(dst_c) = c;
      }
    }
    if (rows > kTile) {
      bs += kTile * p.b_stride;
      cs += kTile * p.c_stride;
    }
  };

  T* yp = static_cast<T*>(p.y) + (k.t0 + 4 * quad) * p.dim + c;
  f32x2 sum = pack2(0.f, 0.f);  // of this thread's steps (kSummary)
  Raw2<T> x_next[4], x_now[4], x_last[4];  // x of tiles i + 1, i, i - 1 (the skip)
  const bool gate = kFinish && p.z;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (kStage) {
      copy(0, p.x_stride, i);
      copy(1, p.dt_stride, i);
      if (i < kBcAhead - 1) copy_bc(i);
    }
    if (i == 0 && gate) copy(2, p.z_stride, 0);
    cp_async_commit();
    if (kStage) {
      copy_late(0, i);
      copy_late(1, i);
    }
    if (i == 0 && gate) copy_late(2, 0);
  }
  cp_async_wait<2>();
  if (kStage) named_sync(1, C::kHelpers);
  for (int i = -1; i <= nt; ++i) {
    if (kStage) {
      copy(0, p.x_stride, i + kRing);
      copy(1, p.dt_stride, i + kRing);
      copy_bc(i + kBcAhead);
    }
    if (gate) copy(2, p.z_stride, i + 2);
    cp_async_commit();
    if (kStage && i + 1 < nt) {
      const float4* rx = smem + C::kX + ((i + 1) & (C::kRingX - 1)) * C::kRawTile;
      const float4* rd = smem + C::kDt + ((i + 1) & (kRing - 1)) * C::kRawTile;
      float4* du = smem + C::kDu + ((i + 1) & 1) * C::kDuTile + pair * (kTile + 1) + 4 * quad;
      const int rows = len - (i + 1) * kTile - 4 * quad;
      // (branches around the four tokens, not within: their chains run side by side)
      f32x2 d[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        Raw2<T> d2;
        x_next[u].load(rx + (4 * quad + u) * C::kPitch, pair);
        d2.load(rd + (4 * quad + u) * C::kPitch, pair);
        d[u] = add2(d2.get(), bias);
      }
      if (p.softplus) {
#pragma unroll
        for (int u = 0; u < 4; ++u) d[u] = softplus2(d[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (kSummary) sum = add2(sum, u < rows ? d[u] : pack2(0.f, 0.f));
        float d0, d1, u0, u1;
        unpack2(d[u], d0, d1);
        unpack2(mul2(d[u], x_next[u].get()), u0, u1);
        du[u] = make_float4(d0, u0, d1, u1);
      }
      if (C::kWiden) {
        const float4* raw = smem + C::kBc + ((i + 1) & (kRing - 1)) * C::kBcTile;
        float4* wide = smem + C::kWide + ((i + 1) & 1) * C::kWideTile;
#pragma unroll
        for (int j = 0; j < C::kPerHelper; ++j) {
          const int id = tid + j * C::kHelpers;
          if (C::kFours % C::kHelpers == 0 || id < C::kFours) {
            const float4 v = raw[id];
            wide[2 * id] = wide4(v.x, v.y);
            if (!kSummary) wide[2 * id + 1] = wide4(v.z, v.w);
          }
        }
      }
    }
    if (kFinish && i >= 1 && left > 0) {
      const float4* part = smem + C::kPart + ((i - 1) & 1) * C::kPartTile + pair * C::kPartPair +
                           2 * quad;
      f32x2 v[4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        ulonglong2 w;  // tokens 2 q and 2 q + 1 of the quad: one channel, and the other
#pragma unroll
        for (int l = 0; l < C::kParts; ++l) {
          const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(part + l * C::kPartRow + q);
          w.x = l ? add2(w.x, o.x) : o.x;
          w.y = l ? add2(w.y, o.y) : o.y;
        }
        float a0, a1, b0, b1;
        unpack2(w.x, a0, a1);
        unpack2(w.y, b0, b1);
        v[2 * q] = pack2(a0, b0);
        v[2 * q + 1] = pack2(a1, b1);
      }
      const float4* rz = smem + C::kZ + ((i - 1) & (kRing - 1)) * C::kRawTile;
      const int rows = len - (i - 1) * kTile - 4 * quad;
      if (p.D) {
        if (!kStage) {
          const float4* rx = smem + C::kX + ((i - 1) & (C::kRingX - 1)) * C::kRawTile;
#pragma unroll
          for (int u = 0; u < 4; ++u) x_last[u].load(rx + (4 * quad + u) * C::kPitch, pair);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = fma2(skip, x_last[u].get(), v[u]);
      }
      if (p.z) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          Raw2<T> z2;
          z2.load(rz + (4 * quad + u) * C::kPitch, pair);
          v[u] = mul2(v[u], silu2(z2.get()));
        }
      }
      if (rows >= 4 && p.vec2) {
#pragma unroll
        for (int u = 0; u < 4; ++u) store2(yp + u * (long long)p.dim, v[u], 2, true);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (u < rows) store2(yp + u * (long long)p.dim, v[u], left, p.vec2);
      }
      yp += kTile * (long long)p.dim;
    }
    if (kStage && kFinish) {
#pragma unroll
      for (int u = 0; u < 4; ++u) x_last[u] = x_now[u], x_now[u] = x_next[u];
    }
    if (kStage) {
      copy_late(0, i + kRing);
      copy_late(1, i + kRing);
    }
    if (gate) copy_late(2, i + 2);
    cp_async_wait<2>();
    named_sync(2, C::kThreads);
  }

  if (kSummary) {  // the sum of the chunk's steps: kTile / 4 threads hold parts of each pair's
    f32x2* parts = reinterpret_cast<f32x2*>(smem + C::kPart);
    parts[tid] = sum;
    named_sync(1, C::kHelpers);
    const int off = p.whole * kCh;
    if (tid < kCh && k.ch0 + tid < p.dim) {
      float a = 0.f;
#pragma unroll
      for (int q = 0; q < kTile / 4; ++q) a += reinterpret_cast<const float*>(parts)[q * kCh + tid];
      p.ws_sum[(first_slot(p, k.n) + k.c) * (p.dim - off) + k.ch0 + tid - off] = a;
    }
  }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kBlocks) s6_kernel(const S6Params p, int tiles) {
  extern __shared__ float4 smem[];
  Task k;
  if (!find_task(p, C::kSummary, tiles, &k)) {
    if (!C::kSummary && p.chunk) griddep_wait();
    return;
  }
  if (C::kSummary) griddep_launch_dependents();
  // nothing starts from a sequence's last chunk: of that only h0 is kept, where it has to be
  const bool idle = C::kSummary && k.last;
  const int nt = idle ? 0 : (int)((k.t1 - k.t0 + C::kTile - 1) / C::kTile);
  if (idle && !(k.c == 0 && p.ws_h0)) return;
  int tid = threadIdx.x;
  if (C::kPlace) {
    // The computing warps go to schedulers 0 and 1, or 2 and 3 for every other CTA (by the
    // hardware's slots), so that two CTAs of an SM do not have them on the same ones: 59 cycles
    // a token of 32 channels otherwise, 38 with it (the recurrence alone, two CTAs).  Should the
    // slots not be four schedulers in turn, warps keep their order.
    __shared__ unsigned s_base, s_seen;
    unsigned slot;
    asm volatile("mov.u32 %0, %%warpid;" : "=r"(slot));
    if (tid == 0) s_base = slot, s_seen = 0u;
    __syncthreads();
    const int w = (int)((slot & 3) ^ (s_base / 4 & 1 ? 2 : 0));
    if (tid % 32 == 0) atomicOr(&s_seen, 1u << w);
    __syncthreads();
    if (s_seen == 15u) tid = w * 32 + tid % 32;
  }
  if (tid < C::kCompute) {
    s6_compute<C>(p, k, smem, nt, tid);
  } else if constexpr (C::kApart) {
    if (tid < C::kCompute + C::kHelpers) s6_help<C, true, false>(p, k, smem, nt, tid - C::kCompute);
    else s6_help<C, false, true>(p, k, smem, nt, tid - C::kCompute - C::kHelpers);
  } else {
    s6_help<C, true, !C::kSummary>(p, k, smem, nt, tid - C::kCompute);
  }
  // every block of the scan outlives the summaries, so what follows in the stream may reuse
  // the workspace
  if (!C::kSummary && p.chunk) griddep_wait();
}

template <class C>
cudaError_t launch_k(const S6Params& p, cudaStream_t stream) {
  const auto kernel = s6_kernel<C>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kAsked);
  if (e != cudaSuccess) return e;
  const int tiles = (p.dim + kCh - 1) / kCh;
  const long long whole = C::kSummary ? 0 : (long long)p.N * p.whole;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = !C::kSummary && p.chunk ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(whole + (long long)(tiles - p.whole) * p.slots));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kAsked;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, tiles);
}

template <typename T, int LPC, Fill kFill>
cudaError_t launch_l(const S6Params& p, cudaStream_t stream) {
  if (p.chunk) {  // (summaries have no sums over the lanes)
    constexpr Fill kStates = kFill == Fill::kPart ? kFill : Fill::kAll;
    const cudaError_t e = launch_k<Cfg<T, LPC, 2, 16, kStates, true>>(p, stream);
    if (e != cudaSuccess) return e;
  }
  // whole sequences and first chunks need no summary, so the scan may start beside them
  // One channel a lane where every CTA has an SM for itself (1024 tokens of 4864 channels, us,
  // against two channels a lane; bf16 with Ns 4, 8, 32, 64: 37 : 56, 35 : 47, 57 : 82, 98 : 138;
  // fp32: 29 : 47, 31 : 47, but 95 : 74, 182 : 127, where B and C are twice the bytes).
  if constexpr (kFill != Fill::kPart && (sizeof(T) == 2 || LPC <= 4)) {
    if (p.lone) return launch_k<Cfg<T, LPC, 1, 32, kFill, false>>(p, stream);
  }
  return launch_k<Cfg<T, LPC, 2, 16, kFill, false>>(p, stream);
}

template <typename T>
cudaError_t launch_scan(const S6Params& p, cudaStream_t stream) {
  constexpr Fill kAll = Fill::kAll, kSome = Fill::kSome, kPart = Fill::kPart;
  if (p.Ns % 4)
    return p.Ns < 16   ? launch_l<T, 4, kPart>(p, stream)
           : p.Ns < 32 ? launch_l<T, 8, kPart>(p, stream)
                       : launch_l<T, 16, kPart>(p, stream);
  switch (p.Ns) {
    case 4: return launch_l<T, 1, kAll>(p, stream);
    case 8: return launch_l<T, 2, kAll>(p, stream);
    case 16: return launch_l<T, 4, kAll>(p, stream);
    case 32: return launch_l<T, 8, kAll>(p, stream);
    case 64: return launch_l<T, 16, kAll>(p, stream);
  }
  return p.Ns < 16   ? launch_l<T, 4, kSome>(p, stream)
         : p.Ns < 32 ? launch_l<T, 8, kSome>(p, stream)
                     : launch_l<T, 16, kSome>(p, stream);
}

}  // namespace
}  // namespace gdn
