// s6_scan.cu - the selective state space scan with a diagonal A (S6, the Mamba-1 member of
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
// Layout.  A lane keeps four states of two neighbouring channels in registers and LPC =
// Ns / 4 lanes share the pair; a CTA has 32 channels and walks its tokens in tiles of 32.  The
// recurrence of one or two warps cannot hide a load or a quotient, so the warps are of two
// kinds: the 16 LPC computing threads do nothing but the recurrence, out of shared memory, and
// 128 helper threads beside them prepare the next tile and finish the last one.  Per tile the
// helpers form (D_t, D_t x_t) once per token and channel, and B and C as fp32; add the lanes'
// partial sums over n, the skip and the gate into y; and keep the copies of the coming tiles in
// flight (cp.async, a ring of four).  One barrier a tile.
//
// Splitting over time.  A CTA per 32 channels leaves SMs idle when there are few of them.
// Channels beyond the whole-sequence ones are split over time: a first launch computes the
// state that each chunk of tokens ends in from a zero state, and the sum of its steps (the
// decay over the chunk is exp(A sum D_t)); the scan then starts each chunk from the chunks
// before it.  That computes the exponentials twice; s6_split says where it pays.
#include "gdn_common.cuh"
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {
namespace {

constexpr int kTile = 32;  // tokens per tile
constexpr int kCh = 32;    // channels per CTA
constexpr int kSms = 152;
constexpr int kRing = 4;   // tiles of raw inputs in shared memory
constexpr int kPairs = kCh / 2;
constexpr int kQuads = kTile / 4;
constexpr int kHelpers = kPairs * kQuads;  // a helper thread has 2 channels x 4 tokens of a tile

// Shared memory, in pieces of 16 bytes, and the warps, for T inputs and LPC lanes per channel
// pair.
template <typename T, int LPC, bool kSummary>
struct Cfg {
  static constexpr int kCompute = kPairs * LPC < 32 ? 32 : kPairs * LPC;
  // Two computing warps (LPC = 4) sit on two of the four schedulers; the helpers go to the
  // other two, where there are four of them with two warps in between that end at once.
  static constexpr bool kPlace = LPC == 4;
  static constexpr int kGap = kPlace && kHelpers == 128 ? 64 : 0;
  static constexpr int kThreads = kCompute + kHelpers + kGap;
  // a raw row: 32 channels and 16 bytes more, so that rows 4 apart meet other banks
  static constexpr int kRowPieces = kCh * (int)sizeof(T) / 16, kPitch = kRowPieces + 1;
  static constexpr int kRawTile = kTile * kPitch;
  static constexpr int kCopies = kTile * kRowPieces / kHelpers;  // per helper, tensor and tile
  static constexpr int kDuTile = kPairs * (kTile + 1);  // (D0, D1, D0 x0, D1 x1) a pair and token
  // four states' B and C of a token: one piece in bf16, two in fp32; bf16 ones are widened
  // into two further tiles, fp32 ones are used where they arrive
  static constexpr bool kWiden = sizeof(T) == 2;
  static constexpr int kBcPieces = (int)sizeof(T) / 2, kBcTile = kTile * LPC * kBcPieces;
  static constexpr int kWideTile = kTile * LPC * 2;
  // partial sums of y: kParts rows a pair (8 or 16 lanes add up to 4 by shuffles first) of
  // kTile / 2 pieces, each two tokens of both channels.  Rows of kTile / 2 + 2 pieces, moved
  // on by one every pair: with 4 lanes a pair the writes (8 lanes: 2 pairs x 4 rows) and the
  // reads (8 pairs) both spread over the banks.
  static constexpr int kParts = LPC < 4 ? LPC : 4, kLanes = LPC / kParts;
  static constexpr int kPartPair = kParts * (kTile / 2 + 2) + 1;
  static constexpr int kPartTile = kSummary ? 0 : kPairs * kPartPair;
  static constexpr int kRaw = 0, kTensors = kSummary ? 2 : 3;
  static constexpr int kDu = kRaw + kRing * kTensors * kRawTile;
  static constexpr int kBc = kDu + 2 * kDuTile;
  static constexpr int kWide = kBc + kRing * kBcTile;
  static constexpr int kPart = kWide + (kWiden ? 2 * kWideTile : 0);
  static constexpr int kPieces = kPart + (kSummary ? kQuads * kCh / 4 : 2 * kPartTile);
  static constexpr int kBytes = kPieces * 16;
  static constexpr int kBlocks = kBytes <= 113 * 1024 && kThreads <= 512 ? 2 : 1;  // per SM
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
// One piece (16 bytes) of a raw row, element by element: the first n elements exist.
__device__ __forceinline__ float4 load_piece(const __nv_bfloat16* p, int n) {
  Raw8<__nv_bfloat16> r;
  r.load_n(p, n);
  return make_float4(__uint_as_float(r.v.x), __uint_as_float(r.v.y), __uint_as_float(r.v.z),
                     __uint_as_float(r.v.w));
}
__device__ __forceinline__ float4 load_piece(const float* p, int n) {
  return make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f,
                     n > 3 ? p[3] : 0.f);
}

// Four states' B or C of one token, as stored.
template <typename T>
struct Raw4;
template <>
struct Raw4<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void zero() { v = make_uint2(0u, 0u); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int n, bool vec) {
    if (vec) {
      v = *reinterpret_cast<const uint2*>(p);
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
      v.x = (n > 0 ? q[0] : 0u) | (n > 1 ? (uint32_t)q[1] << 16 : 0u);
      v.y = (n > 2 ? q[2] : 0u) | (n > 3 ? (uint32_t)q[3] << 16 : 0u);
    }
  }
  __device__ __forceinline__ float4 get() const {
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  }
};
template <>
struct Raw4<float> {
  float4 v;
  __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p, int n, bool vec) {
    if (vec) v = *reinterpret_cast<const float4*>(p);
    else v = make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
  }
  __device__ __forceinline__ float4 get() const { return v; }
};
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
// Four states of the recurrence (n of them exist): rows of Ns floats, 16-byte aligned bases.
__device__ __forceinline__ float4 load_h(const float* p, int n, int Ns) {
  if ((Ns & 3) == 0) return n > 0 ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
  return make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f,
                     n > 3 ? p[3] : 0.f);
}
__device__ __forceinline__ void store_h(float* p, float4 v, int n, int Ns) {
  if ((Ns & 3) == 0) {
    if (n > 0) *reinterpret_cast<float4*>(p) = v;
    return;
  }
  if (n > 0) p[0] = v.x;
  if (n > 1) p[1] = v.y;
  if (n > 2) p[2] = v.z;
  if (n > 3) p[3] = v.w;
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
      int lo = 0, hi = p.N - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (border(p, mid) / p.chunk + mid <= slot) lo = mid; else hi = mid - 1;
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

// The computing threads' part: the recurrence over the tiles.  A lane has four states of two
// neighbouring channels: what limits it is the bandwidth of shared memory (4 bytes a lane and
// clock, whatever lanes share), and the second channel takes B and C from registers.
template <typename T, int LPC, bool kPad, bool kSummary>
__device__ __forceinline__ void s6_compute(const S6Params& p, const Task& k, float4* smem, int nt,
                                           int tid) {
  using C = Cfg<T, LPC, kSummary>;
  const int pair = tid / LPC, ln = tid % LPC;  // LPC = 1: only 16 of the 32 lanes have a pair
  const int ch = k.ch0 + 2 * pair, n0 = ln * 4;
  const int chs = pair < kPairs ? max(0, min(2, p.dim - ch)) : 0;  // channels that exist
  const int nst = chs > 0 ? max(0, min(4, p.Ns - n0)) : 0;         // and states of them
  const long long hsize = (long long)p.dim * p.Ns;
  // the workspace holds the split channels only
  const int off = p.whole * kCh, wdim = p.dim - off;
  const long long wsize = (long long)wdim * p.Ns;

  float a[2][4];
  f32x2 h[2][2];
  const bool kept = k.split && p.ws_h0;  // hT == h0: the scan reads the copy
  if (!kSummary && (k.c > 0 || kept)) griddep_wait();
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int n = j < chs ? nst : 0;
    const long long hrow = (long long)(ch + j) * p.Ns + n0, wrow = hrow - (long long)off * p.Ns;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n > 0) v = load_h(p.A + hrow, n, p.Ns);
    a[j][0] = v.x * kLog2e, a[j][1] = v.y * kLog2e, a[j][2] = v.z * kLog2e, a[j][3] = v.w * kLog2e;
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
        const float s = p.ws_sum[(s0 + i) * wdim + ch + j - off];
        h[j][0] = fma2(pack2(ex2(a[j][0] * s), ex2(a[j][1] * s)), h[j][0], pack2(v.x, v.y));
        h[j][1] = fma2(pack2(ex2(a[j][2] * s), ex2(a[j][3] * s)), h[j][1], pack2(v.z, v.w));
      }
    }
  }

  struct In {            // a step's operands as they lie in shared memory
    float4 du, b, c;
  };
  struct Ready {         // what the recurrence of a step needs: decays, inputs, C
    f32x2 a[2][2], u[2][2], c01, c23;
  };
  const int lp = pair < kPairs ? pair : 0;
  for (int i = -1; i <= nt; ++i) {
    if (i >= 0 && i < nt) {
      const float4* du = smem + C::kDu + (i & 1) * C::kDuTile + lp * (kTile + 1);
      const float4* bc = (C::kWiden ? smem + C::kWide + (i & 1) * C::kWideTile
                                    : smem + C::kBc + (i & (kRing - 1)) * C::kBcTile) + 2 * ln;
      float4* part = smem + C::kPart + (i & 1) * C::kPartTile + lp * C::kPartPair +
                     ln / C::kLanes * (kTile / 2 + 2);
      auto put = [&](int t, float4 v) {  // both channels' sums of tokens t and t + 1
#pragma unroll
        for (int o = 1; o < C::kLanes; o *= 2) {
          v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
          v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
          v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
          v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
        }
        // (no branch where every lane writes: it would keep the steps apart)
        if ((C::kLanes == 1 || ln % C::kLanes == 0) && (kPairs * LPC >= 32 || pair < kPairs))
          part[t / 2] = v;
      };
      auto fetch = [&](int t) {
        In r;
        r.du = du[t];
        r.b = bc[t * LPC * 2];
        if (!kSummary) r.c = bc[t * LPC * 2 + 1];
        return r;
      };
      auto ready = [&](const In& in) {
        Ready r;
        const float d[2] = {in.du.x, in.du.y}, u[2] = {in.du.z, in.du.w};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          r.a[j][0] = pack2(ex2(a[j][0] * d[j]), ex2(a[j][1] * d[j]));
          r.a[j][1] = pack2(ex2(a[j][2] * d[j]), ex2(a[j][3] * d[j]));
          r.u[j][0] = pack2(in.b.x * u[j], in.b.y * u[j]);
          r.u[j][1] = pack2(in.b.z * u[j], in.b.w * u[j]);
        }
        if (!kSummary) r.c01 = pack2(in.c.x, in.c.y), r.c23 = pack2(in.c.z, in.c.w);
        return r;
      };
      auto step = [&](const Ready& r, int j) -> float {
        h[j][0] = fma2(r.a[j][0], h[j][0], r.u[j][0]);
        h[j][1] = fma2(r.a[j][1], h[j][1], r.u[j][1]);
        if (kPad) {  // states that do not exist stay zero whatever the step
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
        float4 out[2];  // sums wait two steps, so that their store waits for nothing
#pragma unroll
        for (int t = 0; t < kTile; ++t) {
          In later;
          Ready next;
          if (t + 2 < kTile) later = fetch(t + 2);
          if (!kSummary && t >= 2 && t % 2 == 0) put(t - 2, out[t / 2 % 2 ^ 1]);
          if (t + 1 < kTile) next = ready(in);
          const float y0 = step(now, 0), y1 = step(now, 1);
          float4& o = out[t / 2 % 2];
          if (t % 2 == 0) o.x = y0, o.y = y1; else o.z = y0, o.w = y1;
          if (t + 1 < kTile) now = next;
          if (t + 2 < kTile) in = later;
        }
        if (!kSummary) put(kTile - 2, out[(kTile / 2 - 1) % 2]);
      } else {
        float4 out = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int t = 0; t < (int)left; ++t) {
          const Ready r = ready(fetch(t));
          const float y0 = step(r, 0), y1 = step(r, 1);
          if (t % 2 == 0) out.x = y0, out.y = y1; else out.z = y0, out.w = y1;
          if (!kSummary && (t % 2 == 1 || t + 1 == (int)left)) put(t, out);
        }
      }
    }
    named_sync(2, C::kCompute + kHelpers);
  }

#pragma unroll
  for (int j = 0; j < 2; ++j) {
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
// start the copies of tiles to come (x and dt of tile i + 4, B and C of i + 3, z of i + 2: the
// ring's places are free then), stage tile i + 1 and write y of tile i - 1.
template <typename T, int LPC, bool kSummary>
__device__ __forceinline__ void s6_help(const S6Params& p, const Task& k, float4* smem, int nt,
                                        int tid) {
  using C = Cfg<T, LPC, kSummary>;
  const int pair = tid % kPairs, quad = tid / kPairs;
  const int c = k.ch0 + 2 * pair, left = p.dim - c;
  const f32x2 bias = pack2(p.dt_bias && left > 0 ? p.dt_bias[c] : 0.f,
                           p.dt_bias && left > 1 ? p.dt_bias[c + 1] : 0.f);
  const f32x2 skip = pack2(!kSummary && p.D && left > 0 ? p.D[c] : 0.f,
                           !kSummary && p.D && left > 1 ? p.D[c + 1] : 0.f);
  const bool vec = p.vec;

  // one tile of x (0), dt (1) or z (2) into the ring; rows and channels that do not exist: 0
  constexpr int kRowStep = kHelpers / C::kRowPieces;  // rows between a thread's copies
  const int row0 = tid / C::kRowPieces, piece = tid % C::kRowPieces;
  const int ch = k.ch0 + piece * (16 / (int)sizeof(T));
  const int some = max(0, p.dim - ch);                // channels of the piece that exist
  const int len = (int)(k.t1 - k.t0);
  const T* xs = static_cast<const T*>(p.x) + (some ? (k.t0 + row0) * p.x_stride + ch : 0);
  const T* ds = static_cast<const T*>(p.dt) + (some ? (k.t0 + row0) * p.dt_stride + ch : 0);
  const T* zs = static_cast<const T*>(p.z) + (some ? (k.t0 + row0) * p.z_stride + ch : 0);
  auto copy = [&](int tensor, const T*& src, long long stride, int i) {
    float4* dst = smem + C::kRaw + (tensor * kRing + (i & (kRing - 1))) * C::kRawTile +
                  row0 * C::kPitch + piece;
    const int rows = len - i * kTile - row0;  // from this thread's first one on
#pragma unroll
    for (int j = 0; j < C::kCopies; ++j) {
      const bool ok = j * kRowStep < rows && some;
      const T* s = ok ? src + j * kRowStep * stride : src;
      if (vec) cp_async16(dst + j * kRowStep * C::kPitch, s, ok);
      else dst[j * kRowStep * C::kPitch] = load_piece(s, ok ? some : 0);
    }
    if (rows > kTile) src += kTile * stride;  // stays inside the tensor
  };
  auto copy_in = [&](int i) {
    if (i < nt) {
      copy(0, xs, p.x_stride, i);
      copy(1, ds, p.dt_stride, i);
    }
  };
  auto copy_gate = [&](int i) {
    if (!kSummary && p.z && i < nt) copy(2, zs, p.z_stride, i);
  };
  // B and C of a tile, four states of a token at a time, into their ring
  constexpr int kFours = kTile * LPC, kPer = (kFours + kHelpers - 1) / kHelpers;
  static_assert(kPer == 1 || kHelpers % LPC == 0, "every four of a thread has the same states");
  const int brow = tid / LPC, n0 = tid % LPC * 4;
  const int nst = max(0, p.Ns - n0);
  const T* bs = static_cast<const T*>(p.B) + (nst ? (k.t0 + brow) * p.b_stride + n0 : 0);
  const T* cs = static_cast<const T*>(p.C) + (nst ? (k.t0 + brow) * p.c_stride + n0 : 0);
  auto copy_bc = [&](int i) {
    if (i >= nt) return;
    const int rows = len - i * kTile - brow;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int id = tid + j * kHelpers, r = j * (kHelpers / LPC);
      if (id >= kFours) break;
      float4* dst = smem + C::kBc + (i & (kRing - 1)) * C::kBcTile + id * C::kBcPieces;
      T* dst_c = reinterpret_cast<T*>(dst) + 4;
      const bool ok = r < rows && nst;
      const T *sb = ok ? bs + r * p.b_stride : bs, *sc = ok ? cs + r * p.c_stride : cs;
      if (p.vec_bc && sizeof(T) == 2) {
        cp_async8(dst, sb, ok);
        if (!kSummary) cp_async8(dst_c, sc, ok);
      } else if (p.vec_bc) {
        cp_async16(dst, sb, ok);
        if (!kSummary) cp_async16(dst_c, sc, ok);
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
  copy_in(0);
  copy_bc(0);
  copy_gate(0);
  cp_async_commit();
  copy_in(1);
  copy_bc(1);
  cp_async_commit();
  copy_in(2);
  cp_async_commit();
  cp_async_wait<2>();
  named_sync(1, kHelpers);
  for (int i = -1; i <= nt; ++i) {
    copy_in(i + kRing);
    copy_bc(i + 3);
    copy_gate(i + 2);
    cp_async_commit();
    if (i + 1 < nt) {  // stage
      const int s = (i + 1) & (kRing - 1);
      const float4* rx = smem + C::kRaw + s * C::kRawTile;
      const float4* rd = rx + kRing * C::kRawTile;
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
        du[u] = make_float4(d0, d1, u0, u1);
      }
      if (C::kWiden) {
        const float4* raw = smem + C::kBc + s * C::kBcTile;
        float4* wide = smem + C::kWide + ((i + 1) & 1) * C::kWideTile;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int id = tid + j * kHelpers;
          if (kFours % kHelpers == 0 || id < kFours) {
            const float4 v = raw[id];
            wide[2 * id] = wide4(v.x, v.y);
            if (!kSummary) wide[2 * id + 1] = wide4(v.z, v.w);
          }
        }
      }
    }
    if (!kSummary && i >= 1 && left > 0) {  // y of tile i - 1
      const float4* part = smem + C::kPart + ((i - 1) & 1) * C::kPartTile + pair * C::kPartPair +
                           2 * quad;
      ulonglong2 w[2];  // both channels at tokens 0, 1 and 2, 3 of the quad
#pragma unroll
      for (int l = 0; l < C::kParts; ++l) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const ulonglong2 v =
              *reinterpret_cast<const ulonglong2*>(part + l * (kTile / 2 + 2) + q);
          w[q].x = l ? add2(w[q].x, v.x) : v.x;
          w[q].y = l ? add2(w[q].y, v.y) : v.y;
        }
      }
      const float4* rz = smem + C::kRaw + (2 * kRing + ((i - 1) & (kRing - 1))) * C::kRawTile;
      const int rows = len - (i - 1) * kTile - 4 * quad;
      f32x2 v[4] = {w[0].x, w[0].y, w[1].x, w[1].y};
      if (p.D) {
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = fma2(skip, x_last[u].get(), v[u]);
      }
      if (p.z) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          Raw2<T> z2;
          z2.load(rz + (4 * quad + u) * C::kPitch, pair);
          const f32x2 z = z2.get();
          float e0, e1;
          unpack2(mul2(z, dup2(-kLog2e)), e0, e1);
          unpack2(add2(pack2(ex2(e0), ex2(e1)), dup2(1.f)), e0, e1);
          v[u] = mul2(v[u], mul2(z, pack2(rcp(e0), rcp(e1))));
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
#pragma unroll
    for (int u = 0; u < 4; ++u) x_last[u] = x_now[u], x_now[u] = x_next[u];
    cp_async_wait<2>();
    named_sync(2, C::kCompute + kHelpers);
  }

  if (kSummary) {  // the sum of the chunk's steps: kQuads threads hold parts of each pair's
    f32x2* parts = reinterpret_cast<f32x2*>(smem + C::kPart);
    parts[tid] = sum;
    named_sync(1, kHelpers);
    const int off = p.whole * kCh;
    if (tid < kCh && k.ch0 + tid < p.dim) {
      float a = 0.f;
#pragma unroll
      for (int q = 0; q < kQuads; ++q) a += reinterpret_cast<const float*>(parts)[q * kCh + tid];
      p.ws_sum[(first_slot(p, k.n) + k.c) * (p.dim - off) + k.ch0 + tid - off] = a;
    }
  }
}

template <typename T, int LPC, bool kPad, bool kSummary>
__global__ void __launch_bounds__(Cfg<T, LPC, kSummary>::kThreads,
                                  Cfg<T, LPC, kSummary>::kBlocks)
    s6_kernel(const S6Params p, int tiles) {
  using C = Cfg<T, LPC, kSummary>;
  extern __shared__ float4 smem[];
  Task k;
  if (!find_task(p, kSummary, tiles, &k)) {
    if (!kSummary && p.chunk) griddep_wait();
    return;
  }
  if (kSummary) griddep_launch_dependents();
  // nothing starts from a sequence's last chunk: of that only h0 is kept, where it has to be
  const bool idle = kSummary && k.last;
  const int nt = idle ? 0 : (int)((k.t1 - k.t0 + kTile - 1) / kTile);
  if (idle && !(k.c == 0 && p.ws_h0)) return;
  int tid = threadIdx.x;
  if (C::kPlace) {
    // The computing warps go to schedulers 0 and 1, or 2 and 3 for every other CTA (by the
    // hardware's slots), so that two CTAs of an SM do not have them on the same ones.  Should
    // the slots not be four schedulers in turn, warps keep their order.
    __shared__ unsigned s_base, s_seen;
    unsigned slot;
    asm volatile("mov.u32 %0, %%warpid;" : "=r"(slot));
    if (tid == 0) s_base = slot, s_seen = 0u;
    __syncthreads();
    const int w = (int)((slot & 3) ^ (s_base / (C::kThreads / 32) & 1 ? 2 : 0)) + (tid >> 7) * 4;
    if (tid % 32 == 0) atomicOr(&s_seen, 1u << w);
    __syncthreads();
    if (s_seen == (1u << C::kThreads / 32) - 1) tid = w * 32 + tid % 32;
    if (C::kGap && tid >= 128) tid -= tid < 192 ? 256 : 64;
  }
  if (tid >= C::kCompute) s6_help<T, LPC, kSummary>(p, k, smem, nt, tid - C::kCompute);
  else if (tid >= 0) s6_compute<T, LPC, kPad, kSummary>(p, k, smem, nt, tid);
  // every block of the scan outlives the summaries, so what follows in the stream may reuse
  // the workspace
  if (!kSummary && p.chunk) griddep_wait();
}

// ---- one token -------------------------------------------------------------------------
// A lane takes four states of one (sequence, channel): reads them, A, and the token's
// inputs, writes them back; the LPC lanes of a channel add their parts of y by shuffles.
// The states are read and written once, 128 bytes a channel at Ns = 16: HBM bandwidth
// bounds it, launch latency for few sequences.
template <typename T, int LPC>
__global__ void __launch_bounds__(256) s6_step_kernel(const S6Params p, int per_row) {
  const int bx = blockIdx.x % per_row;
  const long long n = blockIdx.x / per_row;
  const int id = bx * 256 + threadIdx.x;
  const bool some = id / LPC < p.dim;  // lanes behind the last channel only join the shuffles
  const int ch = some ? id / LPC : p.dim - 1, n0 = id % LPC * 4;
  const int nst = some ? max(0, min(4, p.Ns - n0)) : 0;
  float* hp = p.hT + (n * p.dim + ch) * p.Ns + n0;
  const float4 h = load_h(hp, nst, p.Ns);
  const float4 a = load_h(p.A + (long long)ch * p.Ns + n0, nst, p.Ns);
  const float x = to_f32(static_cast<const T*>(p.x)[n * p.x_stride + ch]);
  float d = to_f32(static_cast<const T*>(p.dt)[n * p.dt_stride + ch]);
  float4 b = make_float4(0.f, 0.f, 0.f, 0.f), c = b;
  if (nst > 0) {
    Raw4<T> rb, rc;
    rb.load(static_cast<const T*>(p.B) + n * p.b_stride + n0, nst, p.vec_bc);
    rc.load(static_cast<const T*>(p.C) + n * p.c_stride + n0, nst, p.vec_bc);
    b = rb.get();
    c = rc.get();
  }
  const float z = p.z ? to_f32(static_cast<const T*>(p.z)[n * p.z_stride + ch]) : 0.f;
  if (p.dt_bias) d += p.dt_bias[ch];
  if (p.softplus) d = softplus(d);
  const float u = d * x, dl = d;
  float4 o;
  o.x = fmaf(ex2(dl * (a.x * kLog2e)), h.x, u * b.x);
  o.y = fmaf(ex2(dl * (a.y * kLog2e)), h.y, u * b.y);
  o.z = fmaf(ex2(dl * (a.z * kLog2e)), h.z, u * b.z);
  o.w = fmaf(ex2(dl * (a.w * kLog2e)), h.w, u * b.w);
  store_h(hp, o, nst, p.Ns);
  float y = 0.f;  // only of states that exist
  if (nst > 0) y = c.x * o.x;
  if (nst > 1) y = fmaf(c.y, o.y, y);
  if (nst > 2) y = fmaf(c.z, o.z, y);
  if (nst > 3) y = fmaf(c.w, o.w, y);
#pragma unroll
  for (int off = LPC / 2; off > 0; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
  if (some && id % LPC == 0) {
    if (p.D) y = fmaf(p.D[ch], x, y);
    if (p.z) y *= silu(z);
    from_f32(static_cast<T*>(p.y) + n * p.dim + ch, y);
  }
}

template <typename T, int LPC, bool kPad, bool kSummary>
cudaError_t launch_k(const S6Params& p, cudaStream_t stream) {
  using C = Cfg<T, LPC, kSummary>;
  const auto kernel = s6_kernel<T, LPC, kPad, kSummary>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e != cudaSuccess) return e;
  const int tiles = (p.dim + kCh - 1) / kCh;
  const long long whole = kSummary ? 0 : (long long)p.N * p.whole;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = !kSummary && p.chunk ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(whole + (long long)(tiles - p.whole) * p.slots));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, tiles);
}

template <typename T, int LPC, bool kPad>
cudaError_t launch_l(const S6Params& p, cudaStream_t stream) {
  if (p.chunk) {
    const cudaError_t e = launch_k<T, LPC, kPad, true>(p, stream);
    if (e != cudaSuccess) return e;
  }
  // whole sequences and first chunks need no summary, so the scan may start beside them
  return launch_k<T, LPC, kPad, false>(p, stream);
}

template <typename T, int LPC>
cudaError_t launch_p(const S6Params& p, cudaStream_t stream) {
  return p.Ns % 4 ? launch_l<T, LPC, true>(p, stream) : launch_l<T, LPC, false>(p, stream);
}

template <typename T>
cudaError_t launch_t(const S6Params& p, cudaStream_t stream) {
  if (p.Ns <= 4) return launch_p<T, 1>(p, stream);
  if (p.Ns <= 8) return launch_p<T, 2>(p, stream);
  if (p.Ns <= 16) return launch_p<T, 4>(p, stream);
  if (p.Ns <= 32) return launch_p<T, 8>(p, stream);
  return launch_p<T, 16>(p, stream);
}

template <typename T, int LPC>
cudaError_t launch_step_l(const S6Params& p, cudaStream_t stream) {
  const int per_row = (int)(((long long)p.dim * LPC + 255) / 256);
  s6_step_kernel<T, LPC><<<(unsigned)((long long)per_row * p.N), 256, 0, stream>>>(p, per_row);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_step_t(const S6Params& p, cudaStream_t stream) {
  if (p.Ns <= 4) return launch_step_l<T, 1>(p, stream);
  if (p.Ns <= 8) return launch_step_l<T, 2>(p, stream);
  if (p.Ns <= 16) return launch_step_l<T, 4>(p, stream);
  if (p.Ns <= 32) return launch_step_l<T, 8>(p, stream);
  return launch_step_l<T, 16>(p, stream);
}

}  // namespace

S6Split s6_split(int N, int T, int dim, int Ns, bool packed) {
  const int tiles = (dim + kCh - 1) / kCh;
  S6Split s{tiles, 0, 0, 0};
  if (N <= 0) return s;
  const long long ctas = (long long)N * tiles;
  const long long tokens = packed ? T : (long long)N * T;
  const long long per_seq = tokens / N;  // packed: their mean
  if (ctas >= kSms || per_seq < 512) return s;
  long long parts = (2 * kSms) / ctas;
  if (parts > 32) parts = 32;
  long long chunk = (per_seq + parts - 1) / parts;
  if (chunk < 256) chunk = 256;
  s.whole = 0;
  s.chunk = (int)((chunk + kTile - 1) / kTile * kTile);
  s.slots = packed ? (long long)T / s.chunk + N + 1
                   : (long long)N * (((long long)T + s.chunk - 1) / s.chunk);
  const size_t up = 63, wdim = dim - s.whole * kCh;
  s.sum_floats = ((size_t)s.slots * wdim + up) & ~up;
  s.h_floats = ((size_t)s.slots * wdim * Ns + up) & ~up;
  s.ws_bytes = (s.sum_floats + s.h_floats + (size_t)N * wdim * Ns) * sizeof(float);
  return s;
}

cudaError_t launch_s6(const S6Params& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_t<float>(p, stream) : launch_t<__nv_bfloat16>(p, stream);
}
cudaError_t launch_s6_step(const S6Params& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_step_t<float>(p, stream) : launch_step_t<__nv_bfloat16>(p, stream);
}

}  // namespace gdn
