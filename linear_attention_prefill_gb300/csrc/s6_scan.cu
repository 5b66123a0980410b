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
// The arithmetic is in packed fp32 pairs, which halves the instructions issued, not the
// pipe's time.
//
// Layout.  A lane keeps four states of one channel in registers and LPC = Ns / 4 lanes
// share a channel.  A CTA has 32 channels and walks its tokens in tiles of 32:
// the tile's (D_t, D_t x_t) are computed once per token and channel into shared memory,
// twice each, as the operand pairs of the packed instructions; B and C as fp32.  The lanes'
// partial sums over n go to shared memory and are added when the tile is written out.  The
// next tile's inputs are loaded into registers while the present one is computed.
//
// With few channels a sequence is split over time: a first launch computes the state that
// each chunk of tokens ends in from a zero state, and the sum of its steps (the decay over
// the whole chunk is exp(A sum D_t)); the scan proper then starts each chunk from the
// chunks before it.  That computes the exponentials twice, so it is done only where whole
// sequences would leave most of the GPU idle (s6_chunk).
#include "gdn_common.cuh"
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {
namespace {

constexpr int kTile = 32;  // tokens per tile
constexpr int kSms = 152;

constexpr int kCh = 32;    // channels per CTA
constexpr int kPairs = kCh / 2;
constexpr int kQuads = kTile / 4;
constexpr int kPatches = kPairs * kQuads;  // 2 channels x 4 tokens, the unit of staging

// LPC lanes per channel: 32 LPC threads, one thread per token and four states of B and C.
template <int LPC, bool kSummary>
struct Cfg {
  static constexpr int kThreads = kCh * LPC;
  static constexpr int kPerThread = (kPatches + kThreads - 1) / kThreads;
  // shared memory, in pieces of 16 bytes: (D, D, Dx, Dx) per channel and token, B, C, the
  // partial sums of y (the summary: of the steps)
  static constexpr int kDu = 0, kB = kCh * (kTile + 1), kC = kB + kTile * LPC,
                       kPart = kC + (kSummary ? 0 : kTile * LPC),
                       kPieces = kPart + (kSummary ? kQuads * kCh / 4
                                                   : kThreads * 9 + kThreads / 8);
  static constexpr int kBytes = kPieces * 16;
};

// Two neighbouring channels of one row as stored.
template <typename T>
struct Raw2;
template <>
struct Raw2<__nv_bfloat16> {
  uint32_t v = 0u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int n, bool vec) {
    if (vec) {
      v = *reinterpret_cast<const uint32_t*>(p);
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
      v = (n > 0 ? q[0] : 0u) | ((n > 1 ? (uint32_t)q[1] : 0u) << 16);
    }
  }
  __device__ __forceinline__ f32x2 get() const {
    return pack2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
};
template <>
struct Raw2<float> {
  float a = 0.f, b = 0.f;
  __device__ __forceinline__ void load(const float* p, int n, bool vec) {
    if (vec) {
      const float2 t = *reinterpret_cast<const float2*>(p);
      a = t.x, b = t.y;
    } else {
      a = n > 0 ? p[0] : 0.f;
      b = n > 1 ? p[1] : 0.f;
    }
  }
  __device__ __forceinline__ f32x2 get() const { return pack2(a, b); }
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

// Four states' B or C of one token.
template <typename T>
__device__ __forceinline__ float4 load_bc(const T* p, int n, bool vec);
template <>
__device__ __forceinline__ float4 load_bc(const __nv_bfloat16* p, int n, bool vec) {
  if (vec) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  }
  return make_float4(n > 0 ? to_f32(p[0]) : 0.f, n > 1 ? to_f32(p[1]) : 0.f,
                     n > 2 ? to_f32(p[2]) : 0.f, n > 3 ? to_f32(p[3]) : 0.f);
}
template <>
__device__ __forceinline__ float4 load_bc(const float* p, int n, bool vec) {
  if (vec) return *reinterpret_cast<const float4*>(p);
  return make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f,
                     n > 3 ? p[3] : 0.f);
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

// Four fp32 partial sums a lane and four tokens, in rows of 9 pieces of 16 bytes, moved on
// by one piece every 8 rows: the writes (8 lanes, one piece each) and the reads of the
// epilogue (every 2 LPC-th row) both spread over the banks.
__device__ __forceinline__ int part_at(int row, int piece) { return row * 9 + (row >> 3) + piece; }

// What a CTA works on: tokens [t0, t1) of sequence n (rows of the whole batch).
struct Task {
  int n, c;            // sequence, chunk of it
  long long t0, t1;
  bool last;           // the sequence ends here
};
// Slot -> task; false for a slot no chunk uses.  Borders are clamped to the batch.
__device__ __forceinline__ bool find_task(const S6Params& p, int slot, Task* k) {
  if (p.chunk == 0) {
    k->n = slot;
    k->c = 0;
  } else if (!p.cu) {
    const int per = (p.T + p.chunk - 1) / p.chunk;
    k->n = slot / per;
    k->c = slot % per;
  } else {  // chunk c of sequence n lives in slot floor(cu[n] / chunk) + n + c
    int lo = 0, hi = p.N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (min(max(p.cu[mid], 0), p.T) / p.chunk + mid <= slot) lo = mid; else hi = mid - 1;
    }
    k->n = lo;
    k->c = slot - (min(max(p.cu[lo], 0), p.T) / p.chunk + lo);
    if (k->c < 0) return false;
  }
  long long begin, end;
  if (p.cu) {
    begin = min(max(p.cu[k->n], 0), p.T);
    end = max((long long)min(max(p.cu[k->n + 1], 0), p.T), begin);
  } else {
    begin = (long long)k->n * p.T;
    end = begin + p.T;
  }
  k->t0 = begin;
  k->t1 = end;
  k->last = true;
  if (p.chunk) {
    k->t0 = begin + (long long)k->c * p.chunk;
    if (k->t0 >= end && k->c > 0) return false;
    if (k->t0 + p.chunk < end) {
      k->t1 = k->t0 + p.chunk;
      k->last = false;
    }
  }
  return true;
}
__device__ __forceinline__ long long first_slot(const S6Params& p, int n) {
  if (p.cu) return (long long)(min(max(p.cu[n], 0), p.T) / p.chunk) + n;
  return (long long)n * ((p.T + p.chunk - 1) / p.chunk);
}

template <typename T, int LPC, bool kPad, bool kSummary>
__global__ void __launch_bounds__(Cfg<LPC, kSummary>::kThreads)
    s6_kernel(const S6Params p, int tiles) {
  using C = Cfg<LPC, kSummary>;
  extern __shared__ float4 smem[];
  float4* const s_du = smem + C::kDu;      // [kCh][kTile + 1]
  float4* const s_b = smem + C::kB;        // [kTile][LPC]
  float4* const s_c = smem + C::kC;        // [kTile][LPC]
  float4* const s_part = smem + C::kPart;  // part_at(thread, token quad)

  const int tid = threadIdx.x;
  const int ch0 = blockIdx.x % tiles * kCh;
  Task k;
  if (!find_task(p, blockIdx.x / tiles, &k)) return;
  if (kSummary) griddep_launch_dependents();

  // this lane's channel and states
  const int lc = tid / LPC, ln = tid % LPC;
  const int ch = ch0 + lc, n0 = ln * 4;
  const int nst = ch < p.dim ? max(0, min(4, p.Ns - n0)) : 0;  // states that exist
  const long long hrow = (long long)ch * p.Ns + n0;            // within [dim, Ns]
  const long long hsize = (long long)p.dim * p.Ns;

  float4 a4 = make_float4(0.f, 0.f, 0.f, 0.f);
  if (nst > 0) a4 = load_h(p.A + hrow, nst, p.Ns);
  const f32x2 a01 = pack2(a4.x * kLog2e, a4.y * kLog2e), a23 = pack2(a4.z * kLog2e, a4.w * kLog2e);
  f32x2 h01 = pack2(0.f, 0.f), h23 = h01;

  if (kSummary) {
    if (k.c == 0 && nst > 0) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p.h0) v = load_h(p.h0 + k.n * hsize + hrow, nst, p.Ns);
      if (p.ws_h0) store_h(p.ws_h0 + k.n * hsize + hrow, v, nst, p.Ns);
      h01 = pack2(v.x, v.y);
      h23 = pack2(v.z, v.w);
    }
    if (k.last) return;  // nothing starts from a sequence's last chunk
  } else {
    const float* h0 = p.h0;
    if (p.chunk && (k.c > 0 || p.ws_h0)) {
      griddep_wait();
      if (p.ws_h0) h0 = p.ws_h0;
    }
    if (nst == 0) {
    } else if (k.c == 0) {
      if (h0) {
        const float4 v = load_h(h0 + k.n * hsize + hrow, nst, p.Ns);
        h01 = pack2(v.x, v.y);
        h23 = pack2(v.z, v.w);
      }
    } else {  // the state before this chunk, from the summaries of those before it
      const long long s0 = first_slot(p, k.n);
#pragma unroll 4
      for (int j = 0; j < k.c; ++j) {
        const float4 v = load_h(p.ws_h + (s0 + j) * hsize + hrow, nst, p.Ns);
        const f32x2 s = dup2(p.ws_sum[(s0 + j) * p.dim + ch]);
        float e0, e1, e2, e3;
        unpack2(mul2(a01, s), e0, e1);
        unpack2(mul2(a23, s), e2, e3);
        h01 = fma2(pack2(ex2(e0), ex2(e1)), h01, pack2(v.x, v.y));
        h23 = fma2(pack2(ex2(e2), ex2(e3)), h23, pack2(v.z, v.w));
      }
    }
  }

  const T* xp = static_cast<const T*>(p.x);
  const T* dp = static_cast<const T*>(p.dt);
  const T* zp = static_cast<const T*>(p.z);
  Raw2<T> xr[C::kPerThread][4], dr[C::kPerThread][4], zr[C::kPerThread][4];
  float4 br = make_float4(0.f, 0.f, 0.f, 0.f), cr = br;
  f32x2 sum = pack2(0.f, 0.f);  // of this thread's steps (kSummary)

  // staging: patch i of this thread is channels c, c + 1 and tokens 4 quad .. 4 quad + 3 of
  // a tile (kPairs divides the thread count, so the channels are the same for every patch)
  const int pair = tid % kPairs, c = ch0 + 2 * pair, left = p.dim - c;
  const f32x2 bias = pack2(p.dt_bias && left > 0 ? p.dt_bias[c] : 0.f,
                           p.dt_bias && left > 1 ? p.dt_bias[c + 1] : 0.f);
  const f32x2 skip = pack2(!kSummary && p.D && left > 0 ? p.D[c] : 0.f,
                           !kSummary && p.D && left > 1 ? p.D[c + 1] : 0.f);
  auto load_tile = [&](long long t) {
#pragma unroll
    for (int i = 0; i < C::kPerThread; ++i) {
      const int id = tid + i * C::kThreads;
      const int quad = id / kPairs;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const long long r = t + 4 * quad + u;
        const bool ok = id < kPatches && r < k.t1 && left > 0;
        const bool vec = p.vec2;
        xr[i][u] = Raw2<T>();
        dr[i][u] = Raw2<T>();
        if (ok) {
          xr[i][u].load(xp + r * p.x_stride + c, left, vec);
          dr[i][u].load(dp + r * p.dt_stride + c, left, vec);
        }
      }
    }
    const long long r = t + tid / LPC;  // kTile rows of LPC threads
    br = cr = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < k.t1 && n0 < p.Ns) {
      br = load_bc(static_cast<const T*>(p.B) + r * p.b_stride + n0, p.Ns - n0, p.vec_bc);
      if (!kSummary)
        cr = load_bc(static_cast<const T*>(p.C) + r * p.c_stride + n0, p.Ns - n0, p.vec_bc);
    }
  };
  auto load_gate = [&](long long t) {
#pragma unroll
    for (int i = 0; i < C::kPerThread; ++i) {
      const int id = tid + i * C::kThreads;
      const int quad = id / kPairs;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const long long r = t + 4 * quad + u;
        if (id < kPatches && r < k.t1 && left > 0)
          zr[i][u].load(zp + r * p.z_stride + c, left, p.vec2);
      }
    }
  };

  if (k.t0 < k.t1) load_tile(k.t0);
  for (long long t = k.t0; t < k.t1; t += kTile) {
    Raw2<T> xc[C::kPerThread][4];
#pragma unroll
    for (int i = 0; i < C::kPerThread; ++i) {
      const int id = tid + i * C::kThreads;
      const int quad = id / kPairs;
      if (id < kPatches) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          xc[i][u] = xr[i][u];
          f32x2 d = add2(dr[i][u].get(), bias);
          if (p.softplus) d = softplus2(d);
          // tokens behind the end take no step (their softplus would)
          if (t + 4 * quad + u >= k.t1) d = pack2(0.f, 0.f);
          if (kSummary) sum = add2(sum, d);
          float d0, d1, u0, u1;
          unpack2(d, d0, d1);
          unpack2(mul2(d, xr[i][u].get()), u0, u1);
          s_du[2 * pair * (kTile + 1) + 4 * quad + u] = make_float4(d0, d0, u0, u0);
          s_du[(2 * pair + 1) * (kTile + 1) + 4 * quad + u] = make_float4(d1, d1, u1, u1);
        }
      }
    }
    s_b[tid] = br;
    if (!kSummary) s_c[tid] = cr;
    __syncthreads();
    if (!kSummary && p.z) load_gate(t);
    if (t + kTile < k.t1) load_tile(t + kTile);

    const int steps = (int)min((long long)kTile, k.t1 - t);
    auto step = [&](int i) -> float {
      const ulonglong2 du = *reinterpret_cast<const ulonglong2*>(&s_du[lc * (kTile + 1) + i]);
      const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&s_b[i * LPC + ln]);
      float e0, e1, e2, e3;
      unpack2(mul2(a01, du.x), e0, e1);
      unpack2(mul2(a23, du.x), e2, e3);
      h01 = fma2(pack2(ex2(e0), ex2(e1)), h01, mul2(b.x, du.y));
      h23 = fma2(pack2(ex2(e2), ex2(e3)), h23, mul2(b.y, du.y));
      if (kPad) {  // states that do not exist stay zero whatever the step
        float v0, v1, v2, v3;
        unpack2(h01, v0, v1);
        unpack2(h23, v2, v3);
        h01 = pack2(nst > 0 ? v0 : 0.f, nst > 1 ? v1 : 0.f);
        h23 = pack2(nst > 2 ? v2 : 0.f, nst > 3 ? v3 : 0.f);
      }
      if (kSummary) return 0.f;
      const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(&s_c[i * LPC + ln]);
      float y0, y1;
      unpack2(fma2(c.x, h01, mul2(c.y, h23)), y0, y1);
      return y0 + y1;
    };
    if (steps == kTile) {
#pragma unroll 2
      for (int i = 0; i < kTile; i += 4) {
        float4 v;
        v.x = step(i);
        v.y = step(i + 1);
        v.z = step(i + 2);
        v.w = step(i + 3);
        if (!kSummary) s_part[part_at(tid, i / 4)] = v;
      }
    } else {
      for (int i = 0; i < steps; ++i) {
        const float v = step(i);
        if (!kSummary)
          reinterpret_cast<float*>(&s_part[part_at(tid, i / 4)])[i % 4] = v;
      }
    }
    __syncthreads();

    if (!kSummary) {  // y of this thread's patches
#pragma unroll
      for (int i = 0; i < C::kPerThread; ++i) {
        const int id = tid + i * C::kThreads;
        const int quad = id / kPairs;
        if (id >= kPatches || left <= 0) continue;
        float4 y0 = s_part[part_at(2 * pair * LPC, quad)];
        float4 y1 = s_part[part_at((2 * pair + 1) * LPC, quad)];
#pragma unroll
        for (int l = 1; l < LPC; ++l) {
          const float4 v0 = s_part[part_at(2 * pair * LPC + l, quad)];
          const float4 v1 = s_part[part_at((2 * pair + 1) * LPC + l, quad)];
          y0.x += v0.x, y0.y += v0.y, y0.z += v0.z, y0.w += v0.w;
          y1.x += v1.x, y1.y += v1.y, y1.z += v1.z, y1.w += v1.w;
        }
        const float w0[4] = {y0.x, y0.y, y0.z, y0.w}, w1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const long long r = t + 4 * quad + u;
          if (r >= k.t1) break;
          f32x2 y = pack2(w0[u], w1[u]);
          if (p.D) y = fma2(skip, xc[i][u].get(), y);
          if (p.z) {
            float g0, g1;
            unpack2(zr[i][u].get(), g0, g1);
            y = mul2(y, pack2(silu(g0), silu(g1)));
          }
          store2(static_cast<T*>(p.y) + r * p.dim + c, y, left, p.vec2);
        }
      }
    }
  }

  float4 v;
  unpack2(h01, v.x, v.y);
  unpack2(h23, v.z, v.w);
  if (kSummary) {
    const long long slot = first_slot(p, k.n) + k.c;
    if (nst > 0) store_h(p.ws_h + slot * hsize + hrow, v, nst, p.Ns);
    // the sum of the chunk's steps: kParts threads hold parts of each channel pair's
    constexpr int kParts = C::kThreads < kPatches ? C::kThreads / kPairs : kQuads;
    f32x2* parts = reinterpret_cast<f32x2*>(s_part);
    if (tid < kParts * kPairs) parts[tid] = sum;
    __syncthreads();
    if (tid < kCh && ch0 + tid < p.dim) {
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < kParts; ++i) a += reinterpret_cast<const float*>(parts)[i * kCh + tid];
      p.ws_sum[slot * p.dim + ch0 + tid] = a;
    }
  } else if (k.last && p.hT && nst > 0) {
    store_h(p.hT + k.n * hsize + hrow, v, nst, p.Ns);
  }
  // every block of the scan outlives the summaries, so what follows it in the stream may
  // reuse the workspace
  if (!kSummary && p.chunk && k.c == 0 && !p.ws_h0) griddep_wait();
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
    b = load_bc(static_cast<const T*>(p.B) + n * p.b_stride + n0, nst, p.vec_bc);
    c = load_bc(static_cast<const T*>(p.C) + n * p.c_stride + n0, nst, p.vec_bc);
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
cudaError_t launch_k(const S6Params& p, bool after_summary, cudaStream_t stream) {
  using C = Cfg<LPC, kSummary>;
  const auto kernel = s6_kernel<T, LPC, kPad, kSummary>;
  if (C::kBytes > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
    if (e != cudaSuccess) return e;
  }
  const int tiles = (p.dim + kCh - 1) / kCh;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = after_summary ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)tiles * (p.chunk ? p.slots : p.N)));
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
    const cudaError_t e = launch_k<T, LPC, kPad, true>(p, false, stream);
    if (e != cudaSuccess) return e;
  }
  // the scan's first chunks need no summary, so it may start while the summaries run
  return launch_k<T, LPC, kPad, false>(p, p.chunk != 0, stream);
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

int s6_chunk(int N, int T, int dim, int Ns, bool packed) {
  const long long ctas = (long long)N * ((dim + kCh - 1) / kCh);
  const long long tokens = packed ? T : (long long)N * T;
  const long long per_seq = N > 0 ? tokens / N : 0;  // packed: their mean
  if (ctas >= kSms || per_seq < 512) return 0;
  long long parts = (4 * kSms) / ctas;
  if (parts > 32) parts = 32;
  long long chunk = (per_seq + parts - 1) / parts;
  if (chunk < 256) chunk = 256;
  return (int)((chunk + kTile - 1) / kTile * kTile);
}

long long s6_slots(int N, int T, int chunk, bool packed) {
  if (!chunk) return N;
  if (packed) return (long long)T / chunk + N + 1;
  return (long long)N * (((long long)T + chunk - 1) / chunk);
}

size_t s6_ws_bytes(int N, int T, int dim, int Ns, bool packed) {
  const int chunk = s6_chunk(N, T, dim, Ns, packed);
  if (!chunk) return 0;
  const size_t up = 63;
  const size_t slots = (size_t)s6_slots(N, T, chunk, packed);
  const size_t sum = (slots * dim + up) & ~up, h = (slots * dim * Ns + up) & ~up;
  return (sum + h + (size_t)N * dim * Ns) * sizeof(float);
}

cudaError_t launch_s6(const S6Params& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_t<float>(p, stream) : launch_t<__nv_bfloat16>(p, stream);
}
cudaError_t launch_s6_step(const S6Params& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_step_t<float>(p, stream) : launch_step_t<__nv_bfloat16>(p, stream);
}

}  // namespace gdn
