// s6_step.cu - one token of the S6 recurrence per sequence (the decode step of s6_scan.cuh).
//
// The states are read and written once, 128 bytes a channel at Ns = 16: HBM bandwidth bounds
// many sequences, launch latency few.  A lane takes four states of one channel, LPC lanes a
// channel, and kSeqs sequences at once: that keeps enough reads in flight, shares A, and lets
// the lanes of a channel share what is computed once per sequence and channel (the step, the
// gate): each lane does it for its own sequence, and the parts of y are summed so that they
// end where they are needed.  128 x 5120, 16 states (bf16, 89 MB): 16.5 us in a graph (5.4 TB/s);
// 1 x 5120 2.0.
#include "layer_common.cuh"
#include "layer_internal.h"

namespace gdn {
namespace {

constexpr int kStepThreads = 256;

// kFull: Ns is 4 LPC and rows of B and C are aligned, so every lane has four states.  Bounds of
// four blocks an SM: 64 registers have the loads in flight at once (16.5 us; 56 by the compiler's
// own choice 18.2, bounds of five 17.4, of three 17.5).  Measured in bf16 with 16 states; fp32 with the
// same bounds spills 36 to 100 bytes (1 to 4 states off whole vectors: 332) in every variant but
// whole 16, 32 and 64 states (128 x 5120, events around a call, bf16 and fp32: 16 states 19.9 and
// 21.6 us, 8 states 14.5 and 20.6).
template <typename T, int LPC, int kSeqs, bool kFull>
__global__ void __launch_bounds__(kStepThreads, 4) s6_step_kernel(const S6Params p, int per_row) {
  // sequences a lane prepares and finishes: kOwn from number ln * kOwn on, of the kSeqs
  constexpr int kOwn = (kSeqs + LPC - 1) / LPC;
  const int bx = blockIdx.x % per_row;
  const int first = blockIdx.x / per_row * kSeqs;
  const int id = bx * kStepThreads + threadIdx.x;
  const bool some = id / LPC < p.dim;  // lanes behind the last channel only join the shuffles
  const int ch = some ? id / LPC : p.dim - 1, ln = id % LPC, n0 = ln * 4;
  const int Ns = kFull ? 4 * LPC : p.Ns, vec_bc = kFull ? 1 : p.vec_bc;
  const int nst = kFull ? 4 : some ? max(0, min(4, Ns - n0)) : 0;
  const long long hrow = (long long)ch * Ns + n0, hsize = (long long)p.dim * Ns;
  const bool all = first + kSeqs <= p.N;

  float4 h[kSeqs];
  float* hp = p.hT + first * hsize + hrow;
#pragma unroll
  for (int i = 0; i < kSeqs; ++i)
    h[i] = load_h(hp + (all || first + i < p.N ? i * hsize : 0), nst, Ns);
  Raw4<T> rb[kSeqs], rc[kSeqs];
  const T* bp = static_cast<const T*>(p.B) + first * p.b_stride + n0;
  const T* cp = static_cast<const T*>(p.C) + first * p.c_stride + n0;
#pragma unroll
  for (int i = 0; i < kSeqs; ++i) {
    const long long k = all || first + i < p.N ? i : 0;
    rb[i].zero();
    rc[i].zero();
    if (nst > 0) {
      rb[i].load(bp + k * p.b_stride, nst, vec_bc);
      rc[i].load(cp + k * p.c_stride, nst, vec_bc);
    }
  }
  float x[kOwn], d[kOwn], z[kOwn];
  bool mine[kOwn];
#pragma unroll
  for (int o = 0; o < kOwn; ++o) {
    const int i = ln * kOwn + o;
    mine[o] = i < kSeqs && first + i < p.N;
    const long long n = mine[o] ? first + i : first;
    x[o] = to_f32(static_cast<const T*>(p.x)[n * p.x_stride + ch]);
    d[o] = to_f32(static_cast<const T*>(p.dt)[n * p.dt_stride + ch]);
    z[o] = p.z ? to_f32(static_cast<const T*>(p.z)[n * p.z_stride + ch]) : 0.f;
  }
  const float4 a = load_h(p.A + hrow, nst, Ns);
  const float bias = p.dt_bias ? p.dt_bias[ch] : 0.f, skip = p.D ? p.D[ch] : 0.f;
  const float a0 = a.x * kLog2e, a1 = a.y * kLog2e, a2 = a.z * kLog2e, a3 = a.w * kLog2e;
  float u[kOwn];
#pragma unroll
  for (int o = 0; o < kOwn; ++o) {
    d[o] += bias;
    if (p.softplus) d[o] = softplus(d[o]);
    u[o] = d[o] * x[o];
  }

  float y[kSeqs];
#pragma unroll
  for (int i = 0; i < kSeqs; ++i) {
    // the step of sequence i, from the lane that has it
    float di = d[i % kOwn], ui = u[i % kOwn];
    if (LPC > 1) {
      di = __shfl_sync(0xffffffffu, di, i / kOwn, LPC);
      ui = __shfl_sync(0xffffffffu, ui, i / kOwn, LPC);
    }
    const float4 b = rb[i].get(), c = rc[i].get();
    float4 o;
    o.x = fmaf(ex2(di * a0), h[i].x, ui * b.x);
    o.y = fmaf(ex2(di * a1), h[i].y, ui * b.y);
    o.z = fmaf(ex2(di * a2), h[i].z, ui * b.z);
    o.w = fmaf(ex2(di * a3), h[i].w, ui * b.w);
    if ((!kFull || some) && (all || first + i < p.N)) store_h(hp + i * hsize, o, nst, Ns);
    y[i] = 0.f;  // only of states that exist
    if (nst > 0) y[i] = c.x * o.x;
    if (nst > 1) y[i] = fmaf(c.y, o.y, y[i]);
    if (nst > 2) y[i] = fmaf(c.z, o.z, y[i]);
    if (nst > 3) y[i] = fmaf(c.w, o.w, y[i]);
  }
  // Sums over the LPC lanes.  While there are several sequences a lane gives half of them away
  // for the other half's parts, so that a lane ends with the sequences it has; else plain sums.
#pragma unroll
  for (int off = LPC / 2, have = kSeqs; off > 0; off >>= 1) {
    if (have > 1 && off < kSeqs) {
      have /= 2;
      const bool up = ln & off;
#pragma unroll
      for (int i = 0; i < kSeqs / 2; ++i) {
        if (i >= have) break;
        const float send = up ? y[i] : y[i + have], keep = up ? y[i + have] : y[i];
        y[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kSeqs; ++i)
        if (i < have) y[i] += __shfl_xor_sync(0xffffffffu, y[i], off);
    }
  }
#pragma unroll
  for (int o = 0; o < kOwn; ++o) {
    if (!some || !mine[o]) continue;
    float v = y[o];
    if (p.D) v = fmaf(skip, x[o], v);
    if (p.z) v *= silu(z[o]);
    const long long n = first + ln * kOwn + o;
    from_f32(static_cast<T*>(p.y) + n * p.dim + ch, v);
  }
}

template <typename T, int LPC, bool kFull>
cudaError_t launch_step_f(const S6Params& p, cudaStream_t stream) {
  const int per_row = (int)(((long long)p.dim * LPC + kStepThreads - 1) / kStepThreads);
  const auto blocks = [&](int seqs) { return (long long)per_row * ((p.N + seqs - 1) / seqs); };
  // four sequences a lane once that still leaves two blocks per SM
  if (blocks(4) >= 2 * kSms)
    s6_step_kernel<T, LPC, 4, kFull><<<(unsigned)blocks(4), kStepThreads, 0, stream>>>(p, per_row);
  else
    s6_step_kernel<T, LPC, 1, kFull><<<(unsigned)blocks(1), kStepThreads, 0, stream>>>(p, per_row);
  return cudaGetLastError();
}

template <typename T, int LPC>
cudaError_t launch_step_l(const S6Params& p, cudaStream_t stream) {
  return p.Ns == 4 * LPC && p.vec_bc ? launch_step_f<T, LPC, true>(p, stream)
                                     : launch_step_f<T, LPC, false>(p, stream);
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

cudaError_t launch_s6_step(const S6Params& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_step_t<float>(p, stream) : launch_step_t<__nv_bfloat16>(p, stream);
}

}  // namespace gdn
