// rotary_abi.cu - the extern "C" boundary of rotary positions (declared in include/gdn.h), and the
// table of frequencies, computed on the host.
#include <cmath>

#include "layer_check.h"
#include "layer_internal.h"

namespace {

using gdn::aligned;
using gdn::cuda_fail;
using gdn::fail;
using gdn::range_of;
using gdn::RotaryParams;
using gdn::Strided;

constexpr double kPi = 3.14159265358979323846;

gdn_status turns_of(int R, double base, int scaling, double factor, double original, double fast, double slow,
                    unsigned long long* turns, float* magnitude) {
  if (R < 2 || R % 2 || R > gdn::kRotaryMaxD)
    return fail(GDN_ERR_INVALID_ARG, "R=%d: an even number of columns from 2 to %d is rotated", R, gdn::kRotaryMaxD);
  if (scaling < GDN_ROTARY_PLAIN || scaling > GDN_ROTARY_YARN)
    return fail(GDN_ERR_INVALID_ARG, "scaling=%d is not a GDN_ROTARY_* value", scaling);
  if (!(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor))
    return fail(GDN_ERR_INVALID_ARG, "base=%g must be > 1, factor=%g >= 1", base, factor);
  if (scaling == GDN_ROTARY_YARN &&
      !(original > 0 && fast > slow && slow > 0 && std::isfinite(original) && std::isfinite(fast)))
    return fail(GDN_ERR_INVALID_ARG, "original_length=%g must be > 0, beta_fast=%g > beta_slow=%g > 0", original, fast,
                slow);
  if (!turns || !magnitude) return fail(GDN_ERR_INVALID_ARG, "turns and magnitude must be non-NULL");
  if (scaling == GDN_ROTARY_NTK && R > 2) base *= std::pow(factor, R / (R - 2.0));
  // the pair that makes `count` turns within the original length
  const auto pair_of = [&](double count) {
    return R * std::log(original / (count * 2 * kPi)) / (2 * std::log(base));
  };
  double low = 0, high = 1;
  if (scaling == GDN_ROTARY_YARN) {
    low = std::fmax(std::floor(pair_of(fast)), 0.0);
    high = std::fmin(std::ceil(pair_of(slow)), R - 1.0);
  }
  for (int i = 0; i < R / 2; ++i) {
    double freq = std::pow(base, -2.0 * i / R);
    if (scaling == GDN_ROTARY_LINEAR) freq /= factor;
    if (scaling == GDN_ROTARY_YARN) {
      const double s = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
      freq = freq * (1 - s) + freq / factor * s;
    }
    turns[i] = (unsigned long long)std::llround(std::ldexp(freq / (2 * kPi), 64 - 2)) << 2;  // (below 2^62)
  }
  *magnitude = scaling == GDN_ROTARY_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return GDN_OK;
}

gdn_status rotate(const void* q, const void* k, const unsigned long long* turns, const int32_t* positions,
                  const int32_t* offsets, const int32_t* cu, void* q_out, void* k_out, int N, int T, int Hq, int Hk,
                  int D, int R, long long q_stride, long long k_stride, long long q_out_stride,
                  long long k_out_stride, int interleaved, float magnitude, bool backward, bool f32,
                  gdn_stream_t stream) {
  const int elem = f32 ? 4 : 2;
  long long tokens = 0;
  GDN_TRY(gdn::check_tokens(N, T, D, cu, &tokens));
  if (D > gdn::kRotaryMaxD)
    return fail(GDN_ERR_UNSUPPORTED, "D=%d: heads of at most %d columns", D, gdn::kRotaryMaxD);
  if (R < 2 || R % 2 || R > D) return fail(GDN_ERR_INVALID_ARG, "R=%d must be even, from 2 to D=%d", R, D);
  if (Hq < 1 || Hk < 0 || (Hq > Hk ? Hq : Hk) > 0x7fffffff / 2 / D)
    return fail(GDN_ERR_INVALID_ARG, "Hq=%d must be > 0, Hk=%d >= 0, and not too large", Hq, Hk);
  if ((Hk == 0) != (k == nullptr && k_out == nullptr) && tokens > 0)
    return fail(GDN_ERR_INVALID_ARG, "k and k_out go with Hk > 0");
  if (tokens > gdn::kMaxGrid) return fail(GDN_ERR_INVALID_ARG, "problem too large: %lld tokens", tokens);
  const int cq = Hq * D, ck = Hk * D;
  GDN_TRY(gdn::check_rows("q", q, tokens, q_stride, cq, elem));
  GDN_TRY(gdn::check_rows("q_out", q_out, tokens, q_out_stride, cq, elem));
  if (Hk) {
    GDN_TRY(gdn::check_rows("k", k, tokens, k_stride, ck, elem));
    GDN_TRY(gdn::check_rows("k_out", k_out, tokens, k_out_stride, ck, elem));
  }
  if (tokens > 0 && !turns) return fail(GDN_ERR_INVALID_ARG, "turns must be non-NULL");
  if (!aligned(turns, 8) || !aligned(positions, 4) || !aligned(offsets, 4))
    return fail(GDN_ERR_INVALID_ARG, "turns must be 8-byte aligned, positions and offsets 4-byte");
  if (positions && (offsets || cu))
    return fail(GDN_ERR_INVALID_ARG, "positions stand for themselves: neither offsets nor cu_seqlens with them");
  const Strided iq{q, tokens, q_stride, cq, elem}, oq{q_out, tokens, q_out_stride, cq, elem};
  const Strided ik{k, Hk ? tokens : 0, k_stride, ck, elem}, ok{k_out, Hk ? tokens : 0, k_out_stride, ck, elem};
  const bool q_same = q == q_out && (tokens <= 1 || q_stride == q_out_stride);
  const bool k_same = k == k_out && (tokens <= 1 || k_stride == k_out_stride);
  bool bad = (!q_same && gdn::overlap(oq, iq)) || gdn::overlap(oq, ik) || gdn::overlap(ok, iq) ||
             (!k_same && gdn::overlap(ok, ik)) || gdn::overlap(oq, ok);
  const gdn::Range tables[] = {range_of(turns, R / 2, 8), range_of(positions, tokens, 4), range_of(offsets, N, 4),
                               range_of(cu, (long long)N + 1, 4)};
  for (const gdn::Range& r : tables)
    bad = bad || gdn::overlap(range_of(q_out, tokens, q_out_stride, cq, elem), r) ||
          gdn::overlap(range_of(Hk ? k_out : nullptr, tokens, k_out_stride, ck, elem), r);
  if (bad) return fail(GDN_ERR_INVALID_ARG, "the outputs must not overlap the inputs (each may be its own input)");
  if (tokens == 0) return GDN_OK;
  RotaryParams p{};
  p.q = q; p.k = k; p.q_out = q_out; p.k_out = k_out; p.turns = turns; p.positions = positions;
  p.offsets = offsets; p.cu = cu;
  p.q_stride = q_stride; p.k_stride = k_stride; p.q_out_stride = q_out_stride; p.k_out_stride = k_out_stride;
  p.tokens = tokens; p.N = N; p.T = T; p.Hq = Hq; p.Hk = Hk; p.D = D; p.R = R;
  p.interleaved = interleaved != 0; p.backward = backward; p.magnitude = magnitude;
  p.q_same = q_same; p.k_same = k_same;
  p.by = 1;
  for (int by = 16 / elem; by > 1 && p.by == 1; by /= 2) {
    bool fits = R / 2 % by == 0 && (D - R) % by == 0;
    for (const void* t : {q, k, (const void*)q_out, (const void*)k_out}) fits = fits && aligned(t, by * elem);
    for (const long long s : {q_stride, k ? k_stride : 0, q_out_stride, k ? k_out_stride : 0})
      fits = fits && (tokens <= 1 || s % by == 0);
    if (fits) p.by = by;
  }
  const cudaError_t e = gdn::launch_rotary(p, f32, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GDN_OK : cuda_fail(e, "launching the rotary positions");
}

}  // namespace

extern "C" {

gdn_status gdn_rotary_turns(int R, double base, int scaling, double factor, double original_length, double beta_fast,
                            double beta_slow, unsigned long long* turns, float* magnitude) {
  return turns_of(R, base, scaling, factor, original_length, beta_fast, beta_slow, turns, magnitude);
}

#define GDN_ROTARY_ENTRY(name, type, backward, f32)                                                                  \
  gdn_status name(const type* q, const type* k, const unsigned long long* turns, const int32_t* positions,           \
                  const int32_t* offsets, const int32_t* cu_seqlens, type* q_out, type* k_out, int N, int T, int Hq, \
                  int Hk, int D, int R, long long q_stride, long long k_stride, long long q_out_stride,              \
                  long long k_out_stride, int interleaved, float magnitude, gdn_stream_t stream) {                   \
    return rotate(q, k, turns, positions, offsets, cu_seqlens, q_out, k_out, N, T, Hq, Hk, D, R, q_stride, k_stride, \
                  q_out_stride, k_out_stride, interleaved, magnitude, backward, f32, stream);                        \
  }
GDN_ROTARY_ENTRY(gdn_rotary_fwd, void, false, false)
GDN_ROTARY_ENTRY(gdn_rotary_fwd_f32, float, false, true)
GDN_ROTARY_ENTRY(gdn_rotary_bwd, void, true, false)
GDN_ROTARY_ENTRY(gdn_rotary_bwd_f32, float, true, true)

}  // extern "C"
