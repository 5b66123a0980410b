// layer_abi.cu - the extern "C" boundary of the layer operators (declared in include/gdn.h):
// the short causal convolution, the S6 scan and the RMS norm.
//
// Validates arguments, maps them onto launch parameters and enqueues the kernels on the
// caller's stream.
#include <initializer_list>

#include "layer_check.h"
#include "layer_internal.h"

namespace {

using gdn::aligned;
using gdn::cuda_fail;
using gdn::fail;

using gdn::check_rows;
using gdn::check_tokens;
using gdn::kMaxGrid;
using gdn::overlap;
using gdn::Range;
using gdn::range_of;

constexpr int kMaxChannels = 1 << 30;  // of the scan: tiles of 32 are counted in 31 bits

// ---- short causal convolution --------------------------------------------------------
gdn_status check_conv(const void* x, const float* w, const float* bias, const void* s0, void* y,
                      void* sT, int N, int T, int D, int W, long long x_stride, int activation,
                      const int32_t* cu, int elem, gdn::ConvParams* p) {
  long long tokens = 0;
  GDN_TRY(check_tokens(N, T, D, cu, &tokens));
  if (W < 2 || W > 4) return fail(GDN_ERR_UNSUPPORTED, "W=%d: supported filters have 2 to 4 taps", W);
  if (activation != GDN_ACT_NONE && activation != GDN_ACT_SILU)
    return fail(GDN_ERR_INVALID_ARG, "activation=%d is not a GDN_ACT_* value", activation);
  GDN_TRY(check_rows("x", x, tokens, x_stride, D, elem));
  if (tokens > 0 && (!w || !y)) return fail(GDN_ERR_INVALID_ARG, "w and y must be non-NULL");
  if (!aligned(w, 16)) return fail(GDN_ERR_INVALID_ARG, "w must be 16-byte aligned");
  if (!aligned(bias, 4)) return fail(GDN_ERR_INVALID_ARG, "bias must be 4-byte aligned");
  if (!aligned(y, elem) || !aligned(s0, elem) || !aligned(sT, elem))
    return fail(GDN_ERR_INVALID_ARG, "y, s0 and sT must be %d-byte aligned", elem);
  const long long states = (long long)N * (W - 1) * D;
  const Range ry = range_of(y, tokens * D, elem), r0 = range_of(s0, states, elem),
              rT = range_of(sT, states, elem);
  const Range in[] = {range_of(x, tokens, x_stride, D, elem), range_of(w, (long long)D * W, 4),
                      range_of(bias, D, 4), range_of(cu, (long long)N + 1, 4)};
  for (const Range& r : in)
    if (overlap(ry, r) || overlap(rT, r))
      return fail(GDN_ERR_INVALID_ARG, "y and sT must not overlap the inputs (sT may be s0)");
  if (overlap(ry, r0) || overlap(ry, rT) || (s0 != sT && overlap(r0, rT)))
    return fail(GDN_ERR_INVALID_ARG, "y and sT must not overlap the inputs (sT may be s0)");
  // blocks of 4 or more tokens, one per state; 256 channels a block or more
  if (tokens / 4 + N + 1 > kMaxGrid || D > 65535 * 256)
    return fail(GDN_ERR_INVALID_ARG, "problem too large: %lld tokens, D=%d", tokens, D);
  p->x = x; p->w = w; p->bias = bias; p->s0 = s0; p->y = y; p->sT = sT; p->cu = cu;
  p->x_stride = x_stride;
  p->N = N; p->T = T; p->D = D; p->W = W;
  p->silu = activation == GDN_ACT_SILU;
  const int four = 4 * elem;
  p->vec = D % 4 == 0 && (tokens <= 1 || x_stride % 4 == 0) && aligned(x, four) &&
           aligned(y, four) && aligned(s0, four) && aligned(sT, four);
  return GDN_OK;
}

gdn_status run_conv(const gdn::ConvParams& p, bool f32, gdn_stream_t stream) {
  const long long tokens = p.cu ? (long long)p.T : (long long)p.N * p.T;
  if (p.N == 0 || (tokens == 0 && !p.sT)) return GDN_OK;
  const cudaError_t e = gdn::launch_conv(p, f32, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GDN_OK : cuda_fail(e, "launching the short convolution");
}

gdn_status conv_step(const void* x, const float* w, const float* bias, void* s, void* y, int N,
                     int D, int W, long long x_stride, int activation, bool f32,
                     gdn_stream_t stream) {
  gdn::ConvParams p;
  GDN_TRY(check_conv(x, w, bias, s, y, s, N, 1, D, W, x_stride, activation, nullptr, f32 ? 4 : 2, &p));
  if (N > 0 && !s) return fail(GDN_ERR_INVALID_ARG, "s must be non-NULL");
  if ((long long)N * ((D + 3) / 4) / 64 > kMaxGrid)
    return fail(GDN_ERR_INVALID_ARG, "N=%d, D=%d too large", N, D);
  if (N == 0) return GDN_OK;
  const cudaError_t e = gdn::launch_conv_step(p, f32, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GDN_OK : cuda_fail(e, "launching the short convolution's step");
}

// ---- S6 scan ---------------------------------------------------------------------------
gdn_status check_s6(const void* x, const void* dt, const float* A, const void* B, const void* C,
                    const float* D, const void* z, const float* dt_bias, const float* h0, void* y,
                    float* hT, int N, int T, int dim, int Ns, long long x_stride,
                    long long dt_stride, long long b_stride, long long c_stride,
                    long long z_stride, int dt_softplus, const int32_t* cu, int elem,
                    gdn::S6Params* p) {
  long long tokens = 0;
  GDN_TRY(check_tokens(N, T, dim, cu, &tokens));
  if (Ns < 1) return fail(GDN_ERR_INVALID_ARG, "Ns=%d must be > 0", Ns);
  if (Ns > 64) return fail(GDN_ERR_UNSUPPORTED, "Ns=%d: at most 64 states per channel", Ns);
  if (dim > kMaxChannels) return fail(GDN_ERR_INVALID_ARG, "problem too large: D=%d", dim);
  GDN_TRY(check_rows("x", x, tokens, x_stride, dim, elem));
  GDN_TRY(check_rows("dt", dt, tokens, dt_stride, dim, elem));
  GDN_TRY(check_rows("B", B, tokens, b_stride, Ns, elem));
  GDN_TRY(check_rows("C", C, tokens, c_stride, Ns, elem));
  if (z) GDN_TRY(check_rows("z", z, tokens, z_stride, dim, elem));
  if (N > 0 && !A) return fail(GDN_ERR_INVALID_ARG, "A must be non-NULL");
  if (tokens > 0 && !y) return fail(GDN_ERR_INVALID_ARG, "y must be non-NULL");
  if (!aligned(A, 16) || !aligned(h0, 16) || !aligned(hT, 16))
    return fail(GDN_ERR_INVALID_ARG, "A, h0 and hT must be 16-byte aligned");
  if (!aligned(D, 4) || !aligned(dt_bias, 4) || !aligned(y, elem))
    return fail(GDN_ERR_INVALID_ARG, "D and dt_bias must be 4-byte aligned, y %d-byte", elem);
  const long long states = (long long)N * dim * Ns;
  const Range ry = range_of(y, tokens * dim, elem), r0 = range_of(h0, states, 4),
              rT = range_of(hT, states, 4);
  const Range in[] = {range_of(x, tokens, x_stride, dim, elem),
                      range_of(dt, tokens, dt_stride, dim, elem),
                      range_of(B, tokens, b_stride, Ns, elem),
                      range_of(C, tokens, c_stride, Ns, elem),
                      range_of(z, tokens, z_stride, dim, elem),
                      range_of(A, (long long)dim * Ns, 4),
                      range_of(D, dim, 4),
                      range_of(dt_bias, dim, 4),
                      range_of(cu, (long long)N + 1, 4)};
  for (const Range& r : in)
    if (overlap(ry, r) || overlap(rT, r))
      return fail(GDN_ERR_INVALID_ARG, "y and hT must not overlap the inputs (hT may be h0)");
  if (overlap(ry, r0) || overlap(ry, rT) || (h0 != hT && overlap(r0, rT)))
    return fail(GDN_ERR_INVALID_ARG, "y and hT must not overlap the inputs (hT may be h0)");
  p->x = x; p->dt = dt; p->B = B; p->C = C; p->z = z;
  p->A = A; p->D = D; p->dt_bias = dt_bias; p->h0 = h0; p->y = y; p->hT = hT; p->cu = cu;
  p->x_stride = x_stride; p->dt_stride = dt_stride; p->b_stride = b_stride;
  p->c_stride = c_stride; p->z_stride = z_stride;
  p->N = N; p->T = T; p->dim = dim; p->Ns = Ns;
  p->softplus = dt_softplus != 0;
  // How wide rows can be copied: their first elements, strides and lengths decide.
  const bool one = tokens <= 1;
  const auto rows_are = [&](int n, std::initializer_list<const void*> ptrs,
                            std::initializer_list<long long> strides, int cols) {
    bool ok = cols % n == 0;
    for (const void* q : ptrs) ok = ok && aligned(q, n * elem);
    for (const long long st : strides) ok = ok && (one || st % n == 0);
    return ok;
  };
  const long long zst = z ? z_stride : 0;
  p->copy = rows_are(16 / elem, {x, dt, z}, {x_stride, dt_stride, zst}, dim) ? 16
            : rows_are(4 / elem, {x, dt, z}, {x_stride, dt_stride, zst}, dim) ? 4 : 2;
  p->vec_bc = rows_are(4, {B, C}, {b_stride, c_stride}, Ns);
  p->copy_bc = p->vec_bc ? 4 * elem : rows_are(4 / elem, {B, C}, {b_stride, c_stride}, Ns) ? 4 : 2;
  p->vec2 = dim % 2 == 0 && aligned(y, 2 * elem);
  p->lone = 0;
  p->whole = 0; p->chunk = 0; p->slots = 0;
  p->ws_sum = nullptr; p->ws_h = nullptr; p->ws_h0 = nullptr;
  return GDN_OK;
}

gdn_status run_s6(gdn::S6Params p, bool f32, void* ws, size_t ws_bytes, gdn_stream_t stream) {
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const long long tokens = p.cu ? (long long)p.T : (long long)p.N * p.T;
  if (p.N == 0 || (tokens == 0 && !p.hT)) return GDN_OK;
  const gdn::S6Split split = gdn::s6_split(p.N, p.T, p.dim, p.Ns, p.cu != nullptr);
  const long long tiles = (p.dim + 31) / 32;
  if ((split.slots + p.N) * tiles > kMaxGrid)
    return fail(GDN_ERR_INVALID_ARG, "problem too large: N=%d T=%d D=%d", p.N, p.T, p.dim);
  p.whole = split.whole;
  p.chunk = split.chunk;
  p.lone = split.lone;
  p.slots = (int)split.slots;
  const size_t need = split.ws_bytes;
  void* pool = nullptr;
  if (need) {
    if (ws) {
      if (!aligned(ws, 256) || ws_bytes < need)
        return fail(GDN_ERR_INVALID_ARG, "workspace %p of %zu bytes: need %zu bytes, 256-byte aligned",
                    ws, ws_bytes, need);
    } else {
      const cudaError_t e = cudaMallocAsync(&pool, need, st);
      if (e != cudaSuccess) return cuda_fail(e, "allocating the workspace");
      ws = pool;
    }
    p.ws_sum = static_cast<float*>(ws);
    p.ws_h = p.ws_sum + split.sum_floats;
    if (p.h0 && p.h0 == p.hT) p.ws_h0 = p.ws_h + split.h_floats;
  }
  const cudaError_t e = gdn::launch_s6(p, f32, st);
  const cudaError_t ef = pool ? cudaFreeAsync(pool, st) : cudaSuccess;
  if (e != cudaSuccess) return cuda_fail(e, "launching the S6 scan");
  return ef == cudaSuccess ? GDN_OK : cuda_fail(ef, "freeing the workspace");
}

gdn_status s6_step(const void* x, const void* dt, const float* A, const void* B, const void* C,
                   const float* D, const void* z, const float* dt_bias, float* h, void* y, int N,
                   int dim, int Ns, long long x_stride, long long dt_stride, long long b_stride,
                   long long c_stride, long long z_stride, int dt_softplus, bool f32,
                   gdn_stream_t stream) {
  gdn::S6Params p;
  GDN_TRY(check_s6(x, dt, A, B, C, D, z, dt_bias, h, y, h, N, 1, dim, Ns, x_stride, dt_stride,
                   b_stride, c_stride, z_stride, dt_softplus, nullptr, f32 ? 4 : 2, &p));
  if (N > 0 && !h) return fail(GDN_ERR_INVALID_ARG, "h must be non-NULL");
  // (a lane's four sequences are counted in 31 bits)
  if ((long long)N * ((long long)dim * 16 / 256 + 1) > kMaxGrid - 4 || dim > (1 << 26))
    return fail(GDN_ERR_INVALID_ARG, "N=%d, D=%d too large", N, dim);
  if (N == 0) return GDN_OK;
  const cudaError_t e = gdn::launch_s6_step(p, f32, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GDN_OK : cuda_fail(e, "launching the S6 step");
}

// ---- RMS norm ----------------------------------------------------------------------------
gdn_status run_norm(const void* x, const float* w, const void* residual, const void* gate, void* y,
                    float* scales, void* residual_out, long long tokens, int heads, int D,
                    long long x_stride, long long gate_stride, int group, float eps, bool f32,
                    bool fp8, gdn_stream_t stream) {
  const int elem = f32 ? 4 : 2;
  if (tokens < 0 || heads <= 0 || D <= 0)
    return fail(GDN_ERR_INVALID_ARG, "tokens=%lld must be >= 0, heads=%d and D=%d > 0", tokens,
                heads, D);
  if (D > gdn::kNormMaxD)
    return fail(GDN_ERR_UNSUPPORTED, "D=%d: rows of at most %d columns", D, gdn::kNormMaxD);
  if (!(eps >= 0.f)) return fail(GDN_ERR_INVALID_ARG, "eps must be >= 0");
  if (tokens > kMaxGrid / heads || (long long)heads * D > 0x7fffffffll)
    return fail(GDN_ERR_INVALID_ARG, "problem too large: tokens=%lld heads=%d D=%d", tokens, heads, D);
  if (group != 0 && group != 32 && group != 64 && group != 128)
    return fail(GDN_ERR_UNSUPPORTED, "group=%d: scales cover 32, 64, 128 columns or a row (0)", group);
  const long long rows = tokens * heads;
  const long long cols = (long long)heads * D;
  GDN_TRY(check_rows("x", x, tokens, x_stride, (int)cols, elem));
  if (gate) GDN_TRY(check_rows("gate", gate, tokens, gate_stride, (int)cols, elem));
  if (rows > 0 && (!w || !y || (fp8 && !scales)))
    return fail(GDN_ERR_INVALID_ARG, "w, y (and scales) must be non-NULL");
  if ((residual == nullptr) != (residual_out == nullptr))
    return fail(GDN_ERR_INVALID_ARG, "residual and residual_out go together");
  if (!aligned(w, 4) || !aligned(scales, 4) || !aligned(y, fp8 ? 1 : elem) ||
      !aligned(residual, elem) || !aligned(residual_out, elem))
    return fail(GDN_ERR_INVALID_ARG, "misaligned pointer (each to its element size)");
  const int ycols = fp8 ? 1 : elem;
  const int span = group ? group : D;
  const Range ry = range_of(y, rows * D, ycols), ro = range_of(residual_out, rows * D, elem),
              rs = range_of(scales, fp8 ? rows * ((D + span - 1) / span) : 0, 4),
              rr = range_of(residual, rows * D, elem);
  const Range in[] = {range_of(x, tokens, x_stride, cols, elem),
                      range_of(gate, tokens, gate_stride, cols, elem), range_of(w, D, 4)};
  for (const Range& r : in)
    if (overlap(ry, r) || overlap(ro, r) || overlap(rs, r))
      return fail(GDN_ERR_INVALID_ARG, "the outputs must not overlap the inputs");
  if (overlap(ry, ro) || overlap(ry, rs) || overlap(ro, rs) || overlap(ry, rr) || overlap(rs, rr) ||
      (residual != residual_out && overlap(ro, rr)))
    return fail(GDN_ERR_INVALID_ARG,
                "the outputs must not overlap each other or the inputs (residual_out may be residual)");
  if (rows == 0) return GDN_OK;
  gdn::NormParams p;
  p.x = x; p.residual = residual; p.gate = gate; p.w = w; p.y = y;
  p.residual_out = residual_out; p.scales = scales;
  p.rows = rows; p.x_stride = x_stride; p.gate_stride = gate_stride;
  p.heads = heads; p.D = D; p.eps = eps;
  p.inv_d = 1.f / (float)D;
  p.group_log = group == 32 ? 5 : group == 64 ? 6 : 7;
  p.group = span < D ? span : D;
  p.groups = (D + p.group - 1) / p.group;
  const bool one = tokens <= 1;
  // the widest accesses that every tensor allows: of 8, 4 or 2 columns, 16 bytes at most
  const auto fits = [&](int by) {
    const size_t wide = by * elem < 16 ? by * elem : 16, of_w = by * 4 < 16 ? by * 4 : 16;
    return D % by == 0 && aligned(x, wide) && aligned(residual, wide) && aligned(residual_out, wide) &&
           aligned(gate, wide) && aligned(w, of_w) && aligned(y, fp8 ? by : wide) &&
           (one || x_stride * elem % (long long)wide == 0) &&
           (one || !gate || gate_stride * elem % (long long)wide == 0);
  };
  p.by = fits(8) ? 8 : fits(4) ? 4 : fits(2) ? 2 : 1;
  p.err = nullptr;
  const cudaError_t e = gdn::launch_norm(p, f32, fp8, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GDN_OK : cuda_fail(e, "launching the RMS norm");
}

}  // namespace

extern "C" {

gdn_status gdn_short_conv_fwd(const void* x, const float* w, const float* bias, const void* s0,
                              void* y, void* sT, int N, int T, int D, int W, long long x_stride,
                              int activation, const int32_t* cu_seqlens, gdn_stream_t stream) {
  gdn::ConvParams p;
  GDN_TRY(check_conv(x, w, bias, s0, y, sT, N, T, D, W, x_stride, activation, cu_seqlens, 2, &p));
  return run_conv(p, false, stream);
}

gdn_status gdn_short_conv_fwd_f32(const float* x, const float* w, const float* bias,
                                  const float* s0, float* y, float* sT, int N, int T, int D, int W,
                                  long long x_stride, int activation, const int32_t* cu_seqlens,
                                  gdn_stream_t stream) {
  gdn::ConvParams p;
  GDN_TRY(check_conv(x, w, bias, s0, y, sT, N, T, D, W, x_stride, activation, cu_seqlens, 4, &p));
  return run_conv(p, true, stream);
}

gdn_status gdn_short_conv_step(const void* x, const float* w, const float* bias, void* s, void* y,
                               int N, int D, int W, long long x_stride, int activation,
                               gdn_stream_t stream) {
  return conv_step(x, w, bias, s, y, N, D, W, x_stride, activation, false, stream);
}

gdn_status gdn_short_conv_step_f32(const float* x, const float* w, const float* bias, float* s,
                                   float* y, int N, int D, int W, long long x_stride,
                                   int activation, gdn_stream_t stream) {
  return conv_step(x, w, bias, s, y, N, D, W, x_stride, activation, true, stream);
}

size_t gdn_s6_chunk_fwd_workspace_size(int N, int T, int dim, int Ns, int has_cu_seqlens) {
  if (N < 0 || T < 0 || dim <= 0 || dim > kMaxChannels || Ns < 1 || Ns > 64 || (has_cu_seqlens && N < 1))
    return 0;
  return gdn::s6_split(N, T, dim, Ns, has_cu_seqlens != 0).ws_bytes;
}

gdn_status gdn_s6_chunk_fwd(const void* x, const void* dt, const float* A, const void* B,
                            const void* C, const float* D, const void* z, const float* dt_bias,
                            const float* h0, void* y, float* hT, int N, int T, int dim, int Ns,
                            long long x_stride, long long dt_stride, long long b_stride,
                            long long c_stride, long long z_stride, int dt_softplus,
                            const int32_t* cu_seqlens, void* workspace, size_t workspace_bytes,
                            gdn_stream_t stream) {
  gdn::S6Params p;
  GDN_TRY(check_s6(x, dt, A, B, C, D, z, dt_bias, h0, y, hT, N, T, dim, Ns, x_stride, dt_stride,
                   b_stride, c_stride, z_stride, dt_softplus, cu_seqlens, 2, &p));
  return run_s6(p, false, workspace, workspace_bytes, stream);
}

gdn_status gdn_s6_chunk_fwd_f32(const float* x, const float* dt, const float* A, const float* B,
                                const float* C, const float* D, const float* z,
                                const float* dt_bias, const float* h0, float* y, float* hT, int N,
                                int T, int dim, int Ns, long long x_stride, long long dt_stride,
                                long long b_stride, long long c_stride, long long z_stride,
                                int dt_softplus, const int32_t* cu_seqlens, void* workspace,
                                size_t workspace_bytes, gdn_stream_t stream) {
  gdn::S6Params p;
  GDN_TRY(check_s6(x, dt, A, B, C, D, z, dt_bias, h0, y, hT, N, T, dim, Ns, x_stride, dt_stride,
                   b_stride, c_stride, z_stride, dt_softplus, cu_seqlens, 4, &p));
  return run_s6(p, true, workspace, workspace_bytes, stream);
}

gdn_status gdn_s6_recurrent_step(const void* x, const void* dt, const float* A, const void* B,
                                 const void* C, const float* D, const void* z,
                                 const float* dt_bias, float* h, void* y, int N, int dim, int Ns,
                                 long long x_stride, long long dt_stride, long long b_stride,
                                 long long c_stride, long long z_stride, int dt_softplus,
                                 gdn_stream_t stream) {
  return s6_step(x, dt, A, B, C, D, z, dt_bias, h, y, N, dim, Ns, x_stride, dt_stride, b_stride,
                 c_stride, z_stride, dt_softplus, false, stream);
}

gdn_status gdn_s6_recurrent_step_f32(const float* x, const float* dt, const float* A,
                                     const float* B, const float* C, const float* D,
                                     const float* z, const float* dt_bias, float* h, float* y,
                                     int N, int dim, int Ns, long long x_stride,
                                     long long dt_stride, long long b_stride, long long c_stride,
                                     long long z_stride, int dt_softplus, gdn_stream_t stream) {
  return s6_step(x, dt, A, B, C, D, z, dt_bias, h, y, N, dim, Ns, x_stride, dt_stride, b_stride,
                 c_stride, z_stride, dt_softplus, true, stream);
}

gdn_status gdn_rms_norm_fwd(const void* x, const float* w, const void* residual, const void* gate,
                            void* y, void* residual_out, long long tokens, int heads, int D,
                            long long x_stride, long long gate_stride, float eps,
                            gdn_stream_t stream) {
  return run_norm(x, w, residual, gate, y, nullptr, residual_out, tokens, heads, D, x_stride,
                  gate_stride, 0, eps, false, false, stream);
}

gdn_status gdn_rms_norm_fwd_f32(const float* x, const float* w, const float* residual,
                                const float* gate, float* y, float* residual_out, long long tokens,
                                int heads, int D, long long x_stride, long long gate_stride,
                                float eps, gdn_stream_t stream) {
  return run_norm(x, w, residual, gate, y, nullptr, residual_out, tokens, heads, D, x_stride,
                  gate_stride, 0, eps, true, false, stream);
}

gdn_status gdn_rms_norm_fwd_e4m3(const void* x, const float* w, const void* residual,
                                 const void* gate, void* y, float* scales, void* residual_out,
                                 long long tokens, int heads, int D, long long x_stride,
                                 long long gate_stride, int group, float eps,
                                 gdn_stream_t stream) {
  return run_norm(x, w, residual, gate, y, scales, residual_out, tokens, heads, D, x_stride,
                  gate_stride, group, eps, false, true, stream);
}

gdn_status gdn_rms_norm_fwd_e4m3_f32(const float* x, const float* w, const float* residual,
                                     const float* gate, void* y, float* scales,
                                     float* residual_out, long long tokens, int heads, int D,
                                     long long x_stride, long long gate_stride, int group,
                                     float eps, gdn_stream_t stream) {
  return run_norm(x, w, residual, gate, y, scales, residual_out, tokens, heads, D, x_stride,
                  gate_stride, group, eps, true, true, stream);
}

}  // extern "C"
