// glr_abi.cu - the extern "C" boundary of the gated linear recurrence (declared in include/gdn.h).
#include <initializer_list>

#include "layer_check.h"
#include "layer_internal.h"

namespace {

using gdn::aligned;
using gdn::cuda_fail;
using gdn::fail;
using gdn::GlrParams;
using gdn::range_of;

constexpr int kMaxChannels = 1 << 30;

bool known(int gate, int norm) {
  return gate >= GDN_GLR_GATE_LOG && gate <= GDN_GLR_GATE_RATE && norm >= GDN_GLR_INPUT_PLAIN &&
         norm <= GDN_GLR_INPUT_SQRT;
}

// What every call shares.
gdn_status check(const void* x, const void* g, const float* rate, int N, int T, int D, long long x_stride,
                 long long g_stride, int gate, int norm, const int32_t* cu, int elem, long long* tokens,
                 GlrParams* p) {
  GDN_TRY(gdn::check_tokens(N, T, D, cu, tokens));
  if (D > kMaxChannels) return fail(GDN_ERR_INVALID_ARG, "problem too large: D=%d", D);
  if (!known(gate, norm))
    return fail(GDN_ERR_INVALID_ARG, "gate=%d, input_norm=%d: no GDN_GLR_GATE_*, GDN_GLR_INPUT_* values", gate, norm);
  if ((gate == GDN_GLR_GATE_RATE) != (rate != nullptr))
    return fail(GDN_ERR_INVALID_ARG, "rate belongs to GDN_GLR_GATE_RATE, and that gate needs one");
  GDN_TRY(gdn::check_rows("x", x, *tokens, x_stride, D, elem));
  GDN_TRY(gdn::check_rows("g", g, *tokens, g_stride, D, elem));
  *p = GlrParams{};
  p->x = x; p->g = g; p->rate = rate; p->cu = cu;
  p->x_stride = x_stride; p->g_stride = g_stride;
  p->N = N; p->T = T; p->D = D; p->gate = gate; p->norm = norm;
  p->tiles = (D - 1) / 64 + 1;
  p->chunks = ((long long)T + gdn::kGlrChunk - 1) / gdn::kGlrChunk;
  if (gdn::glr_units(*p) * gdn::glr_most_blocks(*p) > gdn::kMaxGrid)
    return fail(GDN_ERR_INVALID_ARG, "problem too large: N=%d D=%d", N, D);
  return GDN_OK;
}
gdn_status floats_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    if (!aligned(q, 4)) return fail(GDN_ERR_INVALID_ARG, "fp32 operands must be 4-byte aligned");
  return GDN_OK;
}
// Whether pairs of channels can be accessed together.
int pairs(const GlrParams& p, long long tokens, int elem, std::initializer_list<const void*> rows,
          std::initializer_list<const void*> floats) {
  bool ok = p.D % 2 == 0 && (tokens <= 1 || (p.x_stride % 2 == 0 && p.g_stride % 2 == 0 && p.dy_stride % 2 == 0));
  for (const void* q : rows) ok = ok && aligned(q, 2 * elem);
  for (const void* q : floats) ok = ok && aligned(q, 8);
  return ok;
}
// The widest pieces that rows of x and g (and dy) can be copied in.
int piece_of(const GlrParams& p, long long tokens, int elem, std::initializer_list<const void*> rows) {
  for (const int piece : {16, 4}) {
    const int n = piece / elem;
    bool ok = p.D % n == 0 &&
              (tokens <= 1 || (p.x_stride % n == 0 && p.g_stride % n == 0 && p.dy_stride % n == 0));
    for (const void* q : rows) ok = ok && aligned(q, piece);
    if (ok) return piece;
  }
  return 2;
}

gdn_status forward(const void* x, const void* g, const float* rate, const float* h0, void* y, float* hT,
                   float* states, int N, int T, int D, long long x_stride, long long g_stride, int gate, int norm,
                   const int32_t* cu, bool f32, gdn_stream_t stream) {
  const int elem = f32 ? 4 : 2;
  long long tokens = 0;
  GlrParams p;
  GDN_TRY(check(x, g, rate, N, T, D, x_stride, g_stride, gate, norm, cu, elem, &tokens, &p));
  if (tokens > 0 && !y) return fail(GDN_ERR_INVALID_ARG, "y must be non-NULL");
  if (!aligned(y, elem)) return fail(GDN_ERR_INVALID_ARG, "y must be %d-byte aligned", elem);
  GDN_TRY(floats_aligned({rate, h0, hT, states}));
  const long long rows = cu ? 1 : N, all = (long long)N * D;
  const gdn::Range outs[] = {range_of(y, tokens * D, elem), range_of(hT, all, 4),
                             range_of(states, rows * p.chunks * D, 4)};
  const gdn::Range in[] = {range_of(x, tokens, x_stride, D, elem), range_of(g, tokens, g_stride, D, elem),
                           range_of(rate, D, 4), range_of(cu, (long long)N + 1, 4), range_of(h0, all, 4)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 5; ++j)
      if (gdn::overlap(outs[i], in[j]) && !(i == 1 && j == 4 && h0 == hT))
        return fail(GDN_ERR_INVALID_ARG, "the outputs must not overlap the inputs (hT may be h0)");
    for (int j = 0; j < i; ++j)
      if (gdn::overlap(outs[i], outs[j])) return fail(GDN_ERR_INVALID_ARG, "the outputs must not overlap each other");
  }
  if (N == 0 || (tokens == 0 && !hT)) return GDN_OK;
  p.h0 = h0; p.y = y; p.hT = hT; p.states = states;
  p.vec = pairs(p, tokens, elem, {x, g, y}, {rate, h0, hT, states});
  p.piece = piece_of(p, tokens, elem, {x, g});
  const cudaError_t e = gdn::launch_glr(p, f32, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GDN_OK : cuda_fail(e, "launching the gated recurrence");
}

gdn_status step(const void* x, const void* g, const float* rate, float* h, void* y, int N, int D, long long x_stride,
                long long g_stride, int gate, int norm, bool f32, gdn_stream_t stream) {
  const int elem = f32 ? 4 : 2;
  long long tokens = 0;
  GlrParams p;
  GDN_TRY(check(x, g, rate, N, 1, D, x_stride, g_stride, gate, norm, nullptr, elem, &tokens, &p));
  if (N > 0 && (!y || !h)) return fail(GDN_ERR_INVALID_ARG, "h and y must be non-NULL");
  if (!aligned(y, elem)) return fail(GDN_ERR_INVALID_ARG, "y must be %d-byte aligned", elem);
  GDN_TRY(floats_aligned({rate, h}));
  const gdn::Range ry = range_of(y, tokens * D, elem), rh = range_of(h, tokens * D, 4);
  for (const gdn::Range& r : {range_of(x, tokens, x_stride, D, elem), range_of(g, tokens, g_stride, D, elem),
                              range_of(rate, D, 4)})
    if (gdn::overlap(ry, r) || gdn::overlap(rh, r))
      return fail(GDN_ERR_INVALID_ARG, "h and y must not overlap the inputs");
  if (gdn::overlap(ry, rh)) return fail(GDN_ERR_INVALID_ARG, "h and y must not overlap");
  if (N == 0) return GDN_OK;
  p.h0 = p.hT = h;
  p.y = y;
  p.vec = pairs(p, tokens, elem, {x, g, y}, {rate, h});
  const cudaError_t e = gdn::launch_glr_step(p, f32, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GDN_OK : cuda_fail(e, "launching the gated recurrence's step");
}

size_t partial_bytes(const GlrParams& p) {
  return p.gate == GDN_GLR_GATE_RATE ? (size_t)(p.cu ? 1 : p.N) * gdn::glr_most_blocks(p) * p.D * 4 : 0;
}

gdn_status backward(const void* dy, const void* x, const void* g, const float* rate, const float* h0,
                    const float* states, const float* dhT, void* dx, void* dg, float* drate, float* dh0, int N,
                    int T, int D, long long dy_stride, long long x_stride, long long g_stride, int gate, int norm,
                    const int32_t* cu, void* ws, size_t ws_bytes, bool f32, gdn_stream_t stream) {
  const int elem = f32 ? 4 : 2;
  long long tokens = 0;
  GlrParams p;
  GDN_TRY(check(x, g, rate, N, T, D, x_stride, g_stride, gate, norm, cu, elem, &tokens, &p));
  GDN_TRY(gdn::check_rows("dy", dy, tokens, dy_stride, D, elem));
  if (tokens > 0 && (!dx || !dg || !states))
    return fail(GDN_ERR_INVALID_ARG, "dx, dg and states must be non-NULL");
  if ((rate == nullptr) != (drate == nullptr)) return fail(GDN_ERR_INVALID_ARG, "rate and drate go together");
  if (!aligned(dx, elem) || !aligned(dg, elem))
    return fail(GDN_ERR_INVALID_ARG, "dx and dg must be %d-byte aligned", elem);
  GDN_TRY(floats_aligned({rate, h0, states, dhT, drate, dh0}));
  const long long rows = cu ? 1 : N, all = (long long)N * D;
  const gdn::Range outs[] = {range_of(dx, tokens * D, elem), range_of(dg, tokens * D, elem), range_of(drate, D, 4),
                             range_of(dh0, all, 4)};
  const gdn::Range in[] = {range_of(dy, tokens, dy_stride, D, elem), range_of(x, tokens, x_stride, D, elem),
                           range_of(g, tokens, g_stride, D, elem),   range_of(rate, D, 4),
                           range_of(h0, all, 4),                     range_of(states, rows * p.chunks * D, 4),
                           range_of(dhT, all, 4),                    range_of(cu, (long long)N + 1, 4)};
  for (int i = 0; i < 4; ++i) {
    for (const gdn::Range& r : in)
      if (gdn::overlap(outs[i], r)) return fail(GDN_ERR_INVALID_ARG, "the outputs must not overlap the inputs");
    for (int j = 0; j < i; ++j)
      if (gdn::overlap(outs[i], outs[j])) return fail(GDN_ERR_INVALID_ARG, "the outputs must not overlap each other");
  }
  if (rows * gdn::glr_most_blocks(p) > gdn::kMaxGrid) return fail(GDN_ERR_INVALID_ARG, "problem too large: N=%d", N);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0 || (tokens == 0 && !dh0)) {  // the rate's gradient is a sum over nothing
    const cudaError_t e = drate ? cudaMemsetAsync(drate, 0, (size_t)D * 4, st) : cudaSuccess;
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "clearing drate");
  }
  p.dy = dy; p.dy_stride = dy_stride; p.h0 = h0; p.kept = states; p.dhT = dhT; p.dx = dx; p.dg = dg; p.dh0 = dh0;
  p.vec = pairs(p, tokens, elem, {x, g, dy, dx, dg}, {rate, h0, states, dhT, dh0});
  p.piece = piece_of(p, tokens, elem, {x, g, dy});
  const size_t need = partial_bytes(p);
  void* pool = nullptr;
  if (need) {
    if (ws) {
      if (!aligned(ws, 256) || ws_bytes < need)
        return fail(GDN_ERR_INVALID_ARG, "workspace %p of %zu bytes: need %zu bytes, 256-byte aligned", ws, ws_bytes,
                    need);
    } else {
      const cudaError_t e = cudaMallocAsync(&pool, need, st);
      if (e != cudaSuccess) return cuda_fail(e, "allocating the workspace");
      ws = pool;
    }
    p.partial = static_cast<float*>(ws);
  }
  p.drate = drate;
  const cudaError_t e = gdn::launch_glr_bwd(p, f32, st);
  const cudaError_t ef = pool ? cudaFreeAsync(pool, st) : cudaSuccess;
  if (e != cudaSuccess) return cuda_fail(e, "launching the gated recurrence's gradient");
  return ef == cudaSuccess ? GDN_OK : cuda_fail(ef, "freeing the workspace");
}

}  // namespace

extern "C" {

gdn_status gdn_glr_chunk_fwd(const void* x, const void* g, const float* rate, const float* h0, void* y, float* hT,
                             float* states, int N, int T, int D, long long x_stride, long long g_stride, int gate,
                             int input_norm, const int32_t* cu_seqlens, gdn_stream_t stream) {
  return forward(x, g, rate, h0, y, hT, states, N, T, D, x_stride, g_stride, gate, input_norm, cu_seqlens, false,
                 stream);
}

gdn_status gdn_glr_chunk_fwd_f32(const float* x, const float* g, const float* rate, const float* h0, float* y,
                                 float* hT, float* states, int N, int T, int D, long long x_stride,
                                 long long g_stride, int gate, int input_norm, const int32_t* cu_seqlens,
                                 gdn_stream_t stream) {
  return forward(x, g, rate, h0, y, hT, states, N, T, D, x_stride, g_stride, gate, input_norm, cu_seqlens, true,
                 stream);
}

gdn_status gdn_glr_recurrent_step(const void* x, const void* g, const float* rate, float* h, void* y, int N, int D,
                                  long long x_stride, long long g_stride, int gate, int input_norm,
                                  gdn_stream_t stream) {
  return step(x, g, rate, h, y, N, D, x_stride, g_stride, gate, input_norm, false, stream);
}

gdn_status gdn_glr_recurrent_step_f32(const float* x, const float* g, const float* rate, float* h, float* y, int N,
                                      int D, long long x_stride, long long g_stride, int gate, int input_norm,
                                      gdn_stream_t stream) {
  return step(x, g, rate, h, y, N, D, x_stride, g_stride, gate, input_norm, true, stream);
}

size_t gdn_glr_chunk_bwd_workspace_size(int N, int T, int D, int gate, int has_cu_seqlens) {
  if (N < 0 || T < 0 || D <= 0 || D > kMaxChannels || !known(gate, GDN_GLR_INPUT_PLAIN) || (has_cu_seqlens && N < 1))
    return 0;
  GlrParams p{};
  const int32_t some = 0;
  p.N = N; p.T = T; p.D = D; p.gate = gate;
  p.cu = has_cu_seqlens ? &some : nullptr;
  return partial_bytes(p);
}

gdn_status gdn_glr_chunk_bwd(const void* dy, const void* x, const void* g, const float* rate, const float* h0,
                             const float* states, const float* dhT, void* dx, void* dg, float* drate, float* dh0,
                             int N, int T, int D, long long dy_stride, long long x_stride, long long g_stride,
                             int gate, int input_norm, const int32_t* cu_seqlens, void* workspace,
                             size_t workspace_bytes, gdn_stream_t stream) {
  return backward(dy, x, g, rate, h0, states, dhT, dx, dg, drate, dh0, N, T, D, dy_stride, x_stride, g_stride, gate,
                  input_norm, cu_seqlens, workspace, workspace_bytes, false, stream);
}

gdn_status gdn_glr_chunk_bwd_f32(const float* dy, const float* x, const float* g, const float* rate,
                                 const float* h0, const float* states, const float* dhT, float* dx, float* dg,
                                 float* drate, float* dh0, int N, int T, int D, long long dy_stride,
                                 long long x_stride, long long g_stride, int gate, int input_norm,
                                 const int32_t* cu_seqlens, void* workspace, size_t workspace_bytes,
                                 gdn_stream_t stream) {
  return backward(dy, x, g, rate, h0, states, dhT, dx, dg, drate, dh0, N, T, D, dy_stride, x_stride, g_stride, gate,
                  input_norm, cu_seqlens, workspace, workspace_bytes, true, stream);
}

}  // extern "C"
