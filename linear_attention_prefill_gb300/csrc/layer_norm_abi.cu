// layer_norm_abi.cu - the extern "C" boundary of layer norm (declared in include/gdn.h).
#include "layer_check.h"
#include "layer_internal.h"

namespace {

using gdn::aligned;
using gdn::cuda_fail;
using gdn::fail;
using gdn::LnParams;
using gdn::range_of;

gdn_status check(const void* x, long long rows, int D, long long x_stride, float eps, int elem) {
  if (rows < 0 || D <= 0) return fail(GDN_ERR_INVALID_ARG, "rows=%lld must be >= 0, D=%d > 0", rows, D);
  if (D > gdn::kLnMaxD) return fail(GDN_ERR_UNSUPPORTED, "D=%d: rows of at most %d columns", D, gdn::kLnMaxD);
  if (!(eps >= 0.f)) return fail(GDN_ERR_INVALID_ARG, "eps must be >= 0");
  if (rows > gdn::kMaxGrid) return fail(GDN_ERR_INVALID_ARG, "problem too large: rows=%lld", rows);
  return gdn::check_rows("x", x, rows, x_stride, D, elem);
}

// Whether rows are made of vectors of 8 columns, 16 bytes aligned in every tensor.
int whole(const LnParams& p, int elem) {
  bool ok = p.D % 8 == 0;
  for (const void* q : {p.x, p.dy, p.residual, (const void*)p.y, (const void*)p.residual_out, (const void*)p.w,
                        (const void*)p.b})
    ok = ok && aligned(q, 16);
  for (const long long s : {p.x_stride, p.dy_stride}) ok = ok && (p.rows <= 1 || s * elem % 16 == 0);
  return ok;
}
// Blocks of a row, and the columns of each (whole vectors of 8).
void cut(LnParams* p) {
  p->inv_d = 1.f / (float)p->D;
  p->blocks = p->D <= gdn::kLnSlice ? 1 : p->D <= 2 * gdn::kLnSlice ? 2 : 4;
  p->slice = ((p->D + p->blocks - 1) / p->blocks + 7) / 8 * 8;
}

gdn_status forward(const void* x, const float* w, const float* b, const void* residual, void* y, void* residual_out,
                   long long rows, int D, long long x_stride, float eps, bool f32, gdn_stream_t stream) {
  const int elem = f32 ? 4 : 2;
  GDN_TRY(check(x, rows, D, x_stride, eps, elem));
  if (rows > 0 && !y) return fail(GDN_ERR_INVALID_ARG, "y must be non-NULL");
  if ((residual == nullptr) != (residual_out == nullptr))
    return fail(GDN_ERR_INVALID_ARG, "residual and residual_out go together");
  if (!aligned(w, 4) || !aligned(b, 4) || !aligned(y, elem) || !aligned(residual, elem) ||
      !aligned(residual_out, elem))
    return fail(GDN_ERR_INVALID_ARG, "misaligned pointer (each to its element size)");
  const gdn::Range ry = range_of(y, rows * D, elem), ro = range_of(residual_out, rows * D, elem),
                   rr = range_of(residual, rows * D, elem);
  for (const gdn::Range& r : {range_of(x, rows, x_stride, D, elem), range_of(w, D, 4), range_of(b, D, 4)})
    if (gdn::overlap(ry, r) || gdn::overlap(ro, r))
      return fail(GDN_ERR_INVALID_ARG, "the outputs must not overlap the inputs");
  if (gdn::overlap(ry, ro) || gdn::overlap(ry, rr) || (residual != residual_out && gdn::overlap(ro, rr)))
    return fail(GDN_ERR_INVALID_ARG,
                "the outputs must not overlap each other or the inputs (residual_out may be residual)");
  if (rows == 0) return GDN_OK;
  LnParams p{};
  p.x = x; p.w = w; p.b = b; p.residual = residual; p.y = y; p.residual_out = residual_out;
  p.rows = rows; p.x_stride = x_stride; p.D = D; p.eps = eps;
  cut(&p);
  p.whole = whole(p, elem);
  const cudaError_t e = gdn::launch_layer_norm(p, f32, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? GDN_OK : cuda_fail(e, "launching the layer norm");
}

size_t partial_bytes(long long rows, int D) {
  const long long most = gdn::ln_partials(D);
  return (size_t)(rows < most ? rows : most) * 2 * D * 4;
}

gdn_status backward(const void* dy, const void* x, const float* w, const void* dres, void* dx, float* dw, float* db,
                    long long rows, int D, long long dy_stride, long long x_stride, float eps, void* ws,
                    size_t ws_bytes, bool f32, gdn_stream_t stream) {
  const int elem = f32 ? 4 : 2;
  GDN_TRY(check(x, rows, D, x_stride, eps, elem));
  GDN_TRY(gdn::check_rows("dy", dy, rows, dy_stride, D, elem));
  if (rows > 0 && !dx) return fail(GDN_ERR_INVALID_ARG, "dx must be non-NULL");
  if ((dw == nullptr) != (db == nullptr)) return fail(GDN_ERR_INVALID_ARG, "dw and db go together");
  if (!aligned(w, 4) || !aligned(dw, 4) || !aligned(db, 4) || !aligned(dx, elem) || !aligned(dres, elem))
    return fail(GDN_ERR_INVALID_ARG, "misaligned pointer (each to its element size)");
  const gdn::Range rx = range_of(dx, rows * D, elem), rw = range_of(dw, D, 4), rb = range_of(db, D, 4),
                   rr = range_of(dres, rows * D, elem);
  for (const gdn::Range& r :
       {range_of(dy, rows, dy_stride, D, elem), range_of(x, rows, x_stride, D, elem), range_of(w, D, 4)})
    if (gdn::overlap(rx, r) || gdn::overlap(rw, r) || gdn::overlap(rb, r))
      return fail(GDN_ERR_INVALID_ARG, "the outputs must not overlap the inputs");
  if (gdn::overlap(rx, rw) || gdn::overlap(rx, rb) || gdn::overlap(rw, rb) || gdn::overlap(rw, rr) ||
      gdn::overlap(rb, rr) || (dx != dres && gdn::overlap(rx, rr)))
    return fail(GDN_ERR_INVALID_ARG, "the outputs must not overlap each other or the inputs (dx may be dres)");
  if (rows == 0 && !dw) return GDN_OK;
  LnParams p{};
  p.x = x; p.dy = dy; p.w = w; p.residual = dres; p.y = dx; p.dw = dw; p.db = db;
  p.rows = rows; p.x_stride = x_stride; p.dy_stride = dy_stride; p.D = D; p.eps = eps;
  cut(&p);
  p.whole = whole(p, elem);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t need = dw ? partial_bytes(rows, D) : 0;
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
  const cudaError_t e = gdn::launch_layer_norm_bwd(p, f32, st);
  const cudaError_t ef = pool ? cudaFreeAsync(pool, st) : cudaSuccess;
  if (e != cudaSuccess) return cuda_fail(e, "launching the layer norm's gradient");
  return ef == cudaSuccess ? GDN_OK : cuda_fail(ef, "freeing the workspace");
}

}  // namespace

extern "C" {

gdn_status gdn_layer_norm_fwd(const void* x, const float* w, const float* b, const void* residual, void* y,
                              void* residual_out, long long rows, int D, long long x_stride, float eps,
                              gdn_stream_t stream) {
  return forward(x, w, b, residual, y, residual_out, rows, D, x_stride, eps, false, stream);
}

gdn_status gdn_layer_norm_fwd_f32(const float* x, const float* w, const float* b, const float* residual, float* y,
                                  float* residual_out, long long rows, int D, long long x_stride, float eps,
                                  gdn_stream_t stream) {
  return forward(x, w, b, residual, y, residual_out, rows, D, x_stride, eps, true, stream);
}

size_t gdn_layer_norm_bwd_workspace_size(long long rows, int D) {
  return rows < 0 || D <= 0 || D > gdn::kLnMaxD ? 0 : partial_bytes(rows, D);
}

gdn_status gdn_layer_norm_bwd(const void* dy, const void* x, const float* w, const void* dres, void* dx, float* dw,
                              float* db, long long rows, int D, long long dy_stride, long long x_stride, float eps,
                              void* workspace, size_t workspace_bytes, gdn_stream_t stream) {
  return backward(dy, x, w, dres, dx, dw, db, rows, D, dy_stride, x_stride, eps, workspace, workspace_bytes, false,
                  stream);
}

gdn_status gdn_layer_norm_bwd_f32(const float* dy, const float* x, const float* w, const float* dres, float* dx,
                                  float* dw, float* db, long long rows, int D, long long dy_stride,
                                  long long x_stride, float eps, void* workspace, size_t workspace_bytes,
                                  gdn_stream_t stream) {
  return backward(dy, x, w, dres, dx, dw, db, rows, D, dy_stride, x_stride, eps, workspace, workspace_bytes, true,
                  stream);
}

}  // extern "C"
