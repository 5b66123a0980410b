// layer_check.h - checks that the layer operators' C entry points share.
#pragma once

#include "abi_common.h"

namespace gdn {

constexpr long long kMaxGrid = 0x7fffffffll;

// Bytes from `base` that `rows` rows of `cols` elements, `stride` elements apart, span.
struct Range {
  uintptr_t begin, end;
};
inline Range range_of(const void* base, long long rows, long long stride, long long cols, int elem) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(base);
  if (!base || rows <= 0 || cols <= 0) return {b, b};
  return {b, b + (uintptr_t)((rows - 1) * stride + cols) * (uintptr_t)elem};
}
inline Range range_of(const void* base, long long count, int elem) {
  return range_of(base, 1, 0, count, elem);
}
inline bool overlap(const Range& a, const Range& b) { return a.begin < b.end && b.begin < a.end; }

// The sizes every prompt call shares: N sequences (rows of T tokens, or one packed row).
inline gdn_status check_tokens(int N, int T, int D, const int32_t* cu, long long* tokens) {
  if (N < 0 || T < 0) return fail(GDN_ERR_INVALID_ARG, "N=%d and T=%d must be >= 0", N, T);
  if (D <= 0) return fail(GDN_ERR_INVALID_ARG, "%d channels: must be > 0", D);
  if (cu && N < 1) return fail(GDN_ERR_INVALID_ARG, "cu_seqlens needs N >= 1 sequences");
  if (!aligned(cu, 4)) return fail(GDN_ERR_INVALID_ARG, "cu_seqlens must be 4-byte aligned");
  *tokens = cu ? (long long)T : (long long)N * T;
  if (*tokens > (1ll << 36) || (long long)N * D > (1ll << 40))
    return fail(GDN_ERR_INVALID_ARG, "problem too large: N=%d T=%d D=%d", N, T, D);
  return GDN_OK;
}

// A strided row operand: element alignment, and rows that do not run into each other.
inline gdn_status check_rows(const char* name, const void* p, long long rows, long long stride, int cols,
                      int elem) {
  if (rows > 0 && !p) return fail(GDN_ERR_INVALID_ARG, "%s must be non-NULL", name);
  if (!aligned(p, elem)) return fail(GDN_ERR_INVALID_ARG, "%s must be %d-byte aligned", name, elem);
  if (rows > 1 && (stride < cols || stride > (1ll << 31)))
    return fail(GDN_ERR_INVALID_ARG, "%s: %lld elements from token to token, rows have %d", name,
                stride, cols);
  return GDN_OK;
}

#define GDN_TRY(expr)                  \
  do {                                 \
    const gdn_status s_ = (expr);      \
    if (s_ != GDN_OK) return s_;       \
  } while (0)

// Whether rows of strided operands meet.  Rows the same number of bytes apart may lie between each
// other, as slices of one projection do.
struct Strided {
  const void* p;
  long long rows, stride;
  long long cols;
  int elem;
};
inline bool overlap(const Strided& a, const Strided& b) {
  if (!overlap(range_of(a.p, a.rows, a.stride, a.cols, a.elem), range_of(b.p, b.rows, b.stride, b.cols, b.elem)))
    return false;
  const long long apart = a.stride * a.elem, wa = a.cols * a.elem, wb = b.cols * b.elem;
  if (a.rows < 2 || b.rows < 2 || apart != b.stride * b.elem || wa + wb > apart) return true;
  long long off = (long long)(reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p)) % apart;
  if (off < 0) off += apart;
  return off < wa || off + wb > apart;
}

}  // namespace gdn
