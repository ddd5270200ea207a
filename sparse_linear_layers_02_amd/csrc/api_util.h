// Host-side helpers of the C entry points, shared by the translation units
// that implement include/sbn.h and include/sbn_train.h: status and message of
// the calling thread, argument checks, launch results.
#pragma once

#include "sbn_internal.h"

namespace sbn {

// Records the message sbn_last_error() returns on this thread; returns `s`.
sbn_status fail(sbn_status s, const char* fmt, ...);
// Clears this thread's message; returns SBN_OK.
sbn_status ok();
// SBN_CHECK_FINITE=1: SBN_ERR_VALUE if `x` holds a NaN or Inf (see sbn.h).
sbn_status check_finite(const char* fn, const char* what, const void* x, int64_t rows, int64_t cols, int64_t ld,
                        int elem_bytes, hipStream_t st);
// The same for a value per token, of the tokens whose label is in [0, V) (labels NULL: all).
sbn_status check_finite_tokens(const char* fn, const char* what, const float* x, const void* labels, bool labels64,
                               int64_t V, int64_t T, hipStream_t st);
// The status of the launches of one entry point.
sbn_status hip_result(hipError_t e, hipStream_t st, const char* what);

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

constexpr int64_t K_MAX = int64_t(1) << 18;
constexpr int64_t NUMEL_MAX = int64_t(1) << 37;   // elements of W, Xq, dX, dW
constexpr int64_t ROWS_MAX = int64_t(1) << 40;    // any T or R (so that R*K, T*K fit in int64)
constexpr int64_t SPAN_MAX = int64_t(1) << 40;    // rows times a leading dimension (Y, X, W, dY)

// a * b < limit for 1 <= a, b, decided without forming the product
inline bool prod_below(int64_t a, int64_t b, int64_t limit) { return a <= (limit - 1) / b; }

inline sbn_status check_k(int64_t K) {
  if (K < 64 || K % 64 != 0 || K > K_MAX)
    return fail(SBN_ERR_SHAPE, "K = %lld must be a positive multiple of 64 and <= 2^18", (long long)K);
  return SBN_OK;
}

inline sbn_status check_rows(const char* name, int64_t v) {
  if (v < 1) return fail(SBN_ERR_SHAPE, "%s = %lld must be >= 1", name, (long long)v);
  if (v > ROWS_MAX) return fail(SBN_ERR_SHAPE, "%s = %lld exceeds 2^40", name, (long long)v);
  return SBN_OK;
}

// rows x K elements (rows and K already checked): below NUMEL_MAX
inline sbn_status check_numel(const char* fn, const char* what, int64_t rows, int64_t K) {
  if (!prod_below(rows, K, NUMEL_MAX)) return fail(SBN_ERR_SHAPE, "%s: %s has 2^37 elements or more", fn, what);
  return SBN_OK;
}

// a leading dimension of `len` elements per row, for `rows` rows (rows already checked)
inline sbn_status check_ld(const char* name, int64_t ld, int64_t len, int64_t rows = 1) {
  if (ld < len) return fail(SBN_ERR_SHAPE, "%s = %lld is smaller than the row length %lld", name, (long long)ld, (long long)len);
  if (ld % 8 != 0) return fail(SBN_ERR_ALIGN, "%s = %lld is not a multiple of 8", name, (long long)ld);
  if (!prod_below(rows, ld, SPAN_MAX))
    return fail(SBN_ERR_SHAPE, "%s = %lld times %lld rows reaches 2^40 elements", name, (long long)ld, (long long)rows);
  return SBN_OK;
}

}  // namespace sbn

#define SBN_TRY(expr)                 \
  do {                                \
    const sbn_status s_ = (expr);     \
    if (s_ != SBN_OK) return s_;      \
  } while (0)

#define SBN_NONNULL(p)                                                        \
  do {                                                                        \
    if (!(p)) return fail(SBN_ERR_NULL, "%s: argument '%s' is NULL", fn, #p); \
  } while (0)

#define SBN_ALIGNED(p)                                                                         \
  do {                                                                                         \
    if ((p) && !aligned16(p)) return fail(SBN_ERR_ALIGN, "%s: '%s' is not 16-byte aligned", fn, #p); \
  } while (0)
