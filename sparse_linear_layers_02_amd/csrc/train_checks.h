// Argument checks that the entry points of include/sbn_train.h share with those
// of include/sbn_keep.h and include/sbn_score.h.
#pragma once

#include <cmath>

#include "api_util.h"
#include "sbn_train.h"

namespace sbn {

constexpr int64_t CE_LD_MAX = int64_t(1) << 22;   // row strides of X and W: 256 rows stay within 32-bit byte offsets
constexpr int64_t CE_T_MAX = int64_t(1) << 27;
constexpr int64_t CE_V_MAX = (int64_t(1) << 31) - 256;   // whole tiles of 256 entries end below 2^31

inline sbn_status check_float_dtype(const char* fn, const char* name, sbn_dtype d) {
  if (d != SBN_BF16 && d != SBN_F32)
    return fail(SBN_ERR_DTYPE, "%s: %s = %d must be SBN_BF16 or SBN_F32", fn, name, (int)d);
  return SBN_OK;
}

inline sbn_status check_head_grad_dtype(const char* fn, const char* name, sbn_dtype d) {
  if (d != SBN_BF16 && d != SBN_F32 && d != SBN_F32_FINE)
    return fail(SBN_ERR_DTYPE, "%s: %s = %d must be SBN_BF16, SBN_F32 or SBN_F32_FINE", fn, name, (int)d);
  return SBN_OK;
}

inline int bytes_of(sbn_dtype d) { return d == SBN_BF16 ? 2 : 4; }

// vectors that are read and written one element at a time
#define SBN_ELEM_ALIGNED(p, bytes)                                                                       \
  do {                                                                                                   \
    if ((uintptr_t)(p) & ((bytes) - 1))                                                                  \
      return fail(SBN_ERR_ALIGN, "%s: '%s' is not aligned to its %d-byte elements", fn, #p, (int)(bytes)); \
  } while (0)

inline sbn_status in_place(const char* fn, const char* out, const char* of) {
  return fail(SBN_ERR_SHAPE, "%s: %s cannot be in the place of %s", fn, out, of);
}
// an output in the place of an input that is read row by row before it is written: with the same rows only
#define SBN_SAME_ROWS(out, ldout, in, ldin)                                                        \
  do {                                                                                             \
    if ((out) == (in) && (out) && (ldout) != (ldin)) return in_place(fn, #out, #in " with another row stride"); \
  } while (0)
#define SBN_NOT_IN_PLACE(out, other)                                                               \
  do {                                                                                             \
    if ((const void*)(out) == (const void*)(other) && (out)) return in_place(fn, #out, #other);    \
  } while (0)

inline sbn_status check_t0(const char* fn, int64_t T) {
  if (T < 0) return fail(SBN_ERR_SHAPE, "%s: T = %lld is negative", fn, (long long)T);
  if (T > ROWS_MAX) return fail(SBN_ERR_SHAPE, "%s: T = %lld exceeds 2^40", fn, (long long)T);
  return SBN_OK;
}

inline sbn_status check_norm_shape(const char* fn, int64_t T, int64_t K) {
  SBN_TRY(check_t0(fn, T));
  if (K < 8 || K % 8 != 0 || K > SBN_RMSNORM_MAX_K)
    return fail(SBN_ERR_SHAPE, "%s: K = %lld must be a positive multiple of 8 and <= %d", fn, (long long)K,
                SBN_RMSNORM_MAX_K);
  if (T > 0) SBN_TRY(check_numel(fn, "X (T*K)", T, K));
  return SBN_OK;
}

// what the forward forms of the norm share
inline sbn_status check_norm(const char* fn, const void* X, int64_t ldx, const void* residual, int64_t ldres, sbn_dtype dt,
                      const void* gain, sbn_dtype gaindt, int64_t T, int64_t K, float eps, void* H, int64_t ldh,
                      float* rstd) {
  SBN_TRY(check_norm_shape(fn, T, K));
  SBN_TRY(check_float_dtype(fn, "dt", dt));
  SBN_TRY(check_float_dtype(fn, "gaindt", gaindt));
  if (!(eps >= 0.0f) || std::isinf(eps)) return fail(SBN_ERR_VALUE, "%s: eps must be finite and >= 0", fn);
  if (T == 0) return SBN_OK;
  SBN_NONNULL(X);
  SBN_NONNULL(gain);
  SBN_TRY(check_ld("ldx", ldx, K, T));
  SBN_ALIGNED(X);
  SBN_ALIGNED(gain);
  SBN_ELEM_ALIGNED(rstd, 4);
  if (residual) {
    SBN_NONNULL(H);
    SBN_TRY(check_ld("ldres", ldres, K, T));
    SBN_TRY(check_ld("ldh", ldh, K, T));
    SBN_ALIGNED(residual);
    SBN_ALIGNED(H);
    if ((H == X && ldh != ldx) || (H == residual && ldh != ldres))
      return fail(SBN_ERR_SHAPE, "%s: H in the place of an input must have that input's row stride", fn);
  }
  return SBN_OK;
}

inline sbn_status finite_norm(const char* fn, const void* X, int64_t ldx, const void* residual, int64_t ldres, sbn_dtype dt,
                       const void* gain, sbn_dtype gaindt, int64_t T, int64_t K, hipStream_t st) {
  SBN_TRY(check_finite(fn, "X", X, T, K, ldx, bytes_of(dt), st));
  if (residual) SBN_TRY(check_finite(fn, "residual", residual, T, K, ldres, bytes_of(dt), st));
  return check_finite(fn, "gain", gain, 1, K, K, bytes_of(gaindt), st);
}

inline sbn_status check_ce_shape(const char* fn, int64_t T, int64_t V, int64_t K) {
  SBN_TRY(check_t0(fn, T));
  SBN_TRY(check_rows("V", V));
  SBN_TRY(check_k(K));
  if (V > CE_V_MAX) return fail(SBN_ERR_SHAPE, "%s: V = %lld must be <= 2^31 - 256", fn, (long long)V);
  SBN_TRY(check_numel(fn, "W (V*K)", V, K));
  if (T > 0) {
    SBN_TRY(check_numel(fn, "X (T*K)", T, K));
    // tiles are counted in 32 bits; the launches' grids stay below 2^32 threads
    if (T >= CE_T_MAX || !prod_below(cdiv(T, 64), cdiv(V, 128), int64_t(1) << 24))
      return fail(SBN_ERR_SHAPE, "%s: T = %lld with V = %lld exceeds the limits of one call", fn, (long long)T,
                  (long long)V);
  }
  return SBN_OK;
}

inline sbn_status check_ce(const char* fn, const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
                    const void* labels, int label_bytes, int64_t T, int64_t V, int64_t K) {
  SBN_TRY(check_ce_shape(fn, T, V, K));
  if (label_bytes != 4 && label_bytes != 8)
    return fail(SBN_ERR_DTYPE, "%s: label_bytes = %d must be 4 or 8", fn, label_bytes);
  if (T == 0) return SBN_OK;
  SBN_NONNULL(X);
  SBN_NONNULL(W);
  SBN_NONNULL(labels);
  SBN_TRY(check_ld("ldx", ldx, K, T));
  SBN_TRY(check_ld("ldw", ldw, K, V));
  if (ldx > CE_LD_MAX || ldw > CE_LD_MAX)
    return fail(SBN_ERR_SHAPE, "%s: ldx = %lld and ldw = %lld must be <= 2^22", fn, (long long)ldx, (long long)ldw);
  SBN_ALIGNED(X);
  SBN_ALIGNED(W);
  SBN_ELEM_ALIGNED(labels, label_bytes);
  return SBN_OK;
}

}  // namespace sbn
