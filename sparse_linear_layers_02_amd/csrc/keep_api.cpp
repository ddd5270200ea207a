// Host side of the C ABI declared in include/sbn_keep.h: argument validation,
// workspace sizing and dispatch to the HIP launchers.  A rejected call launches
// nothing and touches no output.
#include "keep_internal.h"
#include "train_checks.h"

using namespace sbn;

namespace {

sbn_status check_eps(const char* fn, float eps) {
  if (!(eps >= 0.0f) || std::isinf(eps)) return fail(SBN_ERR_VALUE, "%s: eps must be finite and >= 0", fn);
  return SBN_OK;
}

sbn_status check_act(const char* fn, sbn_act act) {
  if (act != SBN_RELU2 && act != SBN_SILU)
    return fail(SBN_ERR_VALUE, "%s: act = %d must be SBN_RELU2 or SBN_SILU", fn, (int)act);
  return SBN_OK;
}

// a checkpoint's two arrays
#define SBN_CHECKPOINT(codes, scales) \
  do {                                \
    SBN_NONNULL(codes);               \
    SBN_NONNULL(scales);              \
    SBN_ALIGNED(codes);               \
    SBN_ELEM_ALIGNED(scales, 4);      \
  } while (0)

}  // namespace

extern "C" {

sbn_status sbn_keep8_encode(const void* X, int64_t ldx, sbn_dtype dt, int64_t T, int64_t K, int8_t* codes,
                            float* scales, void* stream) {
  const char* fn = "sbn_keep8_encode";
  SBN_TRY(check_norm_shape(fn, T, K));
  SBN_TRY(check_float_dtype(fn, "dt", dt));
  if (T == 0) return ok();
  SBN_NONNULL(X);
  SBN_TRY(check_ld("ldx", ldx, K, T));
  SBN_ALIGNED(X);
  SBN_CHECKPOINT(codes, scales);
  SBN_NOT_IN_PLACE(codes, X);
  SBN_NOT_IN_PLACE(scales, X);
  SBN_NOT_IN_PLACE(scales, codes);
  hipStream_t st = (hipStream_t)stream;
  SBN_TRY(check_finite(fn, "X", X, T, K, ldx, bytes_of(dt), st));
  return hip_result(launch_keep8_encode(X, ldx, dt == SBN_F32, T, K, codes, scales, st), st, fn);
}

sbn_status sbn_keep8_decode(const int8_t* codes, const float* scales, int64_t T, int64_t K, void* Y, int64_t ldy,
                            sbn_dtype dt, void* stream) {
  const char* fn = "sbn_keep8_decode";
  SBN_TRY(check_norm_shape(fn, T, K));
  SBN_TRY(check_float_dtype(fn, "dt", dt));
  if (T == 0) return ok();
  SBN_CHECKPOINT(codes, scales);
  SBN_NONNULL(Y);
  SBN_TRY(check_ld("ldy", ldy, K, T));
  SBN_ALIGNED(Y);
  SBN_NOT_IN_PLACE(Y, codes);
  SBN_NOT_IN_PLACE(Y, scales);
  hipStream_t st = (hipStream_t)stream;
  return hip_result(launch_keep8_decode(codes, scales, T, K, Y, ldy, dt == SBN_F32, st), st, fn);
}

sbn_status sbn_rmsnorm_quant_keep(const void* X, int64_t ldx, const void* residual, int64_t ldres, sbn_dtype dt,
                                  const void* gain, sbn_dtype gaindt, int64_t T, int64_t K, float eps, void* H,
                                  int64_t ldh, int8_t* Xq, float* s_x, int8_t* codes, float* scales, void* stream) {
  const char* fn = "sbn_rmsnorm_quant_keep";
  SBN_TRY(check_norm(fn, X, ldx, residual, ldres, dt, gain, gaindt, T, K, eps, H, ldh, nullptr));
  if (T == 0) return ok();
  SBN_NONNULL(Xq);
  SBN_NONNULL(s_x);
  SBN_ALIGNED(Xq);
  SBN_ELEM_ALIGNED(s_x, 4);
  SBN_CHECKPOINT(codes, scales);
  for (const void* in : {X, residual, residual ? (const void*)H : nullptr}) {
    SBN_NOT_IN_PLACE(Xq, in);
    SBN_NOT_IN_PLACE(codes, in);
  }
  SBN_NOT_IN_PLACE(codes, Xq);
  SBN_NOT_IN_PLACE(scales, s_x);
  hipStream_t st = (hipStream_t)stream;
  SBN_TRY(finite_norm(fn, X, ldx, residual, ldres, dt, gain, gaindt, T, K, st));
  return hip_result(launch_rmsnorm_quant_keep(X, ldx, residual, ldres, dt == SBN_F32, gain, gaindt == SBN_F32, T, K, eps,
                                              H, ldh, Xq, s_x, codes, scales, st),
                    st, fn);
}

sbn_status sbn_rmsnorm_backward_kept_workspace_bytes(int64_t T, int64_t K, size_t* bytes) {
  const char* fn = "sbn_rmsnorm_backward_kept_workspace_bytes";
  SBN_NONNULL(bytes);
  SBN_TRY(check_norm_shape(fn, T, K));
  *bytes = kept_bwd_ws_bytes(T, K);
  return ok();
}

sbn_status sbn_rmsnorm_backward_kept(const void* dY, int64_t lddy, const void* dH, int64_t lddh, sbn_dtype dt,
                                     const int8_t* codes, const float* scales, const void* gain, sbn_dtype gaindt,
                                     int64_t T, int64_t K, float eps, void* dX, int64_t lddx, float* dgain, void* ws,
                                     size_t ws_bytes, void* stream) {
  const char* fn = "sbn_rmsnorm_backward_kept";
  SBN_TRY(check_norm_shape(fn, T, K));
  SBN_TRY(check_float_dtype(fn, "dt", dt));
  SBN_TRY(check_float_dtype(fn, "gaindt", gaindt));
  SBN_TRY(check_eps(fn, eps));
  SBN_NONNULL(dgain);
  SBN_ALIGNED(dgain);
  hipStream_t st = (hipStream_t)stream;
  if (T > 0) {
    SBN_NONNULL(dY);
    SBN_NONNULL(gain);
    SBN_NONNULL(dX);
    SBN_NONNULL(ws);
    SBN_CHECKPOINT(codes, scales);
    SBN_TRY(check_ld("lddy", lddy, K, T));
    if (dH) SBN_TRY(check_ld("lddh", lddh, K, T));
    SBN_TRY(check_ld("lddx", lddx, K, T));
    SBN_ALIGNED(dY);
    SBN_ALIGNED(dH);
    SBN_ALIGNED(gain);
    SBN_ALIGNED(dX);
    SBN_ALIGNED(ws);
    SBN_SAME_ROWS(dX, lddx, dY, lddy);
    SBN_SAME_ROWS(dX, lddx, dH, lddh);
    SBN_NOT_IN_PLACE(dX, codes);
    SBN_NOT_IN_PLACE(dX, scales);
    SBN_NOT_IN_PLACE(dX, gain);
    const size_t need = kept_bwd_ws_bytes(T, K);
    if (ws_bytes < need) return fail(SBN_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, ws_bytes, need);
    SBN_TRY(check_finite(fn, "dY", dY, T, K, lddy, bytes_of(dt), st));
    if (dH) SBN_TRY(check_finite(fn, "dH", dH, T, K, lddh, bytes_of(dt), st));
    SBN_TRY(check_finite(fn, "gain", gain, 1, K, K, bytes_of(gaindt), st));
  }
  return hip_result(launch_rmsnorm_backward_kept(dY, lddy, dH, lddh, dt == SBN_F32, codes, scales, gain,
                                                 gaindt == SBN_F32, T, K, eps, dX, lddx, dgain, ws, st),
                    st, fn);
}

sbn_status sbn_activation_quant(const void* A, int64_t lda, const void* B, int64_t ldb, sbn_dtype dt, sbn_act act,
                                const void* gain, sbn_dtype gaindt, int64_t T, int64_t K, float eps, int8_t* Xq,
                                float* s_x, int8_t* codes_a, float* scales_a, int8_t* codes_b, float* scales_b,
                                void* stream) {
  const char* fn = "sbn_activation_quant";
  SBN_TRY(check_norm_shape(fn, T, K));
  SBN_TRY(check_float_dtype(fn, "dt", dt));
  SBN_TRY(check_act(fn, act));
  if (gain) SBN_TRY(check_float_dtype(fn, "gaindt", gaindt));
  SBN_TRY(check_eps(fn, eps));
  if (T == 0) return ok();
  SBN_NONNULL(A);
  SBN_NONNULL(Xq);
  SBN_NONNULL(s_x);
  SBN_TRY(check_ld("lda", lda, K, T));
  if (B) SBN_TRY(check_ld("ldb", ldb, K, T));
  SBN_ALIGNED(A);
  SBN_ALIGNED(B);
  SBN_ALIGNED(gain);
  SBN_ALIGNED(Xq);
  SBN_ELEM_ALIGNED(s_x, 4);
  if (codes_a || scales_a || codes_b || scales_b) {
    SBN_CHECKPOINT(codes_a, scales_a);
    if (B) SBN_CHECKPOINT(codes_b, scales_b);
    else if (codes_b || scales_b)
      return fail(SBN_ERR_NULL, "%s: a checkpoint of B without B", fn);
  }
  for (const void* in : {A, B}) {
    SBN_NOT_IN_PLACE(Xq, in);
    SBN_NOT_IN_PLACE(codes_a, in);
    SBN_NOT_IN_PLACE(codes_b, in);
  }
  SBN_NOT_IN_PLACE(codes_a, Xq);
  SBN_NOT_IN_PLACE(codes_b, Xq);
  SBN_NOT_IN_PLACE(codes_b, codes_a);
  SBN_NOT_IN_PLACE(scales_a, s_x);
  SBN_NOT_IN_PLACE(scales_b, s_x);
  SBN_NOT_IN_PLACE(scales_b, scales_a);
  hipStream_t st = (hipStream_t)stream;
  SBN_TRY(check_finite(fn, "A", A, T, K, lda, bytes_of(dt), st));
  if (B) SBN_TRY(check_finite(fn, "B", B, T, K, ldb, bytes_of(dt), st));
  if (gain) SBN_TRY(check_finite(fn, "gain", gain, 1, K, K, bytes_of(gaindt), st));
  return hip_result(launch_activation_quant(A, lda, B, ldb, dt == SBN_F32, act, gain, gaindt == SBN_F32, T, K, eps, Xq,
                                            s_x, codes_a, scales_a, codes_b, scales_b, st),
                    st, fn);
}

sbn_status sbn_activation_backward_workspace_bytes(int64_t T, int64_t K, size_t* bytes) {
  const char* fn = "sbn_activation_backward_workspace_bytes";
  SBN_NONNULL(bytes);
  SBN_TRY(check_norm_shape(fn, T, K));
  *bytes = kept_bwd_ws_bytes(T, K);
  return ok();
}

sbn_status sbn_activation_backward(const void* dY, int64_t lddy, sbn_dtype dt, const int8_t* codes_a,
                                   const float* scales_a, const int8_t* codes_b, const float* scales_b, sbn_act act,
                                   const void* gain, sbn_dtype gaindt, int64_t T, int64_t K, float eps, void* dA,
                                   int64_t ldda, void* dB, int64_t lddb, float* dgain, void* ws, size_t ws_bytes,
                                   void* stream) {
  const char* fn = "sbn_activation_backward";
  SBN_TRY(check_norm_shape(fn, T, K));
  SBN_TRY(check_float_dtype(fn, "dt", dt));
  SBN_TRY(check_act(fn, act));
  SBN_TRY(check_eps(fn, eps));
  if (dgain) {
    SBN_TRY(check_float_dtype(fn, "gaindt", gaindt));
    SBN_ALIGNED(dgain);
    if (T > 0) SBN_NONNULL(gain);
  } else if (gain) {
    return fail(SBN_ERR_NULL, "%s: dgain is NULL, with a gain", fn);
  }
  if (T == 0 && !dgain) return ok();
  hipStream_t st = (hipStream_t)stream;
  if (T > 0) {
    SBN_NONNULL(dY);
    SBN_NONNULL(dA);
    SBN_CHECKPOINT(codes_a, scales_a);
    if (codes_b || scales_b || dB) {
      SBN_CHECKPOINT(codes_b, scales_b);
      SBN_NONNULL(dB);
      SBN_TRY(check_ld("lddb", lddb, K, T));
      SBN_ALIGNED(dB);
    }
    SBN_TRY(check_ld("lddy", lddy, K, T));
    SBN_TRY(check_ld("ldda", ldda, K, T));
    SBN_ALIGNED(dY);
    SBN_ALIGNED(dA);
    SBN_ALIGNED(gain);
    SBN_SAME_ROWS(dA, ldda, dY, lddy);
    SBN_SAME_ROWS(dB, lddb, dY, lddy);
    SBN_NOT_IN_PLACE(dB, dA);
    for (const void* in : {(const void*)codes_a, (const void*)scales_a, (const void*)codes_b, (const void*)scales_b, gain}) {
      SBN_NOT_IN_PLACE(dA, in);
      SBN_NOT_IN_PLACE(dB, in);
    }
    if (gain) {
      SBN_NONNULL(ws);
      SBN_ALIGNED(ws);
      const size_t need = kept_bwd_ws_bytes(T, K);
      if (ws_bytes < need) return fail(SBN_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, ws_bytes, need);
    }
    SBN_TRY(check_finite(fn, "dY", dY, T, K, lddy, bytes_of(dt), st));
    if (gain) SBN_TRY(check_finite(fn, "gain", gain, 1, K, K, bytes_of(gaindt), st));
  }
  return hip_result(launch_activation_backward(dY, lddy, dt == SBN_F32, codes_a, scales_a, codes_b, scales_b, act, gain,
                                               gaindt == SBN_F32, T, K, eps, dA, ldda, dB, lddb, dgain, ws, st),
                    st, fn);
}

}  // extern "C"
