// Host side of the C ABI declared in include/sbn_train.h: argument validation,
// workspace sizing and dispatch to the HIP launchers.  As in api.cpp, a
// rejected call launches nothing and touches no output.
#include <cmath>

#include "api_util.h"
#include "train_internal.h"

using namespace sbn;

namespace {

constexpr int64_t CE_LD_MAX = int64_t(1) << 22;   // row strides of X and W: 256 rows stay within 32-bit byte offsets
constexpr int64_t CE_T_MAX = int64_t(1) << 27;
constexpr int64_t CE_V_MAX = (int64_t(1) << 31) - 256;   // whole tiles of 256 entries end below 2^31
constexpr int64_t I32_MAX = (int64_t(1) << 31) - 1;

sbn_status check_float_dtype(const char* fn, const char* name, sbn_dtype d) {
  if (d != SBN_BF16 && d != SBN_F32)
    return fail(SBN_ERR_DTYPE, "%s: %s = %d must be SBN_BF16 or SBN_F32", fn, name, (int)d);
  return SBN_OK;
}

sbn_status check_head_grad_dtype(const char* fn, const char* name, sbn_dtype d) {
  if (d != SBN_BF16 && d != SBN_F32 && d != SBN_F32_FINE)
    return fail(SBN_ERR_DTYPE, "%s: %s = %d must be SBN_BF16, SBN_F32 or SBN_F32_FINE", fn, name, (int)d);
  return SBN_OK;
}

int bytes_of(sbn_dtype d) { return d == SBN_BF16 ? 2 : 4; }

// vectors that are read and written one element at a time
#define SBN_ELEM_ALIGNED(p, bytes)                                                                       \
  do {                                                                                                   \
    if ((uintptr_t)(p) & ((bytes) - 1))                                                                  \
      return fail(SBN_ERR_ALIGN, "%s: '%s' is not aligned to its %d-byte elements", fn, #p, (int)(bytes)); \
  } while (0)

sbn_status in_place(const char* fn, const char* out, const char* of) {
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

sbn_status check_t0(const char* fn, int64_t T) {
  if (T < 0) return fail(SBN_ERR_SHAPE, "%s: T = %lld is negative", fn, (long long)T);
  if (T > ROWS_MAX) return fail(SBN_ERR_SHAPE, "%s: T = %lld exceeds 2^40", fn, (long long)T);
  return SBN_OK;
}

sbn_status check_norm_shape(const char* fn, int64_t T, int64_t K) {
  SBN_TRY(check_t0(fn, T));
  if (K < 8 || K % 8 != 0 || K > SBN_RMSNORM_MAX_K)
    return fail(SBN_ERR_SHAPE, "%s: K = %lld must be a positive multiple of 8 and <= %d", fn, (long long)K,
                SBN_RMSNORM_MAX_K);
  if (T > 0) SBN_TRY(check_numel(fn, "X (T*K)", T, K));
  return SBN_OK;
}

// what the two forward forms share
sbn_status check_norm(const char* fn, const void* X, int64_t ldx, const void* residual, int64_t ldres, sbn_dtype dt,
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

sbn_status finite_norm(const char* fn, const void* X, int64_t ldx, const void* residual, int64_t ldres, sbn_dtype dt,
                       const void* gain, sbn_dtype gaindt, int64_t T, int64_t K, hipStream_t st) {
  SBN_TRY(check_finite(fn, "X", X, T, K, ldx, bytes_of(dt), st));
  if (residual) SBN_TRY(check_finite(fn, "residual", residual, T, K, ldres, bytes_of(dt), st));
  return check_finite(fn, "gain", gain, 1, K, K, bytes_of(gaindt), st);
}

sbn_status check_ce_shape(const char* fn, int64_t T, int64_t V, int64_t K) {
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

sbn_status check_ce(const char* fn, const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
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

sbn_status check_state_bits(const char* fn, int bits) {
  if (bits != 32 && bits != 8) return fail(SBN_ERR_DTYPE, "%s: state_bits = %d must be 32 or 8", fn, bits);
  return SBN_OK;
}

}  // namespace

extern "C" {

sbn_status sbn_rmsnorm(const void* X, int64_t ldx, const void* residual, int64_t ldres, sbn_dtype dt,
                       const void* gain, sbn_dtype gaindt, int64_t T, int64_t K, float eps, void* H, int64_t ldh,
                       void* Y, int64_t ldy, float* rstd, void* stream) {
  const char* fn = "sbn_rmsnorm";
  SBN_TRY(check_norm(fn, X, ldx, residual, ldres, dt, gain, gaindt, T, K, eps, H, ldh, rstd));
  if (T == 0) return ok();
  SBN_NONNULL(Y);
  SBN_TRY(check_ld("ldy", ldy, K, T));
  SBN_ALIGNED(Y);
  SBN_SAME_ROWS(Y, ldy, X, ldx);
  SBN_SAME_ROWS(Y, ldy, residual, ldres);
  if (residual) SBN_NOT_IN_PLACE(Y, H);
  hipStream_t st = (hipStream_t)stream;
  SBN_TRY(finite_norm(fn, X, ldx, residual, ldres, dt, gain, gaindt, T, K, st));
  return hip_result(launch_rmsnorm(X, ldx, residual, ldres, dt == SBN_F32, gain, gaindt == SBN_F32, T, K, eps, H, ldh,
                                   Y, ldy, nullptr, nullptr, rstd, st),
                    st, fn);
}

sbn_status sbn_rmsnorm_quant(const void* X, int64_t ldx, const void* residual, int64_t ldres, sbn_dtype dt,
                             const void* gain, sbn_dtype gaindt, int64_t T, int64_t K, float eps, void* H,
                             int64_t ldh, int8_t* Xq, float* s_x, float* rstd, void* stream) {
  const char* fn = "sbn_rmsnorm_quant";
  SBN_TRY(check_norm(fn, X, ldx, residual, ldres, dt, gain, gaindt, T, K, eps, H, ldh, rstd));
  if (T == 0) return ok();
  SBN_NONNULL(Xq);
  SBN_NONNULL(s_x);
  SBN_ALIGNED(Xq);
  SBN_ELEM_ALIGNED(s_x, 4);
  SBN_NOT_IN_PLACE(Xq, X);
  SBN_NOT_IN_PLACE(Xq, residual);
  if (residual) SBN_NOT_IN_PLACE(Xq, H);
  hipStream_t st = (hipStream_t)stream;
  SBN_TRY(finite_norm(fn, X, ldx, residual, ldres, dt, gain, gaindt, T, K, st));
  return hip_result(launch_rmsnorm(X, ldx, residual, ldres, dt == SBN_F32, gain, gaindt == SBN_F32, T, K, eps, H, ldh,
                                   nullptr, 0, Xq, s_x, rstd, st),
                    st, fn);
}

sbn_status sbn_rmsnorm_backward_workspace_bytes(int64_t T, int64_t K, size_t* bytes) {
  const char* fn = "sbn_rmsnorm_backward_workspace_bytes";
  SBN_NONNULL(bytes);
  SBN_TRY(check_norm_shape(fn, T, K));
  *bytes = rmsnorm_bwd_ws_bytes(T, K);
  return ok();
}

sbn_status sbn_rmsnorm_backward(const void* dY, int64_t lddy, const void* H, int64_t ldh, const void* dH,
                                int64_t lddh, sbn_dtype dt, const void* gain, sbn_dtype gaindt, const float* rstd,
                                int64_t T, int64_t K, void* dX, int64_t lddx, float* dgain, void* ws,
                                size_t ws_bytes, void* stream) {
  const char* fn = "sbn_rmsnorm_backward";
  SBN_TRY(check_norm_shape(fn, T, K));
  SBN_TRY(check_float_dtype(fn, "dt", dt));
  SBN_TRY(check_float_dtype(fn, "gaindt", gaindt));
  SBN_NONNULL(dgain);
  SBN_ALIGNED(dgain);
  hipStream_t st = (hipStream_t)stream;
  if (T > 0) {
    SBN_NONNULL(dY);
    SBN_NONNULL(H);
    SBN_NONNULL(gain);
    SBN_NONNULL(rstd);
    SBN_NONNULL(dX);
    SBN_NONNULL(ws);
    SBN_TRY(check_ld("lddy", lddy, K, T));
    SBN_TRY(check_ld("ldh", ldh, K, T));
    if (dH) SBN_TRY(check_ld("lddh", lddh, K, T));
    SBN_TRY(check_ld("lddx", lddx, K, T));
    SBN_ALIGNED(dY);
    SBN_ALIGNED(H);
    SBN_ALIGNED(dH);
    SBN_ALIGNED(gain);
    SBN_ELEM_ALIGNED(rstd, 4);
    SBN_ALIGNED(dX);
    SBN_ALIGNED(ws);
    SBN_SAME_ROWS(dX, lddx, dY, lddy);
    SBN_SAME_ROWS(dX, lddx, H, ldh);
    SBN_SAME_ROWS(dX, lddx, dH, lddh);
    const size_t need = rmsnorm_bwd_ws_bytes(T, K);
    if (ws_bytes < need)
      return fail(SBN_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, ws_bytes, need);
    SBN_TRY(check_finite(fn, "dY", dY, T, K, lddy, bytes_of(dt), st));
    SBN_TRY(check_finite(fn, "H", H, T, K, ldh, bytes_of(dt), st));
    if (dH) SBN_TRY(check_finite(fn, "dH", dH, T, K, lddh, bytes_of(dt), st));
    SBN_TRY(check_finite(fn, "gain", gain, 1, K, K, bytes_of(gaindt), st));
  }
  return hip_result(launch_rmsnorm_backward(dY, lddy, H, ldh, dH, lddh, dt == SBN_F32, gain, gaindt == SBN_F32, rstd,
                                            T, K, dX, lddx, dgain, ws, st),
                    st, fn);
}

sbn_status sbn_cross_entropy_workspace_bytes(int64_t T, int64_t V, int64_t K, size_t* bytes) {
  const char* fn = "sbn_cross_entropy_workspace_bytes";
  SBN_NONNULL(bytes);
  SBN_TRY(check_ce_shape(fn, T, V, K));
  *bytes = T > 0 ? ce_ws_bytes(T, V, K) : 0;
  return ok();
}

sbn_status sbn_cross_entropy(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, const void* labels,
                             int label_bytes, int64_t T, int64_t V, int64_t K, float* loss, float* lse, void* ws,
                             size_t ws_bytes, void* stream) {
  const char* fn = "sbn_cross_entropy";
  SBN_TRY(check_ce(fn, X, ldx, W, ldw, labels, label_bytes, T, V, K));
  if (T == 0) return ok();
  SBN_NONNULL(loss);
  SBN_NONNULL(lse);
  SBN_NONNULL(ws);
  SBN_ELEM_ALIGNED(loss, 4);
  SBN_ELEM_ALIGNED(lse, 4);
  SBN_ALIGNED(ws);
  const size_t need = ce_ws_bytes(T, V, K);
  if (ws_bytes < need) return fail(SBN_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, ws_bytes, need);
  hipStream_t st = (hipStream_t)stream;
  SBN_TRY(check_finite(fn, "X", X, T, K, ldx, 2, st));
  SBN_TRY(check_finite(fn, "W", W, V, K, ldw, 2, st));
  return hip_result(launch_ce(X, ldx, W, ldw, labels, label_bytes == 8, T, V, K, loss, lse, ws, st), st, fn);
}

sbn_status sbn_cross_entropy_backward_workspace_bytes(int64_t T, int64_t V, int64_t K, size_t* bytes) {
  const char* fn = "sbn_cross_entropy_backward_workspace_bytes";
  SBN_NONNULL(bytes);
  SBN_TRY(check_ce_shape(fn, T, V, K));
  const size_t one = T > 0 ? ce_bwd_ws_bytes(T, V, K, false) : 0, two = T > 0 ? ce_bwd_ws_bytes(T, V, K, true) : 0;
  *bytes = one > two ? one : two;
  return ok();
}

sbn_status sbn_cross_entropy_backward(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
                                      const void* labels, int label_bytes, const float* lse, const float* dloss,
                                      int64_t T, int64_t V, int64_t K, void* dX, sbn_dtype dxdt, int64_t lddx,
                                      void* dW, sbn_dtype dwdt, int64_t lddw, void* ws, size_t ws_bytes,
                                      void* stream) {
  const char* fn = "sbn_cross_entropy_backward";
  SBN_TRY(check_ce(fn, X, ldx, W, ldw, labels, label_bytes, T, V, K));
  SBN_TRY(check_head_grad_dtype(fn, "dxdt", dxdt));
  SBN_TRY(check_head_grad_dtype(fn, "dwdt", dwdt));
  if (dX && T > 0) SBN_TRY(check_ld("lddx", lddx, K, T));
  if (dW) SBN_TRY(check_ld("lddw", lddw, K, V));
  SBN_ALIGNED(dX);
  SBN_ALIGNED(dW);
  hipStream_t st = (hipStream_t)stream;
  if (T == 0) {
    if (!dW) return ok();
    return hip_result(launch_zero_rows(dW, V, K, lddw, bytes_of(dwdt), st), st, fn);
  }
  SBN_NONNULL(lse);
  SBN_NONNULL(dloss);
  SBN_NONNULL(ws);
  SBN_ELEM_ALIGNED(lse, 4);
  SBN_ELEM_ALIGNED(dloss, 4);
  SBN_ALIGNED(ws);
  const size_t need = ce_bwd_ws_bytes(T, V, K, (dX && dxdt == SBN_F32_FINE) || (dW && dwdt == SBN_F32_FINE));
  if (ws_bytes < need) return fail(SBN_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, ws_bytes, need);
  if (!dX && !dW) return ok();
  if (dW) SBN_NOT_IN_PLACE(dX, X);                   // which dW's product reads after dX's last
  SBN_NOT_IN_PLACE(dX, W);
  SBN_NOT_IN_PLACE(dW, X);
  if (dwdt != SBN_BF16 || lddw != ldw) SBN_NOT_IN_PLACE(dW, W);   // the same rows: a piece's are read before they are written
  SBN_NOT_IN_PLACE(dX, dW);
  SBN_TRY(check_finite(fn, "X", X, T, K, ldx, 2, st));
  SBN_TRY(check_finite(fn, "W", W, V, K, ldw, 2, st));
  SBN_TRY(check_finite_tokens(fn, "dloss", dloss, labels, label_bytes == 8, V, T, st));
  return hip_result(launch_ce_backward(X, ldx, W, ldw, labels, label_bytes == 8, lse, dloss, T, V, K, dX,
                                       dxdt, lddx, dW, dwdt, lddw, ws, st),
                    st, fn);
}

sbn_status sbn_adamw_plan(const sbn_adamw_entry* entries, int64_t count, sbn_dtype pdt, sbn_dtype gdt,
                          int state_bits, int32_t* map, int64_t* blocks) {
  const char* fn = "sbn_adamw_plan";
  SBN_NONNULL(blocks);
  SBN_TRY(check_float_dtype(fn, "pdt", pdt));
  SBN_TRY(check_float_dtype(fn, "gdt", gdt));
  SBN_TRY(check_state_bits(fn, state_bits));
  if (count < 0 || count > I32_MAX)
    return fail(SBN_ERR_SHAPE, "%s: count = %lld must be in [0, 2^31)", fn, (long long)count);
  if (count > 0) SBN_NONNULL(entries);
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) {
    const sbn_adamw_entry& e = entries[i];
    const long long at = (long long)i;
    if (e.n < 0 || e.n >= NUMEL_MAX)
      return fail(SBN_ERR_SHAPE, "%s: n = %lld must be in [0, 2^37) (entry %lld)", fn, (long long)e.n, at);
    if (!std::isfinite(e.weight_decay))
      return fail(SBN_ERR_VALUE, "%s: weight_decay is not finite (entry %lld)", fn, at);
    if (e.n > 0) {
      if (!e.p || !e.grad || !e.m || !e.v)
        return fail(SBN_ERR_NULL, "%s: p, grad, m or v is NULL (entry %lld)", fn, at);
      if (state_bits == 8 && (!e.m_scale || !e.v_scale))
        return fail(SBN_ERR_NULL, "%s: 8-bit states need m_scale and v_scale (entry %lld)", fn, at);
      if (e.shadow && pdt != SBN_F32)
        return fail(SBN_ERR_DTYPE, "%s: a bf16 shadow goes with float32 parameters only (entry %lld)", fn, at);
      if (!aligned16(e.p) || !aligned16(e.grad) || !aligned16(e.m) || !aligned16(e.v) || !aligned16(e.shadow) ||
          ((uintptr_t)e.m_scale & 3u) || ((uintptr_t)e.v_scale & 3u))
        return fail(SBN_ERR_ALIGN, "%s: a tensor is not 16-byte aligned, or a scale not 4-byte (entry %lld)", fn, at);
    }
    const int64_t nb = cdiv(e.n, ADAMW_CHUNK);
    if (map)
      for (int64_t b = 0; b < nb; ++b) {
        map[2 * (total + b)] = (int32_t)i;
        map[2 * (total + b) + 1] = (int32_t)b;
      }
    total += nb;
  }
  *blocks = total;
  return ok();
}

sbn_status sbn_adamw_step(const sbn_adamw_entry* entries, const int32_t* map, int64_t blocks, sbn_dtype pdt,
                          sbn_dtype gdt, int state_bits, double lr, double beta1, double beta2, double eps,
                          int64_t step, const float* dyn, void* stream) {
  const char* fn = "sbn_adamw_step";
  SBN_TRY(check_float_dtype(fn, "pdt", pdt));
  SBN_TRY(check_float_dtype(fn, "gdt", gdt));
  SBN_TRY(check_state_bits(fn, state_bits));
  if (!std::isfinite(lr)) return fail(SBN_ERR_VALUE, "%s: lr is not finite", fn);
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0))
    return fail(SBN_ERR_VALUE, "%s: beta1 and beta2 must be in [0, 1)", fn);
  if (!(eps >= 0.0) || std::isinf(eps)) return fail(SBN_ERR_VALUE, "%s: eps must be finite and >= 0", fn);
  if (state_bits == 8 && !((float)eps > 0.0f))
    return fail(SBN_ERR_VALUE, "%s: eps must be > 0 in float32 with 8-bit states", fn);
  if (step < 1) return fail(SBN_ERR_VALUE, "%s: step = %lld must be >= 1", fn, (long long)step);
  if (blocks < 0 || blocks >= NUMEL_MAX)
    return fail(SBN_ERR_SHAPE, "%s: blocks = %lld must be in [0, 2^37)", fn, (long long)blocks);
  if (blocks == 0) return ok();
  SBN_NONNULL(entries);
  SBN_NONNULL(map);
  SBN_ALIGNED(entries);
  SBN_ALIGNED(map);
  SBN_ALIGNED(dyn);
  AdamWScalars s;
  s.beta1 = (float)beta1, s.one_minus_beta1 = (float)(1.0 - beta1);
  s.beta2 = (float)beta2, s.one_minus_beta2 = (float)(1.0 - beta2);
  s.eps = (float)eps, s.lr = (float)lr;
  s.rate = s.lr / (float)(1.0 - std::pow(beta1, (double)step));
  s.rbias2 = 1.0f / std::sqrt((float)(1.0 - std::pow(beta2, (double)step)));
  hipStream_t st = (hipStream_t)stream;
  return hip_result(launch_adamw(entries, map, blocks, pdt == SBN_F32, gdt == SBN_F32, state_bits == 8, s, dyn, st),
                    st, fn);
}

sbn_status sbn_adamw_decode_state(const void* codes, const float* scale, int64_t n, int second, float* out,
                                  void* stream) {
  const char* fn = "sbn_adamw_decode_state";
  if (n < 0 || n >= NUMEL_MAX) return fail(SBN_ERR_SHAPE, "%s: n = %lld must be in [0, 2^37)", fn, (long long)n);
  if (n == 0) return ok();
  SBN_NONNULL(codes);
  SBN_NONNULL(scale);
  SBN_NONNULL(out);
  SBN_ALIGNED(codes);
  SBN_ALIGNED(out);
  hipStream_t st = (hipStream_t)stream;
  return hip_result(launch_adamw_decode(codes, scale, n, second != 0, out, st), st, fn);
}

sbn_status sbn_adamw_encode_state(const float* x, int64_t n, int second, void* codes, float* scale, void* stream) {
  const char* fn = "sbn_adamw_encode_state";
  if (n < 0 || n >= NUMEL_MAX) return fail(SBN_ERR_SHAPE, "%s: n = %lld must be in [0, 2^37)", fn, (long long)n);
  if (n == 0) return ok();
  SBN_NONNULL(x);
  SBN_NONNULL(codes);
  SBN_NONNULL(scale);
  SBN_ALIGNED(x);
  SBN_ALIGNED(codes);
  hipStream_t st = (hipStream_t)stream;
  return hip_result(launch_adamw_encode(x, n, second != 0, codes, scale, st), st, fn);
}

}  // extern "C"
