// Host side of the C ABI declared in include/sbn_score.h: argument validation,
// workspace sizing and dispatch to the HIP launchers.  A rejected call launches
// nothing and touches no output.
#include "score_internal.h"
#include "train_checks.h"

using namespace sbn;

namespace {

sbn_status check_scale(const char* fn, float scale) {
  if (!(scale >= 0x1p-20f && scale <= 0x1p20f)) return fail(SBN_ERR_VALUE, "%s: scale must be in [2^-20, 2^20]", fn);
  return SBN_OK;
}

sbn_status check_top(const char* fn, int top, int64_t V) {
  if (top < 0 || top > SBN_LOGPROBS_MAX_TOP || top > V)
    return fail(SBN_ERR_SHAPE, "%s: top = %d must be in [0, %d] and at most V", fn, top, SBN_LOGPROBS_MAX_TOP);
  return SBN_OK;
}

}  // namespace

extern "C" {

sbn_status sbn_token_logprobs_workspace_bytes(int64_t T, int64_t V, int64_t K, int top, size_t* bytes) {
  const char* fn = "sbn_token_logprobs_workspace_bytes";
  SBN_NONNULL(bytes);
  SBN_TRY(check_ce_shape(fn, T, V, K));
  SBN_TRY(check_top(fn, top, V));
  *bytes = T > 0 ? logprobs_ws_bytes(T, V, K, top) : 0;
  return ok();
}

sbn_status sbn_token_logprobs(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, const void* tokens,
                              int token_bytes, int64_t T, int64_t V, int64_t K, float scale, float* logp,
                              float* entropy, float* lse, int top, int64_t* top_ids, float* top_logp, void* ws,
                              size_t ws_bytes, void* stream) {
  const char* fn = "sbn_token_logprobs";
  // any address does for tokens that are not there
  SBN_TRY(check_ce(fn, X, ldx, W, ldw, tokens || logp ? tokens : X, token_bytes, T, V, K));
  SBN_TRY(check_scale(fn, scale));
  SBN_TRY(check_top(fn, top, V));
  if (T == 0) return ok();
  if (tokens) SBN_NONNULL(logp);
  SBN_NONNULL(lse);
  SBN_NONNULL(ws);
  SBN_ELEM_ALIGNED(logp, 4);
  SBN_ELEM_ALIGNED(entropy, 4);
  SBN_ELEM_ALIGNED(lse, 4);
  SBN_ALIGNED(ws);
  if (top) {
    SBN_NONNULL(top_ids);
    SBN_NONNULL(top_logp);
    SBN_ELEM_ALIGNED(top_ids, 8);
    SBN_ELEM_ALIGNED(top_logp, 4);
  }
  const size_t need = logprobs_ws_bytes(T, V, K, top);
  if (ws_bytes < need) return fail(SBN_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, ws_bytes, need);
  for (const void* out : {(const void*)logp, (const void*)entropy, (const void*)lse, (const void*)top_ids, (const void*)top_logp}) {
    SBN_NOT_IN_PLACE(out, X);
    SBN_NOT_IN_PLACE(out, W);
    SBN_NOT_IN_PLACE(out, tokens);
  }
  SBN_NOT_IN_PLACE(logp, lse);                       // lse is read by the alternatives
  SBN_NOT_IN_PLACE(entropy, lse);
  SBN_NOT_IN_PLACE(entropy, logp);
  hipStream_t st = (hipStream_t)stream;
  SBN_TRY(check_finite(fn, "X", X, T, K, ldx, 2, st));
  SBN_TRY(check_finite(fn, "W", W, V, K, ldw, 2, st));
  return hip_result(launch_logprobs(X, ldx, W, ldw, tokens, token_bytes == 8, T, V, K, scale, logp, entropy, lse, top,
                                    top_ids, top_logp, ws, st),
                    st, fn);
}

sbn_status sbn_token_logprobs_backward_workspace_bytes(int64_t T, int64_t V, int64_t K, size_t* bytes) {
  const char* fn = "sbn_token_logprobs_backward_workspace_bytes";
  SBN_NONNULL(bytes);
  SBN_TRY(check_ce_shape(fn, T, V, K));
  *bytes = 0;
  for (int fine = 0; fine < (T > 0 ? 4 : 0); ++fine) {
    const size_t b = policy_bwd_ws_bytes(T, V, K, fine & 1, fine & 2);
    if (b > *bytes) *bytes = b;
  }
  return ok();
}

sbn_status sbn_token_logprobs_backward(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
                                       const void* tokens, int token_bytes, float scale, const float* lse,
                                       const float* entropy, const float* dlogp, const float* dentropy, int64_t T,
                                       int64_t V, int64_t K, void* dX, sbn_dtype dxdt, int64_t lddx, void* dW,
                                       sbn_dtype dwdt, int64_t lddw, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "sbn_token_logprobs_backward";
  SBN_TRY(check_ce(fn, X, ldx, W, ldw, tokens || dlogp ? tokens : X, token_bytes, T, V, K));
  SBN_TRY(check_scale(fn, scale));
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
  SBN_NONNULL(ws);
  if (dentropy) SBN_NONNULL(entropy);
  SBN_ELEM_ALIGNED(lse, 4);
  SBN_ELEM_ALIGNED(entropy, 4);
  SBN_ELEM_ALIGNED(dlogp, 4);
  SBN_ELEM_ALIGNED(dentropy, 4);
  SBN_ALIGNED(ws);
  const size_t need = policy_bwd_ws_bytes(T, V, K, dX && dxdt == SBN_F32_FINE, dW && dwdt == SBN_F32_FINE);
  if (ws_bytes < need) return fail(SBN_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, ws_bytes, need);
  if (!dX && !dW) return ok();
  if (dW) SBN_NOT_IN_PLACE(dX, X);                   // which dW's product reads after dX's last
  SBN_NOT_IN_PLACE(dX, W);
  SBN_NOT_IN_PLACE(dW, X);
  if (dwdt != SBN_BF16 || lddw != ldw) SBN_NOT_IN_PLACE(dW, W);   // the same rows: a piece's are read before they are written
  SBN_NOT_IN_PLACE(dX, dW);
  SBN_TRY(check_finite(fn, "X", X, T, K, ldx, 2, st));
  SBN_TRY(check_finite(fn, "W", W, V, K, ldw, 2, st));
  if (dlogp) SBN_TRY(check_finite_tokens(fn, "dlogp", dlogp, tokens, token_bytes == 8, V, T, st));
  if (dentropy) SBN_TRY(check_finite_tokens(fn, "dentropy", dentropy, nullptr, false, V, T, st));
  HeadGrad H{tokens, token_bytes == 8, lse, dlogp};
  H.policy = true, H.scale = scale, H.entropy = entropy, H.dentropy = dentropy;
  return hip_result(launch_ce_backward(X, ldx, W, ldw, H, T, V, K, dX, dxdt, lddx, dW, dwdt, lddw, ws, st), st, fn);
}

}  // extern "C"
