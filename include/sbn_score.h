/*
 * sbn_score.h -- C ABI of the output head as a distribution over tokens, for AMD
 * Instinct MI355X (gfx950): log probabilities of given tokens, the entropy of each
 * distribution, its most likely tokens, and the gradients of the first two.  The
 * logits are never in memory as a whole, as with sbn_cross_entropy.
 *
 * The conventions of sbn.h and sbn_train.h hold: device pointers owned by the
 * caller and 16-byte aligned (vectors with an element per token, and the top
 * alternatives: aligned to their elements), row-major tensors with leading
 * dimensions in elements and multiples of 8, work enqueued on `stream`, arguments
 * checked on the host before anything is launched, nothing launched on an error,
 * messages from sbn_last_error(), no allocation, no synchronisation, no exception
 * across the ABI.  Tensors that a call writes overlap no other tensor of the call,
 * except where it says that one may be in another's place.  Every call may be
 * captured into a HIP graph.  Results do not depend on launch geometry from run to
 * run.  Inputs with NaN or Inf are outside the contract; with SBN_CHECK_FINITE=1 the
 * calls scan X, W, dentropy, and dlogp (of the rows with a token).
 */
#ifndef SBN_SCORE_H
#define SBN_SCORE_H

#include "sbn_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 *   l[t,v]     = scale * sum_k X[t,k] * W[v,k]            (float32, not kept)
 *   lse[t]     = log sum_v exp(l[t,v])
 *   logp[t]    = l[t, tokens[t]] - lse[t], 0 where tokens[t] is outside [0, V)
 *   entropy[t] = -sum_v p log p,  p = exp(l[t,v] - lse[t])
 *   top_ids[t,:], top_logp[t,:]   the `top` largest l[t,v] - lse[t], largest first,
 *                 equal ones by their index
 * scale is the inverse of a sampling temperature.  A token outside [0, V), such as
 * -100, marks a row without one; its distribution is there all the same.
 *
 * logp and top_logp are at most 0 and entropy at least 0, and near 0 they keep float32's
 * relative precision: they are formed from differences to the row's largest logit, not from
 * lse.  (The logits themselves are float32 sums, and those of top_logp 64-bit ones.)
 *
 * The order of the alternatives is that of sums in 64 bits: float32 sums only
 * choose who is compared, with a margin of their worst error (K 2^-23 |X[t]| |W[v]|, the
 * norms' product being no less than sum_k |X W|, with the largest |W[v]| of a group of 32 to 128
 * entries), so rows of W whose logits agree to float32's precision, and rows of any
 * size whose large parts cancel, are still told apart.  (Products |X W| below 2^-134, which
 * float32 does not hold exactly, count as rounded to multiples of 2^-149.)
 * Every logit within that margin of the last alternative is summed again: a row
 * whose logits are all equal takes as long as 64-bit sums of all of them (4096 rows
 * of 65536 equal logits, K = 2560: 0.2 s; rows of X that are zero, such as padding, none),
 * and a row of W far larger than the others costs the sums of its group.
 *
 *   X [T x K], W [V x K] bf16, row strides ldx, ldw     as sbn_cross_entropy
 *   tokens  [T] int64 (token_bytes = 8) or int32 (4); or NULL with logp NULL
 *   logp, lse [T] float; entropy [T] float or NULL                       (out)
 *   top     0 .. min(V, SBN_LOGPROBS_MAX_TOP); with 0 top_ids and top_logp may be NULL
 *   top_ids [T x top] int64, top_logp [T x top] float, contiguous        (out)
 *   ws      sbn_token_logprobs_workspace_bytes(T, V, K, top) bytes, no initialisation:
 *           V / 10 to 3 V / 8 bytes a token, with alternatives V / 4 to V more, as far as 4 GiB
 *           (512 MiB for V more); of more tokens it is used for one part after the other
 * 2^-20 <= scale <= 2^20; |l| < 2^30.  Limits of T, V and K as for sbn_cross_entropy
 * (T = 0: nothing to do).
 */
#define SBN_LOGPROBS_MAX_TOP 64

sbn_status sbn_token_logprobs_workspace_bytes(int64_t T, int64_t V, int64_t K, int top, size_t* bytes);
sbn_status sbn_token_logprobs(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, const void* tokens,
                              int token_bytes, int64_t T, int64_t V, int64_t K, float scale, float* logp,
                              float* entropy, float* lse, int top, int64_t* top_ids, float* top_logp, void* ws,
                              size_t ws_bytes, void* stream);

/*
 * Gradients of X and W from the forward's lse and entropy, and the gradients of
 * logp and of entropy per row:
 *   D[t,v] = dlogp[t] * ([v == tokens[t]] - p) - dentropy[t] * p * (log p + entropy[t])
 *   dX = scale * D * W       dW = scale * D^T * X       (float32 sums)
 * Where tokens[t] is outside [0, V) dlogp[t] counts as 0, whatever it holds; where
 * both are 0 the row gives nothing, whatever lse and entropy hold (its row of X has
 * to be finite).  D is held in bf16, as by sbn_cross_entropy_backward, or in two bf16
 * numbers for a gradient of type SBN_F32_FINE and, for any type, of up to 128 tokens.
 *
 *   dlogp, dentropy  [T] float; either NULL for zeros.  tokens NULL: dlogp is NULL.
 *                    entropy may be NULL with dentropy.
 *   dX [T x K] of dtype dxdt, dW [V x K] of dtype dwdt (SBN_BF16, SBN_F32 or
 *   SBN_F32_FINE); either may be NULL.  With T = 0 dW is written as zeros.  dX
 *   without dW may be in X's place, dW of bf16 in W's (same stride).
 *   ws sbn_token_logprobs_backward_workspace_bytes(T, V, K) bytes, for any types
 */
sbn_status sbn_token_logprobs_backward_workspace_bytes(int64_t T, int64_t V, int64_t K, size_t* bytes);
sbn_status sbn_token_logprobs_backward(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
                                       const void* tokens, int token_bytes, float scale, const float* lse,
                                       const float* entropy, const float* dlogp, const float* dentropy, int64_t T,
                                       int64_t V, int64_t K, void* dX, sbn_dtype dxdt, int64_t lddx, void* dW,
                                       sbn_dtype dwdt, int64_t lddw, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SBN_SCORE_H */
