/*
 * sbn_train.h -- C ABI of the operators a training or decoding step needs
 * around the Sparse-BitLinear layer of sbn.h, for AMD Instinct MI355X (gfx950):
 *
 *   RMS norm        the norm in front of the layer, with the residual's
 *                   addition and the layer's 8-bit activations as its output,
 *                   and its gradient;
 *   cross entropy   the loss of the output head over a large vocabulary from
 *                   the hidden states and the head's weights, in pieces of
 *                   the vocabulary, without keeping the logits, and its
 *                   gradients;
 *   AdamW           one optimizer step over many tensors in one launch, with
 *                   states in 32 or in 8 bits.
 *
 * The conventions of sbn.h hold: device pointers owned by the caller and
 * 16-byte aligned (rstd, s_x, labels, loss, lse and dloss: aligned to their
 * elements), row-major tensors with leading dimensions in elements and multiples
 * of 8, work enqueued on `stream`, arguments checked on the host
 * before anything is launched, nothing launched on an error, messages from
 * sbn_last_error(), no allocation, no synchronisation, no exception across the
 * ABI.  Tensors that a call writes overlap no other tensor of the call, except
 * where it says that one may be in another's place.  Every call may be captured
 * into a HIP graph.  Results do not depend on launch geometry from run to run:
 * there are no atomics, every sum has a fixed order.  Inputs with NaN or Inf are outside the contract; with
 * SBN_CHECK_FINITE=1 the norm and cross entropy calls scan X, residual, gain,
 * W, dY, H, dH and dloss (of the tokens with a target) as sbn.h describes.
 */
#ifndef SBN_TRAIN_H
#define SBN_TRAIN_H

#include "sbn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ RMS norm
 *
 *   h[t,k]  = x[t,k] + residual[t,k], rounded to the tensors' type
 *             (h = x without a residual)
 *   rstd[t] = 1 / sqrt(mean_k h[t,k]^2 + eps)                      (float32)
 *   y[t,k]  = h[t,k] * rstd[t] * gain[k], rounded to the tensors' type
 *
 * The stored h is what is normalised: the backward, which is given h, then
 * differentiates the function that the forward computed.  Sums are float32.
 *
 *   X, residual, H, Y   [T x K] of dtype dt (SBN_BF16 or SBN_F32), row strides
 *                       ldx, ldres, ldh, ldy >= K
 *   gain                [K] of dtype gaindt (SBN_BF16 or SBN_F32)
 *   rstd                [T] float, or NULL if the backward is not needed
 *
 * residual may be NULL (then H is not written and may be NULL).  With a
 * residual H is required; it may be X or residual itself (same row stride),
 * and so may Y, but not both in one place.
 * K is a multiple of 8 and at most 32768; T >= 0 (T = 0: nothing to do, and
 * pointers may be NULL); T*K < 2^37.  eps >= 0 and finite; with eps = 0 a row
 * of zeros has no norm (rstd and s_x are Inf, y is NaN, codes are 0).  The sum
 * of a row's squares has to stay below 2^128, which holds for all
 * |h| <= 2^56 in a row of 32768; squares of |h| < 2^-75 count as 0.
 */
#define SBN_RMSNORM_MAX_K 32768

sbn_status sbn_rmsnorm(const void* X, int64_t ldx, const void* residual, int64_t ldres, sbn_dtype dt,
                       const void* gain, sbn_dtype gaindt, int64_t T, int64_t K, float eps,
                       void* H, int64_t ldh, void* Y, int64_t ldy, float* rstd, void* stream);

/*
 * The same norm with the layer's activations as the output: per token absmax
 * int8, the input of sbn_sparse_ternary_gemm and _gemv.  With u = h * gain
 * (float32, one rounding) and a = max(max_k |u|, 2^-100):
 *   Xq[t,k] = rint((127 * u) / a)     round half to even, in [-127, 127]
 *   s_x[t]  = (a * rstd[t]) / 127
 * so Xq * s_x stands for the normalised row.  rstd scales a whole row and
 * cancels from the codes, so they do not depend on the order of the sum of
 * squares.  (sbn_act_quant of a stored Y differs by Y's own rounding and by
 * its floor of 1e-5 under the row's maximum; a row of zeros gives codes 0
 * here as there.)
 *
 *   Xq   [T x K] int8, contiguous      s_x   [T] float
 */
sbn_status sbn_rmsnorm_quant(const void* X, int64_t ldx, const void* residual, int64_t ldres, sbn_dtype dt,
                             const void* gain, sbn_dtype gaindt, int64_t T, int64_t K, float eps,
                             void* H, int64_t ldh, int8_t* Xq, float* s_x, float* rstd, void* stream);

/*
 * Gradient of both forms (the 8-bit form's quantizer is passed straight
 * through, as in sbn_backward).  With n = h * rstd and w = gain * dY:
 *   dX[t,k]  = rstd[t] * (w[t,k] - n[t,k] * mean_k(w[t,:] * n[t,:])) + dH[t,k]
 *   dgain[k] = sum_t dY[t,k] * n[t,k]
 * dX is the gradient of x and of the residual alike.  dH (NULL for none) is
 * the gradient that reaches h along the residual stream.
 *
 *   dY, H, dH, dX  [T x K] of dtype dt; dX may be dY, H or dH itself (same stride)
 *   gain [K] of dtype gaindt, rstd [T] float
 *   dgain [K] float, always written (T = 0: zeros)
 *   ws    sbn_rmsnorm_backward_workspace_bytes(T, K) bytes, no initialisation
 */
sbn_status sbn_rmsnorm_backward_workspace_bytes(int64_t T, int64_t K, size_t* bytes);
sbn_status sbn_rmsnorm_backward(const void* dY, int64_t lddy, const void* H, int64_t ldh, const void* dH,
                                int64_t lddh, sbn_dtype dt, const void* gain, sbn_dtype gaindt,
                                const float* rstd, int64_t T, int64_t K, void* dX, int64_t lddx, float* dgain,
                                void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ cross entropy of the output head
 *
 *   l[t,v]  = sum_k X[t,k] * W[v,k]                       (float32, not kept)
 *   lse[t]  = log sum_v exp(l[t,v])
 *   loss[t] = lse[t] - l[t, labels[t]], 0 where labels[t] is outside [0, V)
 * A label outside [0, V), such as -100, marks a token without a target.  What
 * dloss and lse hold for it does not matter; its row of X has to be finite.
 *
 *   X      [T x K] bf16, row stride ldx >= K     hidden states
 *   W      [V x K] bf16, row stride ldw >= K     the head's weights
 *   labels [T] int64 (label_bytes = 8) or int32 (4)
 *   loss, lse  [T] float                                            (out)
 *   ws     sbn_cross_entropy_workspace_bytes(T, V, K) bytes, no initialisation
 * K is a multiple of 64 (as the layer's); 0 <= T < 2^27, 1 <= V <= 2^31 - 256;
 * T*K and V*K < 2^37, ceil(T/64) * ceil(V/128) < 2^24; ldx, ldw <= 2^22.
 */
sbn_status sbn_cross_entropy_workspace_bytes(int64_t T, int64_t V, int64_t K, size_t* bytes);
sbn_status sbn_cross_entropy(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, const void* labels,
                             int label_bytes, int64_t T, int64_t V, int64_t K, float* loss, float* lse, void* ws,
                             size_t ws_bytes, void* stream);

/*
 * Its gradients, from the lse of the forward and the gradient of each token's
 * loss (1/T for the mean over T tokens):
 *   D[t,v] = dloss[t] * (exp(l[t,v] - lse[t]) - [v == labels[t]])
 *            (0 where the label is outside [0, V)), rounded to bf16
 *   dX = D * W       dW = D^T * X       (float32 sums)
 * D exists for one piece of the vocabulary at a time, in the workspace: the
 * logits are computed again, piece by piece.  Rounding D to bf16 puts it
 * through the bf16 matrix cores; it costs each gradient a relative error of
 * about that of its own bf16 rounding.  A gradient of type SBN_F32_FINE is
 * float32 from a D of two bf16 numbers, a value and what its rounding left
 * (at least 16 bits in all), each with a product of its own: that gradient's
 * product takes twice the time, and its error falls to that of float32 sums.
 *
 *   dX [T x K] of dtype dxdt, dW [V x K] of dtype dwdt (SBN_BF16, SBN_F32 or
 *   SBN_F32_FINE); either may be NULL.  With T = 0 dW is written as zeros.  dX
 *   without dW may be in X's place, dW of bf16 in W's (same stride).
 *   ws sbn_cross_entropy_backward_workspace_bytes(T, V, K) bytes, for any types
 */
sbn_status sbn_cross_entropy_backward_workspace_bytes(int64_t T, int64_t V, int64_t K, size_t* bytes);
sbn_status sbn_cross_entropy_backward(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
                                      const void* labels, int label_bytes, const float* lse, const float* dloss,
                                      int64_t T, int64_t V, int64_t K, void* dX, sbn_dtype dxdt, int64_t lddx,
                                      void* dW, sbn_dtype dwdt, int64_t lddw, void* ws, size_t ws_bytes,
                                      void* stream);

/* ------------------------------------------------------------------ AdamW
 *
 * One step on `count` tensors in one launch, so no element may be in two of
 * the tensors that it writes.  Per element, in float32 and in
 * this order (products and sums rounded one by one):
 *   g  = grad * grad_scale
 *   m <- m * beta1 + g * (1 - beta1)
 *   v <- v * beta2 + (g * g) * (1 - beta2)
 *   p <- p * (1 - lr * weight_decay)
 *          - (m * (lr / (1 - beta1^step))) / (sqrt(v) * (1 / sqrt(1 - beta2^step)) + eps)
 * p is rounded to its own type; the shadow, where there is one, is p rounded
 * to bf16 (the W of the sbn.h calls beside a float32 master weight).
 *
 * States in 8 bits: consecutive blocks of SBN_ADAMW_BLOCK elements of a tensor
 * (the last may be shorter) share one float32 scale s, the block's largest
 * magnitude, 0 if that is under 2^-100.  A code c stands for
 *   m: s * (c/127) * |c/127|, int8 in [-127, 127]: c = rint(127 sqrt(|m|/s)), with m's sign
 *   v: s * (c/255)^4,         uint8:               c = rint(255 (v/s)^(1/4)), at least 1 where v > 0
 * both finer towards zero than at the block's largest value.  In a block with
 * a scale, v > 0 never becomes 0, which its place under a quotient could not
 * bear; where v's scale is 0 (gradients under some 2^-50, whose squares are
 * too small) the step takes the block's m as 0 as well, and so forgets its
 * momentum.  The step uses the new m and v before they are rounded to codes.
 */
#define SBN_ADAMW_BLOCK 256

typedef struct sbn_adamw_entry {
  void* p;              /* parameters, n elements of dtype pdt            (in/out) */
  const void* grad;     /* gradients, n elements of dtype gdt             (in)     */
  void* m;              /* first moment: n float, or n int8 codes         (in/out) */
  void* v;              /* second moment: n float, or n uint8 codes       (in/out) */
  float* m_scale;       /* 8-bit states: ceil(n / SBN_ADAMW_BLOCK) floats (in/out) */
  float* v_scale;       /* the same for v */
  uint16_t* shadow;     /* bf16 copy of float32 parameters, or NULL       (out)    */
  int64_t n;            /* elements, >= 0 */
  float weight_decay;   /* of this tensor, finite */
  float reserved;       /* 0 */
} sbn_adamw_entry;

/*
 * Checks `count` entries in HOST memory (types, alignment, required pointers;
 * state_bits is 32 or 8) and lays out the launch: *blocks is the number of
 * blocks, and `map` (NULL to ask for the number only) receives 2 int32 per
 * block.  The caller copies the entries and the map to device memory once and
 * keeps them as long as the tensors stay where they are.  Host-only.
 */
sbn_status sbn_adamw_plan(const sbn_adamw_entry* entries, int64_t count, sbn_dtype pdt, sbn_dtype gdt,
                          int state_bits, int32_t* map, int64_t* blocks);

/*
 * The step, with `entries` and `map` in DEVICE memory as sbn_adamw_plan
 * accepted and wrote them (blocks = 0: nothing to do).  0 <= beta < 1, lr
 * finite, eps >= 0 finite, and with 8-bit states > 0 (as float32), step >= 1.
 * With eps = 0 an element whose v is 0 becomes the quotient by 0 that the
 * formula says (Inf, or NaN where m is 0 too).  `dyn`, if not NULL, is 4 floats
 * in device memory that take the place of host values, for steps replayed from
 * a graph: lr, 1 - beta1^step, 1 - beta2^step, grad_scale (1 without dyn).
 */
sbn_status sbn_adamw_step(const sbn_adamw_entry* entries, const int32_t* map, int64_t blocks, sbn_dtype pdt,
                          sbn_dtype gdt, int state_bits, double lr, double beta1, double beta2, double eps,
                          int64_t step, const float* dyn, void* stream);

/*
 * 8-bit states to and from float32 (checkpoints, a change of state type): n
 * elements, ceil(n / SBN_ADAMW_BLOCK) scales, the rules above.  second = 0 for
 * m, 1 for v.  n = 0: nothing to do.
 */
sbn_status sbn_adamw_decode_state(const void* codes, const float* scale, int64_t n, int second, float* out,
                                  void* stream);
sbn_status sbn_adamw_encode_state(const float* x, int64_t n, int second, void* codes, float* scale, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SBN_TRAIN_H */
