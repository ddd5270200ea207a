/*
 * sbn_keep.h -- C ABI of what a training step keeps for its backward pass in 8
 * bits, for AMD Instinct MI355X (gfx950).  The layer's own input is kept in 8
 * bits as it is (Xq and s_x of sbn.h); these calls do the same for what lies
 * between the layers:
 *
 *   checkpoints     a matrix in 8 bits, and its values again;
 *   RMS norm        sbn_rmsnorm_quant that also writes the checkpoint of h, and
 *                   the norm's gradient from that checkpoint;
 *   activation      the function between the two products of a feed-forward
 *                   block, u = f(a) b, with an RMS norm if asked, as the next
 *                   layer's 8-bit activations, which also writes the
 *                   checkpoints of a and b, and its gradient from them.
 *
 * The conventions of sbn.h and sbn_train.h hold: device pointers owned by the
 * caller and 16-byte aligned (scales and s_x: aligned to their elements),
 * row-major tensors with leading dimensions in elements and multiples of 8,
 * work enqueued on `stream`, arguments checked on the host before anything is
 * launched, nothing launched on an error, messages from sbn_last_error(), no
 * allocation, no synchronisation, no exception across the ABI.  Tensors that a
 * call writes overlap no other tensor of the call, except where it says that one
 * may be in another's place.  Every call may be captured into a HIP graph.
 * There are no atomics, every sum has a fixed order.  Inputs with NaN or Inf are
 * outside the contract, except where a call says what becomes of them; with
 * SBN_CHECK_FINITE=1 the calls scan their matrices and gains as sbn.h describes
 * (not the codes and scales of checkpoints).
 *
 * K is a multiple of 8 and at most SBN_RMSNORM_MAX_K (32768); T >= 0 (T = 0:
 * nothing to do, and pointers may be NULL; dgain is written as zeros); T*K < 2^37.
 */
#ifndef SBN_KEEP_H
#define SBN_KEEP_H

#include "sbn_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ checkpoints
 *
 * SBN_KEEP_BLOCK neighbours of a row (the last block of a row may be shorter)
 * share one float32 scale s = a / 127, a the block's largest magnitude, 0 if that
 * is under 2^-100, and no more than what 127 times is finite.  A code q in [-127, 127] stands for q * s:
 *   q = rint((127 * x) / a)     round half to even, all in float32 (127 x without
 *                               overflow); 0 where s = 0
 * so a value is off by at most a / 254.  A NaN or Inf in a block becomes its
 * scale, and all values of the block NaN.
 *
 *   X, Y    [T x K] of dtype dt (SBN_BF16 or SBN_F32), row strides ldx, ldy >= K
 *   codes   [T x K] int8, contiguous
 *   scales  [T x ceil(K / SBN_KEEP_BLOCK)] float, contiguous
 */
#define SBN_KEEP_BLOCK 128

sbn_status sbn_keep8_encode(const void* X, int64_t ldx, sbn_dtype dt, int64_t T, int64_t K, int8_t* codes,
                            float* scales, void* stream);
/* q * s, rounded to Y's type */
sbn_status sbn_keep8_decode(const int8_t* codes, const float* scales, int64_t T, int64_t K, void* Y, int64_t ldy,
                            sbn_dtype dt, void* stream);

/* ------------------------------------------------------------------ RMS norm
 *
 * sbn_rmsnorm_quant (h = x + residual, its norm as int8 codes Xq and scales
 * s_x, same values bit for bit), with the checkpoint of the stored h written in
 * the same pass.  The parameters are those of sbn_rmsnorm_quant; there is no
 * rstd, which the gradient forms again.
 */
sbn_status sbn_rmsnorm_quant_keep(const void* X, int64_t ldx, const void* residual, int64_t ldres, sbn_dtype dt,
                                  const void* gain, sbn_dtype gaindt, int64_t T, int64_t K, float eps, void* H,
                                  int64_t ldh, int8_t* Xq, float* s_x, int8_t* codes, float* scales, void* stream);

/*
 * The norm's gradient at the kept values: with h = q * s (float32),
 * r = 1 / sqrt(mean_k h^2 + eps), w = gain * dY:
 *   dX[t,k]  = r * (w[t,k] - h[t,k] * (r^2 * mean_k(w[t,:] * h[t,:]))) + dH[t,k]
 *   dgain[k] = sum_t dY[t,k] * (h[t,k] * r)
 * the 8-bit activations' quantizer passed straight through.  It is the gradient
 * of the norm at the checkpoint, not the forward's r on other values: scaling a
 * row does not change the norm, and dX is orthogonal to the kept row (eps aside).
 *
 *   dY, dH, dX  [T x K] of dtype dt; dH NULL for none; dX may be dY or dH itself (same stride)
 *   gain [K] of dtype gaindt; dgain [K] float, always written
 *   ws    sbn_rmsnorm_backward_kept_workspace_bytes(T, K) bytes, no initialisation
 * eps >= 0 and finite; with eps = 0 a row kept as zeros has no gradient (NaN).  The
 * sum of a row's squares has to stay below 2^128.
 */
sbn_status sbn_rmsnorm_backward_kept_workspace_bytes(int64_t T, int64_t K, size_t* bytes);
sbn_status sbn_rmsnorm_backward_kept(const void* dY, int64_t lddy, const void* dH, int64_t lddh, sbn_dtype dt,
                                     const int8_t* codes, const float* scales, const void* gain, sbn_dtype gaindt,
                                     int64_t T, int64_t K, float eps, void* dX, int64_t lddx, float* dgain, void* ws,
                                     size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ activation of a feed-forward block
 *
 *   u[t,k] = f(a[t,k]) * b[t,k]          (without B: u = f(a))
 *   SBN_RELU2: f(a) = max(a, 0)^2        SBN_SILU: f(a) = a / (1 + exp(-a))
 * out as the next layer's activations.  With a gain, of its RMS norm, as
 * sbn_rmsnorm_quant: v = u * gain, r = 1 / sqrt(mean_k u^2 + eps); without (gain
 * NULL): v = u, r = 1.  With m = max(max_k |v|, 2^-100):
 *   Xq[t,k] = rint((127 * v) / m),  s_x[t] = (m * r) / 127
 * u and v are float32 and never stored.
 *
 *   A, B      [T x K] of dtype dt, row strides lda, ldb >= K; B may be NULL.  Both may
 *             be halves of one matrix, such as one product's output.
 *   gain      [K] of dtype gaindt, or NULL
 *   Xq [T x K] int8, contiguous; s_x [T] float
 *   codes_a, scales_a, codes_b, scales_b   the checkpoints of A and of B: all of them
 *             NULL (inference); or all there, without B those of A
 * |u| has to stay finite, and with a gain a row's sum of u^2 below 2^128; squares of
 * |u| < 2^-75 count as 0 there.  eps >= 0 and finite; with eps = 0 a row of u that counts as
 * zeros, such as relu^2 of a row without positive values, has no norm (s_x is Inf, its gradients NaN).
 */
typedef enum { SBN_RELU2 = 0, SBN_SILU = 1 } sbn_act;

sbn_status sbn_activation_quant(const void* A, int64_t lda, const void* B, int64_t ldb, sbn_dtype dt, sbn_act act,
                                const void* gain, sbn_dtype gaindt, int64_t T, int64_t K, float eps, int8_t* Xq,
                                float* s_x, int8_t* codes_a, float* scales_a, int8_t* codes_b, float* scales_b,
                                void* stream);

/*
 * Its gradient at the kept values a = q_a * s_a, b = q_b * s_b (1 without B), u = f(a) * b:
 *   du = r * (w - u * (r^2 * mean_k(w * u))),  w = gain * dY   (without a gain: du = dY)
 *   dA = du * b * f'(a)      dB = du * f(a)      dgain[k] = sum_t dY[t,k] * (u[t,k] * r)
 * (f'(0) = 0 for SBN_RELU2).
 *
 *   dY, dA, dB  [T x K] of dtype dt; dA or dB may be dY itself (same stride)
 *   codes_b, scales_b, dB   all NULL where the forward had no B
 *   gain, dgain  both NULL where the forward had no gain
 *   ws    sbn_activation_backward_workspace_bytes(T, K) bytes, no initialisation (with a
 *         gain; without one it may be NULL)
 */
sbn_status sbn_activation_backward_workspace_bytes(int64_t T, int64_t K, size_t* bytes);
sbn_status sbn_activation_backward(const void* dY, int64_t lddy, sbn_dtype dt, const int8_t* codes_a,
                                   const float* scales_a, const int8_t* codes_b, const float* scales_b, sbn_act act,
                                   const void* gain, sbn_dtype gaindt, int64_t T, int64_t K, float eps, void* dA,
                                   int64_t ldda, void* dB, int64_t lddb, float* dgain, void* ws, size_t ws_bytes,
                                   void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SBN_KEEP_H */
