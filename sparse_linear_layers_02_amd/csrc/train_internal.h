// Launchers of the operators declared in include/sbn_train.h.
#pragma once

#include "sbn_internal.h"
#include "sbn_train.h"

namespace sbn {

#ifdef __HIPCC__
// ----------------------------------------------------------------- sums and maxima over lanes
// In the vector unit: within 16 lanes by quads, halves and mirrors of a row, then
// by exchanging rows and halves.  (Through LDS each step waits some 60 cycles.)
// Every lane gets the same value.
struct Add {
  __device__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
template <int CTRL>
__device__ inline float row_move(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
template <class Op>
__device__ inline float row16_all(float x, Op op) {
  x = op(x, row_move<0xB1>(x));                      // quad_perm 1 0 3 2
  x = op(x, row_move<0x4E>(x));                      // quad_perm 2 3 0 1
  x = op(x, row_move<0x141>(x));                     // row_half_mirror
  return op(x, row_move<0x140>(x));                  // row_mirror
}
// lanes of equal place in the rows of 16: of the two rows of each half wave, of all four
template <class Op>
__device__ inline float row_pairs_all(float x, Op op) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
template <class Op>
__device__ inline float rows_all(float x, Op op) {
  x = row_pairs_all(x, op);
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
template <class Op>
__device__ inline float half_wave_all(float x, Op op) {
  return row_pairs_all(row16_all(x, op), op);
}
template <class Op>
__device__ inline float wave_all(float x, Op op) {
  return rows_all(row16_all(x, op), op);
}
// sum + the squares of 8 bf16 values, by an instruction that rounds up to three times for
// two of them and may take what is under 2^-126 for 0
__device__ inline float add_squares(v8bf x, float sum) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const v2bf two = {x[j], x[j + 1]};
    sum = __builtin_amdgcn_fdot2_f32_bf16(two, two, sum, false);
  }
  return sum;
}
#endif

// ----------------------------------------------------------------- RMS norm (T >= 1)
// Xq != NULL: the 8-bit form (Y unused); otherwise Y.
hipError_t launch_rmsnorm(const void* X, int64_t ldx, const void* res, int64_t ldr, bool f32, const void* gain,
                          bool gain_f32, int64_t T, int64_t K, float eps, void* H, int64_t ldh, void* Y, int64_t ldy,
                          int8_t* Xq, float* s_x, float* rstd, hipStream_t st);
size_t rmsnorm_bwd_ws_bytes(int64_t T, int64_t K);
// dgain [K] from `blocks` rows of partial sums
hipError_t launch_norm_dgain(const float* part, int blocks, int64_t K, float* dgain, hipStream_t st);
hipError_t launch_rmsnorm_backward(const void* dY, int64_t lddy, const void* H, int64_t ldh, const void* dH,
                                   int64_t lddh, bool f32, const void* gain, bool gain_f32, const float* rstd,
                                   int64_t T, int64_t K, void* dX, int64_t lddx, float* dgain, void* ws,
                                   hipStream_t st);

// ----------------------------------------------------------------- cross entropy (T >= 1)
size_t ce_ws_bytes(int64_t T, int64_t V, int64_t K);
// pair: a gradient of type SBN_F32_FINE is asked for
size_t ce_bwd_ws_bytes(int64_t T, int64_t V, int64_t K, bool pair);
// of log probabilities' gradients, dX, dW of type SBN_F32_FINE
size_t policy_bwd_ws_bytes(int64_t T, int64_t V, int64_t K, bool fine_x, bool fine_w);
hipError_t launch_ce(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, const void* labels,
                     bool labels64, int64_t T, int64_t V, int64_t K, float* loss, float* lse, void* ws,
                     hipStream_t st);
// What the gradients of the logits come from: the losses' gradients, or, with `policy`,
// those of log probabilities (dloss) and entropies, either of which may be NULL, of
// logits times `scale`; labels may then be NULL too.
struct HeadGrad {
  const void* labels;
  bool labels64;
  const float *lse, *dloss;
  bool policy = false;
  float scale = 1.0f;
  const float *entropy = nullptr, *dentropy = nullptr;
};
hipError_t launch_ce_backward(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, const HeadGrad& H, int64_t T,
                              int64_t V, int64_t K, void* dX, sbn_dtype dxdt, int64_t lddx, void* dW, sbn_dtype dwdt,
                              int64_t lddw, void* ws, hipStream_t st);
// rows x len elements of `elem_bytes` at row stride ld, all set to 0
hipError_t launch_zero_rows(void* p, int64_t rows, int64_t len, int64_t ld, int elem_bytes, hipStream_t st);

// ----------------------------------------------------------------- AdamW
constexpr int ADAMW_CHUNK = 2048;   // elements of one block: 8 per thread
struct AdamWScalars {
  float beta1, one_minus_beta1, beta2, one_minus_beta2, eps;
  float lr, rate, rbias2;           // rate = lr / (1 - beta1^step), rbias2 = 1 / sqrt(1 - beta2^step), in float32
};
hipError_t launch_adamw(const sbn_adamw_entry* entries, const int32_t* map, int64_t blocks, bool p_f32, bool g_f32,
                        bool state8, const AdamWScalars& s, const float* dyn, hipStream_t st);
hipError_t launch_adamw_decode(const void* codes, const float* scale, int64_t n, bool second, float* out,
                               hipStream_t st);
hipError_t launch_adamw_encode(const float* x, int64_t n, bool second, void* codes, float* scale, hipStream_t st);

}  // namespace sbn
