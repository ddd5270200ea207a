// Launchers of the operators declared in include/sbn_keep.h (T >= 1, except the
// gradients with a gain, which write dgain for T = 0 too).
#pragma once

#include "sbn_internal.h"
#include "sbn_keep.h"

namespace sbn {

hipError_t launch_keep8_encode(const void* X, int64_t ldx, bool f32, int64_t T, int64_t K, int8_t* codes, float* scales,
                               hipStream_t st);
hipError_t launch_keep8_decode(const int8_t* codes, const float* scales, int64_t T, int64_t K, void* Y, int64_t ldy,
                               bool f32, hipStream_t st);
hipError_t launch_rmsnorm_quant_keep(const void* X, int64_t ldx, const void* res, int64_t ldr, bool f32, const void* gain,
                                     bool gain_f32, int64_t T, int64_t K, float eps, void* H, int64_t ldh, int8_t* Xq,
                                     float* s_x, int8_t* codes, float* scales, hipStream_t st);
hipError_t launch_rmsnorm_backward_kept(const void* dY, int64_t lddy, const void* dH, int64_t lddh, bool f32,
                                        const int8_t* codes, const float* scales, const void* gain, bool gain_f32,
                                        int64_t T, int64_t K, float eps, void* dX, int64_t lddx, float* dgain, void* ws,
                                        hipStream_t st);
// workspace of both gradients with a gain
size_t kept_bwd_ws_bytes(int64_t T, int64_t K);
// B NULL: no second factor; codes_a NULL: nothing kept; gain and dgain NULL: no norm (and ws unused)
hipError_t launch_activation_quant(const void* A, int64_t lda, const void* B, int64_t ldb, bool f32, sbn_act act,
                                   const void* gain, bool gain_f32, int64_t T, int64_t K, float eps, int8_t* Xq,
                                   float* s_x, int8_t* codes_a, float* scales_a, int8_t* codes_b, float* scales_b,
                                   hipStream_t st);
hipError_t launch_activation_backward(const void* dY, int64_t lddy, bool f32, const int8_t* codes_a,
                                      const float* scales_a, const int8_t* codes_b, const float* scales_b, sbn_act act,
                                      const void* gain, bool gain_f32, int64_t T, int64_t K, float eps, void* dA,
                                      int64_t ldda, void* dB, int64_t lddb, float* dgain, void* ws, hipStream_t st);

}  // namespace sbn
