// RMS norm with the residual's addition, output in the tensors' type or as the
// layer's int8 activations, and its gradient.
//
//   h = x + residual;  rstd = (mean h^2 + eps)^-1/2;  y = h rstd gain
//   int8: u = h gain, a = max|u|, Xq = rint(127 u / a), s_x = a rstd / 127
//
// rstd multiplies a whole row, so it cancels from the codes: the maximum of |u|
// and the sum of h^2 come out of one pass over the row, which stays in
// registers until it is written.  The rounding of u / a is act_quant's
// (act_quant.h): bit-equal to the division's rint.
//
// The gradient, with n = h rstd and w = gain dy:
//   dx = rstd (w - n mean(w n)) + dh;  dgain = sum_t dy n
// TPR threads hold a row, each the same columns of every row it sees, so
// dgain's partial sums stay in registers over the rows of a block; blocks
// write them side by side and a second launch adds them in a fixed order.
//
// Both directions are bound by memory traffic: every row is read once and
// written once.
#include "act_quant.h"
#include "train_internal.h"

namespace sbn {
namespace {

constexpr float U_FLOOR = 0x1p-100f;   // least row maximum told from 0 (127 / a stays finite)

// ---------------------------------------------------------------- 8 elements of a row
template <bool F32>
struct Vec8 {
  uint4 a, b;                          // b: elements 4..7 of float32 rows
  __device__ void load(const void* p, int64_t i) {
    if (F32) {
      a = ((const uint4*)p)[2 * i];
      b = ((const uint4*)p)[2 * i + 1];
    } else {
      a = ((const uint4*)p)[i];
    }
  }
  __device__ void to(float* v) const {
    if (F32) {
      v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
      v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
    } else {
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
  __device__ void from(const float* v) {
    if (F32) {
      a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    } else {
      a = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
  }
  __device__ void store(void* p, int64_t i) const {
    if (F32) {
      ((uint4*)p)[2 * i] = a;
      ((uint4*)p)[2 * i + 1] = b;
    } else {
      ((uint4*)p)[i] = a;
    }
  }
};

__device__ inline void gain8(const void* gain, bool f32, int64_t i, float* v) {
  if (f32) {
    Vec8<true> g;
    g.load(gain, i);
    g.to(v);
  } else {
    Vec8<false> g;
    g.load(gain, i);
    g.to(v);
  }
}

__device__ inline float wave_sum(float x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m);
  return x;
}
__device__ inline float wave_max(float x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x = fmaxf(x, __shfl_xor(x, m));
  return x;
}

// ---------------------------------------------------------------- forward
struct FwdArgs {
  const void *X, *res, *gain;
  void *H, *Y;
  int8_t* Xq;
  float *s_x, *rstd;
  int64_t ldx, ldr, ldh, ldy, T;
  int K;
  float eps;
  bool gain_f32;
};

// TPR threads per row, BT / TPR rows per block, CH chunks of 8 elements per
// thread (CH * TPR * 8 >= K).
template <bool F32, bool Q, int BT, int TPR, int CH>
__global__ __launch_bounds__(BT) void rmsnorm_kernel(FwdArgs A) {
  constexpr int ROWS = BT / TPR, WPR = TPR / 64;
  __shared__ float red[2][BT / 64];
  const int g = threadIdx.x % TPR, wave = threadIdx.x >> 6;
  const int kc = A.K / 8, es = F32 ? 4 : 2;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  // every thread of a block makes the same number of rounds (barriers inside)
  for (int64_t t0 = (int64_t)blockIdx.x * ROWS; t0 < A.T; t0 += step) {
    const int64_t t = t0 + threadIdx.x / TPR;
    const bool live = t < A.T;
    const int n = live ? kc : 0;
    const char* xr = (const char*)A.X + t * A.ldx * es;
    const char* rr = (const char*)A.res + t * A.ldr * es;
    Vec8<F32> h[CH], r[CH];
    if (A.res) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (g + TPR * i < n) {
          h[i].load(xr, g + TPR * i);
          r[i].load(rr, g + TPR * i);
        }
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (g + TPR * i < n) h[i].load(xr, g + TPR * i);
    }
    float ss = 0.0f, mx = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = g + TPR * i;
      if (c < n) {
        float v[8];
        h[i].to(v);
        if (A.res) {
          float w[8];
          r[i].to(w);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += w[j];
          h[i].from(v);
          h[i].store((char*)A.H + t * A.ldh * es, c);
          if (!F32) h[i].to(v);                     // the stored h is what is normalised
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += v[j] * v[j];
        if (Q) {
          float w[8];
          gain8(A.gain, A.gain_f32, c, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(v[j] * w[j]));
        }
      }
    }
    ss = wave_sum(ss);
    if (Q) mx = wave_max(mx);
    if (WPR > 1) {
      __syncthreads();                              // the previous round's reads of red
      if ((threadIdx.x & 63) == 0) {
        red[0][wave] = ss;
        red[1][wave] = mx;
      }
      __syncthreads();
      const int w0 = wave / WPR * WPR;
      ss = red[0][w0];
      mx = red[1][w0];
#pragma unroll
      for (int w = 1; w < WPR; ++w) {
        ss += red[0][w0 + w];
        mx = fmaxf(mx, red[1][w0 + w]);
      }
    }
    const float rstd = 1.0f / sqrtf(ss / (float)A.K + A.eps);
    const float a = fmaxf(mx, U_FLOOR);
    if (g == 0 && live) {
      if (A.rstd) A.rstd[t] = rstd;
      if (Q) A.s_x[t] = (a * rstd) / 127.0f;
    }
    const float rcp = 127.0f / a;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = g + TPR * i;
      if (c < n) {
        float v[8], w[8];
        h[i].to(v);
        gain8(A.gain, A.gain_f32, c, w);
        if (Q) {
          uint32_t o[2] = {0u, 0u};
#pragma unroll
          for (int j = 0; j < 8; ++j)
            o[j >> 2] |= (uint32_t)(aq_quant_one(v[j] * w[j], rcp, a) & 0xFF) << (8 * (j & 3));
          *(uint2*)(A.Xq + t * A.K + 8 * c) = make_uint2(o[0], o[1]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = v[j] * rstd * w[j];
          h[i].from(v);
          h[i].store((char*)A.Y + t * A.ldy * es, c);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- backward
struct BwdArgs {
  const void *dY, *H, *dH, *gain;
  const float* rstd;
  void* dX;
  float* part;                         // [gridDim.x][K] partial sums of dgain
  int64_t lddy, ldh, lddh, lddx, T;
  int K;
  bool gain_f32;
};

template <bool F32, int BT, int TPR, int CH>
__global__ __launch_bounds__(BT) void rmsnorm_grad_kernel(BwdArgs A) {
  constexpr int ROWS = BT / TPR, WPR = TPR / 64;
  __shared__ float red[2][BT / 64];
  extern __shared__ float gsum[];                   // [ROWS - 1][K]
  const int g = threadIdx.x % TPR, wave = threadIdx.x >> 6, row = threadIdx.x / TPR;
  const int kc = A.K / 8, es = F32 ? 4 : 2;
  float dg[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = 0.0f;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int turn = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * ROWS; t0 < A.T; t0 += step, turn ^= 1) {
    const int64_t t = t0 + row;
    const bool live = t < A.T;
    const int n = live ? kc : 0;
    const float rstd = live ? A.rstd[t] : 0.0f;
    const char* yr = (const char*)A.dY + t * A.lddy * es;
    const char* hr = (const char*)A.H + t * A.ldh * es;
    const char* dr = (const char*)A.dH + t * A.lddh * es;
    Vec8<F32> y[CH], h[CH], d[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (g + TPR * i < n) {
        y[i].load(yr, g + TPR * i);
        h[i].load(hr, g + TPR * i);
      }
    if (A.dH) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (g + TPR * i < n) d[i].load(dr, g + TPR * i);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = g + TPR * i;
      if (c < n) {
        float yv[8], hv[8], w[8];
        y[i].to(yv);
        h[i].to(hv);
        gain8(A.gain, A.gain_f32, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float yn = yv[j] * (hv[j] * rstd);
          dg[i][j] += yn;
          s += yn * w[j];
        }
      }
    }
    s = wave_sum(s);
    if (WPR > 1) {
      // two rows of red in turn: one barrier a round keeps a fast wave's next
      // write away from a slow wave's read
      if ((threadIdx.x & 63) == 0) red[turn][wave] = s;
      __syncthreads();
      const int w0 = wave / WPR * WPR;
      s = red[turn][w0];
#pragma unroll
      for (int w = 1; w < WPR; ++w) s += red[turn][w0 + w];
    }
    const float mean = s / (float)A.K;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = g + TPR * i;
      if (c < n) {
        float yv[8], hv[8], w[8], dv[8];
        y[i].to(yv);
        h[i].to(hv);
        gain8(A.gain, A.gain_f32, c, w);
        if (A.dH) d[i].to(dv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float x = rstd * (w[j] * yv[j] - (hv[j] * rstd) * mean);
          if (A.dH) x += dv[j];
          yv[j] = x;
        }
        y[i].from(yv);
        y[i].store((char*)A.dX + t * A.lddx * es, c);
      }
    }
  }
  // dgain of the block's ROWS groups, added in their order
  if (ROWS > 1) {
    if (row > 0) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = g + TPR * i;
        if (c < kc)
#pragma unroll
          for (int j = 0; j < 8; ++j) gsum[(row - 1) * A.K + 8 * c + j] = dg[i][j];
      }
    }
    __syncthreads();
    if (row > 0) return;
  }
  float* out = A.part + (int64_t)blockIdx.x * A.K;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = g + TPR * i;
    if (c < kc) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        for (int w = 1; w < ROWS; ++w) dg[i][j] += gsum[(w - 1) * A.K + 8 * c + j];
      Vec8<true> o;
      o.from(dg[i]);
      o.store(out, c);
    }
  }
}

// dgain[k] = sum over the blocks' partials: 64 columns a block, 16 waves take
// every 16th partial each, then the 16 sums are added in order
__global__ __launch_bounds__(1024) void rmsnorm_dgain_kernel(const float* __restrict__ part, int G, int K,
                                                             float* __restrict__ dgain) {
  __shared__ float sm[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int k = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (k < K)
    for (int b = wave; b < G; b += 16) s += part[(int64_t)b * K + k];
  sm[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && k < K) {
    for (int w = 1; w < 16; ++w) s += sm[w][lane];
    dgain[k] = s;
  }
}

constexpr int BWD_BLOCKS = 512;                     // two blocks of 256 threads per compute unit

int bwd_blocks(int64_t T) { return (int)(T < BWD_BLOCKS ? T : BWD_BLOCKS); }

constexpr int64_t GRID_MAX = 1 << 20;               // blocks; rows beyond are taken in further rounds

template <bool F32, bool Q, int BT, int TPR, int CH>
void run_fwd(const FwdArgs& A, hipStream_t st) {
  constexpr int ROWS = BT / TPR;
  int64_t blocks = cdiv(A.T, ROWS);
  if (blocks > GRID_MAX) blocks = GRID_MAX;
  SBN_LAUNCH(Q ? "rmsnorm_quant" : "rmsnorm", (rmsnorm_kernel<F32, Q, BT, TPR, CH>), dim3((unsigned)blocks), dim3(BT), 0,
             st, A);
}

template <bool F32, bool Q>
void pick_fwd(const FwdArgs& A, hipStream_t st) {
  const int kc = A.K / 8;
  if (kc <= 512 && A.T >= 1024) {
    const int ch = (kc + 63) / 64;
    if (ch <= 1) run_fwd<F32, Q, 256, 64, 1>(A, st);
    else if (ch <= 2) run_fwd<F32, Q, 256, 64, 2>(A, st);
    else if (ch <= 3) run_fwd<F32, Q, 256, 64, 3>(A, st);
    else if (ch <= 4) run_fwd<F32, Q, 256, 64, 4>(A, st);
    else if (ch <= 5) run_fwd<F32, Q, 256, 64, 5>(A, st);
    else if (ch <= 6) run_fwd<F32, Q, 256, 64, 6>(A, st);
    else run_fwd<F32, Q, 256, 64, 8>(A, st);
  } else if (kc <= 256) run_fwd<F32, Q, 256, 256, 1>(A, st);
  else if (kc <= 512) run_fwd<F32, Q, 256, 256, 2>(A, st);
  else if (kc <= 1024) run_fwd<F32, Q, 256, 256, 4>(A, st);
  else if (kc <= 2048) run_fwd<F32, Q, 1024, 1024, 2>(A, st);
  else run_fwd<F32, Q, 1024, 1024, 4>(A, st);
}

template <bool F32, int BT, int TPR, int CH>
void run_bwd(const BwdArgs& A, int blocks, hipStream_t st) {
  constexpr int ROWS = BT / TPR;
  SBN_LAUNCH("rmsnorm_grad", (rmsnorm_grad_kernel<F32, BT, TPR, CH>), dim3((unsigned)blocks), dim3(BT),
             (size_t)(ROWS - 1) * A.K * sizeof(float), st, A);
}

template <bool F32>
void pick_bwd(const BwdArgs& A, int blocks, hipStream_t st) {
  const int kc = A.K / 8;
  if (kc <= 256) run_bwd<F32, 256, 256, 1>(A, blocks, st);
  else if (kc <= 512) run_bwd<F32, 256, 256, 2>(A, blocks, st);
  else if (kc <= 1024) run_bwd<F32, 256, 256, 4>(A, blocks, st);
  else if (kc <= 2048) run_bwd<F32, 1024, 1024, 2>(A, blocks, st);
  else run_bwd<F32, 1024, 1024, 4>(A, blocks, st);
}

}  // namespace

hipError_t launch_rmsnorm(const void* X, int64_t ldx, const void* res, int64_t ldr, bool f32, const void* gain,
                          bool gain_f32, int64_t T, int64_t K, float eps, void* H, int64_t ldh, void* Y, int64_t ldy,
                          int8_t* Xq, float* s_x, float* rstd, hipStream_t st) {
  const FwdArgs A{X, res, gain, H, Y, Xq, s_x, rstd, ldx, ldr, ldh, ldy, T, (int)K, eps, gain_f32};
  if (f32) {
    if (Xq) pick_fwd<true, true>(A, st);
    else pick_fwd<true, false>(A, st);
  } else {
    if (Xq) pick_fwd<false, true>(A, st);
    else pick_fwd<false, false>(A, st);
  }
  return hipGetLastError();
}

size_t rmsnorm_bwd_ws_bytes(int64_t T, int64_t K) { return align256((size_t)bwd_blocks(T) * (size_t)K * sizeof(float)); }

hipError_t launch_rmsnorm_backward(const void* dY, int64_t lddy, const void* H, int64_t ldh, const void* dH,
                                   int64_t lddh, bool f32, const void* gain, bool gain_f32, const float* rstd,
                                   int64_t T, int64_t K, void* dX, int64_t lddx, float* dgain, void* ws,
                                   hipStream_t st) {
  const int blocks = bwd_blocks(T);
  if (T > 0) {
    const BwdArgs A{dY, H, dH, gain, rstd, dX, (float*)ws, lddy, ldh, lddh, lddx, T, (int)K, gain_f32};
    if (f32) pick_bwd<true>(A, blocks, st);
    else pick_bwd<false>(A, blocks, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  SBN_LAUNCH("rmsnorm_dgain", rmsnorm_dgain_kernel, dim3((unsigned)cdiv(K, 64)), dim3(1024), 0, st, (const float*)ws,
             blocks, (int)K, dgain);
  return hipGetLastError();
}

}  // namespace sbn
