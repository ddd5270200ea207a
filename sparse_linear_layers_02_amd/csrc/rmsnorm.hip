// RMS norm with the residual's addition, output in the tensors' type or as the
// layer's int8 activations, and its gradient.
//
//   h = x + residual;  rstd = (mean h^2 + eps)^-1/2;  y = h rstd gain
//   int8: u = h gain, a = max|u|, Xq = rint(127 u / a), s_x = a rstd / 127
//
// rstd multiplies a whole row, so it cancels from the codes: the maximum of |u|
// and the sum of h^2 come out of one pass over the row, which stays in
// registers until it is written.
//
// The gradient, with n = h rstd and w = gain dy:
//   dx = rstd (w - n mean(w n)) + dh;  dgain = sum_t dy n
// A thread holds the same columns of every row that its block sees, so dgain's
// partial sums stay in registers over the rows of a block; blocks write them side
// by side and a second launch adds them in a fixed order.
//
// Both directions are bound by memory traffic: every row is read once and
// written once.  Kernel times in bf16: 8-bit output of 4096 x 2560 with the
// residual 15.0 us (4.9 TB/s of 73 MB; a large copy reaches 4.7 to 4.9), gradient
// of 8192 x 4096 with dh 40 us for one set of tensors again and again (6.6 TB/s of
// 268 MB; 202 MB fetched, 76 MB written), 50 for three in turn, and 4.8 us for
// dgain's sums.  One token of 2560: 2.8 us, latency.  Wider rows, 2048 with the
// residual in bf16, 8-bit output / bf16 output / gradient: K = 6912 24.4 / 24.6 /
// 30.7 us, 11008 39 / 40 / 45, 16384 53 / 52 / 63 (4.4, 5.2, 4.3 TB/s).  Above 16384
// a thread holds four chunks, and of the six kernels four keep 76 to 216 bytes a
// lane in scratch memory: K = 28672 104 / 99 / 140 us (4.0, 4.7, 3.4 TB/s), float32
// 244 / 241 / 308 (3.1, 3.9, 3.1).
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

// 8 codes rint((127 u) / a), rcp = 127 / a to two units in the last place.  Added
// to 1.5 2^23, u rcp is rounded to an integer, whose byte the sum's lowest is; u
// rcp is off by under 2^-15.  If one of the 8 lies within 2^-14 of a half-integer,
// all are divided, correctly rounded, both sides scaled so that 127 u is finite
// (about one wave in 17 does).
__device__ inline uint2 codes8(const float* u, float rcp, float a) {
  constexpr float SHIFT = 12582912.0f;
  float q[8], half = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    q[j] = fmaf(u[j], rcp, SHIFT);
    half = fmaxf(half, fabsf(fmaf(u[j], rcp, SHIFT - q[j])));
  }
  if (half > 0.5f - 0x1p-14f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = rintf((127.0f * (u[j] * 0x1p-8f)) / (a * 0x1p-8f)) + SHIFT;
  }
  uint32_t o[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {                      // the four lowest bytes
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(q[4 * j + 1]), __float_as_uint(q[4 * j]), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(q[4 * j + 3]), __float_as_uint(q[4 * j + 2]), 0x0c0c0400u);
    o[j] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
  }
  return make_uint2(o[0], o[1]);
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

// A block holds one row at a time, CH chunks of 8 elements per thread
// (CH * blockDim.x * 8 >= K); rows beyond the grid are taken in further rounds.
template <bool F32, bool Q, int CH, int MAXT>
__global__ __launch_bounds__(MAXT) void rmsnorm_kernel(FwdArgs A) {
  __shared__ float red[2][2][MAXT / 64];
  const int g = threadIdx.x, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int n = A.K / 8, es = F32 ? 4 : 2, TPR = blockDim.x;
  int turn = 0;
  for (int64_t t = blockIdx.x; t < A.T; t += gridDim.x, turn ^= 1) {
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
    // Of one chunk the gain is loaded before the first store, which a later load
    // would wait for.  Microseconds late / early, with the residual: 8-bit output of
    // bf16 4096 x 2560 16.3 / 15.6, 1021 x 4096 9.0 / 8.6, of float32 11.4 / 10.9; bf16
    // output 1021 x 4096 7.5 / 7.0, 8192 x 4096 49.3 / 48.2; all of 333 x 2560 the same.
    // Float32 output gains nothing by it: 12.1 / 12.7 at 1021 x 4096, 94.5 / 94.6 at
    // 8192 x 4096, 4.4 / 4.4 at 333 x 2560 (without the residual 9.2 / 8.7, 50.1 / 49.7,
    // 3.6 / 3.4).  More chunks leave room for fewer blocks: 1024 x 16384 30.1 / 33.2
    // in 8 bits, 28.3 / 31.9 in bf16, 1024 x 6912 13.1 / 12.8 and 10.3 / 11.5.
    constexpr bool EARLY = CH == 1 && (Q || !F32);
    float gain[8];
    if (EARLY && g < n) gain8(A.gain, A.gain_f32, g, gain);
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
          if (!EARLY) gain8(A.gain, A.gain_f32, c, gain);
#pragma unroll
          for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(v[j] * gain[j]));
        }
      }
    }
    ss = wave_all(ss, Add{});
    if (Q) mx = wave_all(mx, Max{});
    if (waves > 1) {
      // two sets of red in turn: one barrier a round keeps a fast wave's next
      // write away from a slow wave's read
      if ((threadIdx.x & 63) == 0) {
        red[turn][0][wave] = ss;
        red[turn][1][wave] = mx;
      }
      __syncthreads();
      const int l = threadIdx.x & 15;               // at most 16 waves
      ss = row16_all(l < waves ? red[turn][0][l] : 0.0f, Add{});
      if (Q) mx = row16_all(l < waves ? red[turn][1][l] : 0.0f, Max{});
    }
    const float rstd = 1.0f / sqrtf(ss / (float)A.K + A.eps);
    const float a = fmaxf(mx, U_FLOOR);
    if (g == 0) {
      if (A.rstd) A.rstd[t] = rstd;
      if (Q) A.s_x[t] = (a * rstd) / 127.0f;
    }
    const float rcp = __builtin_amdgcn_rcpf(a * (1.0f / 127.0f));   // (1 / a itself may be too small for a float)
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = g + TPR * i;
      if (c < n) {
        float v[8];
        h[i].to(v);
        if (!EARLY) gain8(A.gain, A.gain_f32, c, gain);
        if (Q) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] *= gain[j];
          *(uint2*)(A.Xq + t * A.K + 8 * c) = codes8(v, rcp, a);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = v[j] * rstd * gain[j];
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

template <bool F32, int CH, int MAXT>
__global__ __launch_bounds__(MAXT) void rmsnorm_grad_kernel(BwdArgs A) {
  __shared__ float red[2][MAXT / 64];
  const int g = threadIdx.x, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int n = A.K / 8, es = F32 ? 4 : 2, TPR = blockDim.x;
  // up to two chunks of gain stay for all rows (8192 x 4096: 62.5 -> 56.8 us); four would not fit the registers
  constexpr bool KEPT = CH <= 2;
  float dg[CH][8], gain[KEPT ? CH : 1][8];
#pragma unroll
  for (int i = 0; i < CH; ++i)
    if (KEPT && g + TPR * i < n) gain8(A.gain, A.gain_f32, g + TPR * i, gain[i]);
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = 0.0f;
  int turn = 0;
  for (int64_t t = blockIdx.x; t < A.T; t += gridDim.x, turn ^= 1) {
    const float rstd = A.rstd[t];
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
        float yv[8], hv[8], *w = gain[KEPT ? i : 0];
        y[i].to(yv);
        h[i].to(hv);
        if (!KEPT) gain8(A.gain, A.gain_f32, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float yn = yv[j] * (hv[j] * rstd);
          dg[i][j] += yn;
          s += yn * w[j];
        }
      }
    }
    s = wave_all(s, Add{});
    if (waves > 1) {
      if ((threadIdx.x & 63) == 0) red[turn][wave] = s;
      __syncthreads();                              // and the other set of red for the next round
      const int l = threadIdx.x & 15;
      s = row16_all(l < waves ? red[turn][l] : 0.0f, Add{});
    }
    const float mean = s / (float)A.K;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = g + TPR * i;
      if (c < n) {
        float yv[8], hv[8], dv[8], *w = gain[KEPT ? i : 0];
        y[i].to(yv);
        h[i].to(hv);
        if (!KEPT) gain8(A.gain, A.gain_f32, c, w);
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
  float* out = A.part + (int64_t)blockIdx.x * A.K;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = g + TPR * i;
    if (c < n) {
      Vec8<true> o;
      o.from(dg[i]);
      o.store(out, c);
    }
  }
}

// dgain[k] = sum over the blocks' partials: 16 columns a block, 4 a thread, 64
// threads a column take every 64th partial each, then the 64 sums are added in a
// tree.  (64 columns a block and 16 threads a column: 9.4 us for 512 x 4096.)
__global__ __launch_bounds__(256) void rmsnorm_dgain_kernel(const float* __restrict__ part, int G, int K,
                                                            float* __restrict__ dgain) {
  __shared__ v4f sm[64][4];
  const int q = threadIdx.x & 3, r = threadIdx.x >> 2;
  const int k = blockIdx.x * 16 + 4 * q;
  v4f s = (v4f){0.f, 0.f, 0.f, 0.f};
  if (k < K) {
    int b = r;
    for (; b + 192 < G; b += 256) {                 // four loads in flight
      const v4f x0 = *(const v4f*)(part + (int64_t)b * K + k), x1 = *(const v4f*)(part + (int64_t)(b + 64) * K + k);
      const v4f x2 = *(const v4f*)(part + (int64_t)(b + 128) * K + k), x3 = *(const v4f*)(part + (int64_t)(b + 192) * K + k);
      s += (x0 + x1) + (x2 + x3);
    }
    for (; b < G; b += 64) s += *(const v4f*)(part + (int64_t)b * K + k);
  }
  sm[r][q] = s;
  __syncthreads();
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    if (r < d) sm[r][q] += sm[r + d][q];
    __syncthreads();
  }
  if (r == 0 && k < K) *(v4f*)(dgain + k) = sm[0][q];
}

// threads of a block for n chunks at CH a thread
int threads_for(int n, int ch) { return (int)round_up(cdiv(n, ch), 64); }
int chunks_for(int n) { return n <= 512 ? 1 : n <= 2048 ? 2 : 4; }

// Blocks of the gradient: 16 waves a compute unit, but a block's partial of dgain
// costs as much traffic as two rows in 16 bits, so at least 8 rows a block where
// that leaves one block a compute unit.  (bf16, microseconds at 256 / 512 / 1024
// blocks: T = 8192, K = 4096: 61.6 / 56.6 / 63.3; T = 8192, K = 1024: 32.5 / 22.5 /
// 19.2; T = 4096, K = 2560: 24.6 / 21.3 / 23.1; T = 1021, K = 4096: 14.2 / 15.3 /
// 21.6.  With dgain's sums at 64 / 128 / 256 blocks, below the one a compute unit:
// T = 1021, K = 4096 15.0 / 14.4 / 12.5, float32 17.0 / 16.4 / 14.4, K = 1024 10.1 / 9.8
// / 7.9; T = 333, K = 2560 9.3 / 7.9 / 8.2, float32 9.8 / 8.3 / 8.6; 64 rows and fewer
// one a block in any case.)
int bwd_blocks(int64_t T, int64_t K) {
  const int n = (int)(K / 8), most = 256 * 16 / (threads_for(n, chunks_for(n)) / 64);
  int64_t g = T / 8 < 256 ? 256 : T / 8;
  if (g > most) g = most;
  return (int)(g < T ? g : T);
}

constexpr int64_t GRID_MAX = 1 << 20;               // blocks; rows beyond are taken in further rounds

template <bool F32, bool Q, int CH, int MAXT>
void run_fwd(const FwdArgs& A, hipStream_t st) {
  SBN_LAUNCH(Q ? "rmsnorm_quant" : "rmsnorm", (rmsnorm_kernel<F32, Q, CH, MAXT>),
             dim3((unsigned)(A.T < GRID_MAX ? A.T : GRID_MAX)), dim3((unsigned)threads_for(A.K / 8, CH)), 0, st, A);
}

template <bool F32, bool Q>
void pick_fwd(const FwdArgs& A, hipStream_t st) {
  const int n = A.K / 8;
  if (n <= 512) run_fwd<F32, Q, 1, 512>(A, st);
  else if (n <= 1024) run_fwd<F32, Q, 2, 512>(A, st);
  else if (n <= 2048) run_fwd<F32, Q, 2, 1024>(A, st);
  else run_fwd<F32, Q, 4, 1024>(A, st);
}

template <bool F32, int CH, int MAXT>
void run_bwd(const BwdArgs& A, int blocks, hipStream_t st) {
  SBN_LAUNCH("rmsnorm_grad", (rmsnorm_grad_kernel<F32, CH, MAXT>), dim3((unsigned)blocks),
             dim3((unsigned)threads_for(A.K / 8, CH)), 0, st, A);
}

template <bool F32>
void pick_bwd(const BwdArgs& A, int blocks, hipStream_t st) {
  const int n = A.K / 8;
  if (n <= 512) run_bwd<F32, 1, 512>(A, blocks, st);
  else if (n <= 1024) run_bwd<F32, 2, 512>(A, blocks, st);
  else if (n <= 2048) run_bwd<F32, 2, 1024>(A, blocks, st);
  else run_bwd<F32, 4, 1024>(A, blocks, st);
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

size_t rmsnorm_bwd_ws_bytes(int64_t T, int64_t K) { return align256((size_t)bwd_blocks(T, K) * (size_t)K * sizeof(float)); }

hipError_t launch_rmsnorm_backward(const void* dY, int64_t lddy, const void* H, int64_t ldh, const void* dH,
                                   int64_t lddh, bool f32, const void* gain, bool gain_f32, const float* rstd,
                                   int64_t T, int64_t K, void* dX, int64_t lddx, float* dgain, void* ws,
                                   hipStream_t st) {
  const int blocks = bwd_blocks(T, K);
  if (T > 0) {
    const BwdArgs A{dY, H, dH, gain, rstd, dX, (float*)ws, lddy, ldh, lddh, lddx, T, (int)K, gain_f32};
    if (f32) pick_bwd<true>(A, blocks, st);
    else pick_bwd<false>(A, blocks, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  SBN_LAUNCH("rmsnorm_dgain", rmsnorm_dgain_kernel, dim3((unsigned)cdiv(K, 16)), dim3(256), 0, st, (const float*)ws,
             blocks, (int)K, dgain);
  return hipGetLastError();
}

}  // namespace sbn
