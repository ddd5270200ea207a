// What lies between the sparse layers in a training step, kept for the backward
// pass as int8 codes with a scale per 128 neighbours of a row: the RMS norm's
// input and the factors of a feed-forward block's activation.
//
//   checkpoint   s = a / 127, a = max |x| of the block, q = rint(127 x / a)
//   norm         u = x + residual, kept u; out: int8 codes of u gain, scale rstd max / 127
//   activation   u = f(a) b, kept a and b; out: the same of u, with or without the norm
//   gradient, from the kept values alone, with r = (mean u^2 + eps)^-1/2, w = gain dy:
//     du = r (w - u r^2 mean(w u));  dgain = sum_t dy u r;  da = du b f'(a);  db = du f(a)
//
// Both directions hold a row in registers as the plain norm does: one pass over
// memory, which bounds them (a large copy: 4.6 to 4.9 TB/s; rows partly in the Infinity
// Cache, which takes what was written last, go above it).  In bf16 with 8192 rows,
// everything kept: the norm of 4096 with a residual 49 to 54 us (5.0 to 5.5 TB/s), its
// gradient 44 to 48 (4.9 to 5.3); the activation of 11008, gated and normed, 142 to 154
// (4.1 to 4.5; 95 to 107 without keeping; with ROW_SILU 152 to 168), its gradient 143 to
// 152.  A checkpoint's block is 16 threads of 8 elements, one row of lanes, so that its
// maximum takes four lane exchanges and no memory.
#include "keep_internal.h"
#include "once_per_device.h"
#include "row_ops.h"

namespace sbn {
namespace {

constexpr int LANES = SBN_KEEP_BLOCK / 8;            // threads of a checkpoint's block
static_assert(LANES == 16, "a block is one row of lanes");
constexpr float LARGEST_SCALE = 0x1.020406p121f;     // the next one's 127-fold rounds to Inf, and so may a / 127's

template <int CTRL>
__device__ inline uint32_t row_move_bits(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xf, 0xf, true);
}
// max |x| of a block: as integers the bits of magnitudes order alike, NaN above all
__device__ inline float block_max(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  m = max(m, row_move_bits<0xB1>(m));                // as row16_all
  m = max(m, row_move_bits<0x4E>(m));
  m = max(m, row_move_bits<0x141>(m));
  m = max(m, row_move_bits<0x140>(m));
  return __uint_as_float(m);
}

// Chunk c of row t into a checkpoint of rows of K; all 16 lanes of a block come
// here, with zeros past the row.  A maximum that is NaN or Inf makes the scale, and so
// every value, NaN.  BF16: the values are.
template <bool BF16>
__device__ inline void keep_chunk(const float* v, bool live, int64_t t, int c, int K, int nb, int8_t* codes,
                                  float* scales) {
  const float a = block_max(v);
  const bool none = a < U_FLOOR;
  const float rcp = none ? 0.0f : __builtin_amdgcn_rcpf(a * (1.0f / 127.0f));
  if (live) {
    *(uint2*)(codes + t * K + 8 * c) = BF16 ? codes8_bf16(v, rcp) : codes8(v, rcp, a);
    if ((c & (LANES - 1)) == 0)                      // Inf - Inf: NaN
      scales[t * nb + c / LANES] = none ? 0.0f : fminf(a / 127.0f, LARGEST_SCALE) + (a - a);
  }
}

__device__ inline void values8(uint2 q, float s, float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = (float)(int8_t)(q.x >> (8 * j)) * s;
    v[4 + j] = (float)(int8_t)(q.y >> (8 * j)) * s;
  }
}

// ---------------------------------------------------------------- checkpoints alone
// (bf16, 8192 x 11008: encode 44 us, decode 47 to 51, 5.3 to 6.2 TB/s; float32 82 and 113)
// Rows of `lanes` threads (a multiple of 16), one after the other; `rows` of a
// launch keep their number of threads below 2^31.
template <bool F32>
__global__ __launch_bounds__(256) void keep8_encode_kernel(const char* __restrict__ X, int64_t ldx, uint32_t rows,
                                                           int K, uint32_t lanes, int8_t* __restrict__ codes,
                                                           float* __restrict__ scales) {
  const uint32_t n = K / 8, nb = lanes / LANES, total = rows * lanes;
  // whole rows of 16 lanes share a row of X, so all lanes of a block take the same rounds
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
    const uint32_t t = i / lanes, c = i - t * lanes;
    float v[8] = {};
    if (c < n) {
      Vec8<F32> x;
      x.load(X + (int64_t)t * ldx * (F32 ? 4 : 2), c);
      x.to(v);
    }
    keep_chunk<!F32>(v, c < n, t, (int)c, K, (int)nb, codes, scales);
  }
}

template <bool F32>
__global__ __launch_bounds__(256) void keep8_decode_kernel(const int8_t* __restrict__ codes,
                                                           const float* __restrict__ scales, uint32_t rows, int K,
                                                           char* __restrict__ Y, int64_t ldy) {
  const uint32_t n = K / 8, nb = (n + LANES - 1) / LANES, total = rows * n;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
    const uint32_t t = i / n, c = i - t * n;
    float v[8];
    values8(*(const uint2*)(codes + 8 * (int64_t)i), scales[(int64_t)t * nb + c / LANES], v);
    Vec8<F32> y;
    y.from(v);
    y.store(Y + (int64_t)t * ldy * (F32 ? 4 : 2), c);
  }
}

// ---------------------------------------------------------------- the functions
enum RowOp { ROW_NORM, ROW_RELU2, ROW_SILU };        // ROW_NORM: u = x

// 1 / (1 + exp(-a)), the exponential by the base-2 instruction, with what the exponent's
// rounding left and the constant's: within 3 units of 2^-24; where it is Inf, 0
__device__ inline float sigmoid(float a) {
  constexpr float L = -1.44269502f, LOW = -1.925963033e-8f;
  a = fminf(a, 256.0f);                              // of more the product overflows, and 0 Inf is no exponential
  const float z = a * L, low = fmaf(a, LOW, fmaf(a, L, -z));
  const float e = __builtin_amdgcn_exp2f(z) * fmaf(low, 0.6931471806f, 1.0f);
  return __builtin_amdgcn_rcpf(1.0f + e);
}
// f(a), given ROW_SILU's sigmoid g, and, if asked, f'(a)
template <RowOp OP>
__device__ inline float act(float a, float g, float* slope = nullptr) {
  if (OP == ROW_RELU2) {
    const float r = fmaxf(a, 0.0f);
    if (slope) *slope = 2.0f * r;
    return r * r;
  }
  if (OP == ROW_SILU) {
    if (slope) *slope = g * (1.0f + a * (1.0f - g));
    return a * g;
  }
  if (slope) *slope = 1.0f;
  return a;
}
template <RowOp OP>
__device__ inline float act(float a, float* slope = nullptr) {
  return act<OP>(a, OP == ROW_SILU ? sigmoid(a) : 0.0f, slope);
}

// sums or maxima of a row's waves, from LDS `red` of its own; all threads call it
template <class Op>
__device__ inline float across(const float* red, int waves, Op op) {
  const int l = threadIdx.x & 15;                    // at most 16 waves
  return row16_all(l < waves ? red[l] : 0.0f, op);
}

// ---------------------------------------------------------------- forward
struct FwdArgs {
  const void *A, *B, *gain;                          // B: the residual (ROW_NORM), the factor, or NULL
  void* H;                                           // ROW_NORM with a residual
  int8_t *Xq, *kA, *kB;
  float *s_x, *sA, *sB;
  int64_t lda, ldb, ldh, T;
  int K;
  float eps;
  bool gain_f32;
};

// A block holds one row at a time, CH chunks of 8 elements per thread
// (CH * blockDim.x * 8 >= K); rows beyond the grid are taken in further rounds.
template <bool F32, RowOp OP, int CH, int MAXT>
__global__ __launch_bounds__(MAXT) void kept_forward_kernel(FwdArgs P) {
  __shared__ float red[2][2][MAXT / 64];
  const int g = threadIdx.x, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int n = P.K / 8, es = F32 ? 4 : 2, TPR = blockDim.x, nb = (n + LANES - 1) / LANES;
  int turn = 0;
  for (int64_t t = blockIdx.x; t < P.T; t += gridDim.x, turn ^= 1) {
    const char* ar = (const char*)P.A + t * P.lda * es;
    const char* br = (const char*)P.B + t * P.ldb * es;
    Vec8<F32> a[CH], b[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (g + TPR * i < n) {
        a[i].load(ar, g + TPR * i);
        if (P.B) b[i].load(br, g + TPR * i);
      }
    float v[CH][8];                                  // u, then u gain
    float ss = 0.0f, mx = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = g + TPR * i;
      const bool live = c < n;
      float x[8] = {}, y[8] = {}, gain[8];
      if (live) {
        a[i].to(x);
        if (P.B) b[i].to(y);
        if (P.gain) gain8(P.gain, P.gain_f32, c, gain);
      }
      if (OP == ROW_NORM) {
        if (live && P.B) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] += y[j];
          a[i].from(x);
          a[i].store((char*)P.H + t * P.ldh * es, c);
          if (!F32) a[i].to(x);                      // the stored h is what is normalised
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = x[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[i][j] = act<OP>(x[j]);
          if (P.B) v[i][j] *= y[j];
        }
      }
      if (P.kA) {
        keep_chunk<!F32>(x, live, t, c, P.K, nb, P.kA, P.sA);
        if (OP != ROW_NORM && P.B) keep_chunk<!F32>(y, live, t, c, P.K, nb, P.kB, P.sB);
      }
      if (live) {
        if (P.gain) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            ss += v[i][j] * v[i][j];
            v[i][j] *= gain[j];
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(v[i][j]));
      }
    }
    ss = wave_all(ss, Add{});
    mx = wave_all(mx, Max{});
    if (waves > 1) {
      // two sets of red in turn: one barrier a round keeps a fast wave's next
      // write away from a slow wave's read
      if ((threadIdx.x & 63) == 0) red[turn][0][wave] = ss, red[turn][1][wave] = mx;
      __syncthreads();
      ss = across(red[turn][0], waves, Add{});
      mx = across(red[turn][1], waves, Max{});
    }
    const float m = fmaxf(mx, U_FLOOR);
    if (g == 0) {
      const float rstd = P.gain ? 1.0f / sqrtf(ss / (float)P.K + P.eps) : 1.0f;
      P.s_x[t] = (m * rstd) / 127.0f;
    }
    const float rcp = __builtin_amdgcn_rcpf(m * (1.0f / 127.0f));
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = g + TPR * i;
      if (c < n) *(uint2*)(P.Xq + t * P.K + 8 * c) = codes8(v[i], rcp, m);
    }
  }
}

// Rows that do not fit the registers: read twice, the second time from the cache, chunk
// by chunk.  (Holding four chunks a thread spilled up to half of them: 4096 x 20480, gated,
// normed and kept, 289 us; so 154.)  The norm's threads and order of sums are the plain
// norm's.
template <bool F32, RowOp OP>
__global__ __launch_bounds__(1024) void kept_forward_wide_kernel(FwdArgs P) {
  __shared__ float red[2][2][16];
  const int g = threadIdx.x, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int n = P.K / 8, es = F32 ? 4 : 2, TPR = blockDim.x, nb = (n + LANES - 1) / LANES;
  const int all = (n + 63) / 64 * 64;                // whole waves take each round, for the blocks' maxima
  int turn = 0;
  for (int64_t t = blockIdx.x; t < P.T; t += gridDim.x, turn ^= 1) {
    const char* ar = (const char*)P.A + t * P.lda * es;
    const char* br = (const char*)P.B + t * P.ldb * es;
    char* hr = (char*)P.H + t * P.ldh * es;
    // what is normalised, of chunk c, from a and b
    auto make = [&](const Vec8<F32>& a, const Vec8<F32>& b, float* x, float* y, float* v) {
      a.to(x);
      if (OP == ROW_NORM) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = x[j];
        return;
      }
      if (P.B) b.to(y);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = act<OP>(x[j]);
        if (P.B) v[j] *= y[j];
      }
    };
    float ss = 0.0f, mx = 0.0f;
    for (int c = g; c < all; c += TPR) {
      const bool live = c < n;
      float x[8] = {}, y[8] = {}, v[8], gain[8];
      if (live) {
        Vec8<F32> a, b;
        a.load(ar, c);
        if (P.B) b.load(br, c);
        if (P.gain) gain8(P.gain, P.gain_f32, c, gain);
        if (OP == ROW_NORM && P.B) {
          a.to(x), b.to(y);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] += y[j];
          a.from(x);
          a.store(hr, c);
        }
        make(a, b, x, y, v);
        if (P.gain) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            ss += v[j] * v[j];
            v[j] *= gain[j];
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(v[j]));
      }
      if (P.kA) {
        keep_chunk<!F32>(x, live, t, c, P.K, nb, P.kA, P.sA);
        if (OP != ROW_NORM && P.B) keep_chunk<!F32>(y, live, t, c, P.K, nb, P.kB, P.sB);
      }
    }
    ss = wave_all(ss, Add{});
    mx = wave_all(mx, Max{});
    if ((threadIdx.x & 63) == 0) red[turn][0][wave] = ss, red[turn][1][wave] = mx;
    __syncthreads();                                 // and the other set of red for the next round
    ss = across(red[turn][0], waves, Add{});
    mx = across(red[turn][1], waves, Max{});
    const float m = fmaxf(mx, U_FLOOR);
    if (g == 0) {
      const float rstd = P.gain ? 1.0f / sqrtf(ss / (float)P.K + P.eps) : 1.0f;
      P.s_x[t] = (m * rstd) / 127.0f;
    }
    const float rcp = __builtin_amdgcn_rcpf(m * (1.0f / 127.0f));
    for (int c = g; c < n; c += TPR) {
      float x[8], y[8], v[8], gain[8];
      Vec8<F32> a, b;
      a.load(OP == ROW_NORM && P.B ? hr : ar, c);    // h by the thread that wrote it (it may be in an input's place)
      if (OP != ROW_NORM && P.B) b.load(br, c);
      make(a, b, x, y, v);
      if (P.gain) {
        gain8(P.gain, P.gain_f32, c, gain);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= gain[j];
      }
      *(uint2*)(P.Xq + t * P.K + 8 * c) = codes8(v, rcp, m);
    }
  }
}

// ---------------------------------------------------------------- backward
struct BwdArgs {
  const void *dY, *dH, *gain;                        // dH: ROW_NORM, or NULL
  const int8_t *kA, *kB;                             // kB NULL: no second factor
  const float *sA, *sB;
  void *dA, *dB;
  float* part;                                       // [gridDim.x][K] partial sums of dgain
  int64_t lddy, lddh, ldda, lddb, T;
  int K;
  float eps;
  bool gain_f32;
};

// What the gradient reads of a row, CH chunks of a thread.
template <bool F32, RowOp OP, int CH>
struct KeptRow {
  Vec8<F32> dy[CH], dh[OP == ROW_NORM ? CH : 1];
  uint2 qa[CH], qb[CH];
  float sa[CH], sb[CH];
  __device__ void load(const BwdArgs& P, int64_t t, int nb) {
    const int n = P.K / 8, es = F32 ? 4 : 2;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + blockDim.x * i;
      if (c < n) {
        dy[i].load((const char*)P.dY + t * P.lddy * es, c);
        qa[i] = *(const uint2*)(P.kA + t * P.K + 8 * c);
        sa[i] = P.sA[t * nb + c / LANES];
        if (OP == ROW_NORM) {
          if (P.dH) dh[i].load((const char*)P.dH + t * P.lddh * es, c);
        } else if (P.kB) {
          qb[i] = *(const uint2*)(P.kB + t * P.K + 8 * c);
          sb[i] = P.sB[t * nb + c / LANES];
        }
      }
    }
  }
};

// A row is loaded while the one before it is worked on.  Without a gain a block has a
// row, unless there are more than GRID_MAX: nothing is summed over rows, and no wave
// waits for another (8192 x 11008 bf16, ROW_SILU, gated: 129 us, 5.6 TB/s; as many
// blocks as fit at once, rows ahead: 151).  Normed, ROW_RELU2 143 to 152 us, 4.8 to 5.1 TB/s;
// ROW_SILU 192, by its exponentials.  ROW_SILU's sigmoids are kept from
// the sums to the gradients, up to two chunks a thread (8192 x 11008 bf16, gated and
// normed 221 -> 195 us; with four, float32 rows spilled: 182 -> 276).
template <bool F32, RowOp OP, int CH, int MAXT, bool GAIN>
__global__ __launch_bounds__(MAXT) void kept_backward_kernel(BwdArgs P) {
  __shared__ float red[2][2][MAXT / 64];
  const int g = threadIdx.x, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int n = P.K / 8, es = F32 ? 4 : 2, TPR = blockDim.x, nb = (n + LANES - 1) / LANES;
  // true wherever GAIN is, but asked: with it known the schedule of ROW_RELU2's bf16 rows takes 5 to 10% longer
  const bool normed = GAIN && P.gain;
  float dg[CH][8], kept_gain[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = 0.0f;
  if (normed) {
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (g + TPR * i < n) gain8(P.gain, P.gain_f32, g + TPR * i, kept_gain[i]);
  }
  constexpr bool KEEP = GAIN && OP == ROW_SILU && CH <= 2;
  float sig[KEEP ? CH : 1][8];
  int turn = 0;
  KeptRow<F32, OP, CH> row, next;
  next.load(P, blockIdx.x, nb);
  for (int64_t t = blockIdx.x; t < P.T; t += gridDim.x, turn ^= 1) {
    row = next;
    if (GAIN) next.load(P, t + gridDim.x < P.T ? t + gridDim.x : t, nb);
    else if (t + gridDim.x < P.T) next.load(P, t + gridDim.x, nb);
    float r = 1.0f, back = 0.0f;                     // back: r^2 mean(w u)
    if (normed) {
      float uu = 0.0f, wu = 0.0f;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = g + TPR * i;
        if (c < n) {
          float a[8], b[8], w[8], *gain = kept_gain[i];
          values8(row.qa[i], row.sa[i], a);
          if (OP != ROW_NORM && P.kB) values8(row.qb[i], row.sb[i], b);
          row.dy[i].to(w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (KEEP) sig[i][j] = sigmoid(a[j]);
            float u = KEEP ? act<OP>(a[j], sig[i][j]) : act<OP>(a[j]);
            if (OP != ROW_NORM && P.kB) u *= b[j];
            uu += u * u;
            wu += w[j] * gain[j] * u;
          }
        }
      }
      uu = wave_all(uu, Add{});
      wu = wave_all(wu, Add{});
      if (waves > 1) {
        if ((threadIdx.x & 63) == 0) red[turn][0][wave] = uu, red[turn][1][wave] = wu;
        __syncthreads();                             // and the other set of red for the next round
        uu = across(red[turn][0], waves, Add{});
        wu = across(red[turn][1], waves, Add{});
      }
      r = 1.0f / sqrtf(uu / (float)P.K + P.eps);
      back = r * r * (wu / (float)P.K);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = g + TPR * i;
      if (c < n) {
        float a[8], b[8], d[8], da[8], db[8], *gain = kept_gain[i];
        values8(row.qa[i], row.sa[i], a);
        if (OP != ROW_NORM && P.kB) values8(row.qb[i], row.sb[i], b);
        row.dy[i].to(d);
        if (OP == ROW_NORM && P.dH) row.dh[i].to(db);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float slope;
          const float f = KEEP ? act<OP>(a[j], sig[i][j], &slope) : act<OP>(a[j], &slope);
          float du = d[j];
          if (normed) {
            const float u = OP != ROW_NORM && P.kB ? f * b[j] : f;
            dg[i][j] += d[j] * (u * r);
            du = r * (d[j] * gain[j] - u * back);
          }
          if (OP == ROW_NORM) {
            da[j] = P.dH ? du + db[j] : du;
          } else {
            da[j] = (P.kB ? du * b[j] : du) * slope;
            db[j] = du * f;
          }
        }
        Vec8<F32> o;
        o.from(da);
        o.store((char*)P.dA + t * P.ldda * es, c);
        if (OP != ROW_NORM && P.kB) {
          o.from(db);
          o.store((char*)P.dB + t * P.lddb * es, c);
        }
      }
    }
  }
  if (!normed) return;
  float* out = P.part + (int64_t)blockIdx.x * P.K;
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

// Rows of more than 2048 chunks (float32 ones of the norm: 1536): read twice, and dgain's sums in LDS.
template <bool F32, RowOp OP>
__global__ __launch_bounds__(1024) void kept_backward_wide_kernel(BwdArgs P) {
  __shared__ float red[2][2][16];
  extern __shared__ v4f sums[];                      // [2][n] with a gain: each thread its own columns
  const int g = threadIdx.x, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int n = P.K / 8, nb = (n + LANES - 1) / LANES, TPR = blockDim.x, es = F32 ? 4 : 2;
  const bool two = OP != ROW_NORM && P.kB;
  if (P.gain)
    for (int c = g; c < n; c += TPR) sums[c] = sums[n + c] = (v4f){0.f, 0.f, 0.f, 0.f};
  int turn = 0;
  for (int64_t t = blockIdx.x; t < P.T; t += gridDim.x, turn ^= 1) {
    auto load = [&](int c, float* a, float* b, float* d) {
      Vec8<F32> dy;
      dy.load((const char*)P.dY + t * P.lddy * es, c);
      values8(*(const uint2*)(P.kA + t * P.K + 8 * c), P.sA[t * nb + c / LANES], a);
      if (two) values8(*(const uint2*)(P.kB + t * P.K + 8 * c), P.sB[t * nb + c / LANES], b);
      dy.to(d);
    };
    float r = 1.0f, back = 0.0f;                     // back: r^2 mean(w u)
    if (P.gain) {
      float uu = 0.0f, wu = 0.0f;
      for (int c = g; c < n; c += TPR) {
        float a[8], b[8], w[8], gain[8];
        load(c, a, b, w);
        gain8(P.gain, P.gain_f32, c, gain);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float u = act<OP>(a[j]);
          if (two) u *= b[j];
          uu += u * u;
          wu += w[j] * gain[j] * u;
        }
      }
      uu = wave_all(uu, Add{});
      wu = wave_all(wu, Add{});
      if ((threadIdx.x & 63) == 0) red[turn][0][wave] = uu, red[turn][1][wave] = wu;
      __syncthreads();                               // and the other set of red for the next round
      uu = across(red[turn][0], waves, Add{});
      wu = across(red[turn][1], waves, Add{});
      r = 1.0f / sqrtf(uu / (float)P.K + P.eps);
      back = r * r * (wu / (float)P.K);
    }
    for (int c = g; c < n; c += TPR) {
      float a[8], b[8], d[8], gain[8], da[8], db[8];
      v4f dg[2];
      load(c, a, b, d);
      if (P.gain) {
        gain8(P.gain, P.gain_f32, c, gain);
        dg[0] = sums[c], dg[1] = sums[n + c];
      }
      if (OP == ROW_NORM && P.dH) {
        Vec8<F32> dh;
        dh.load((const char*)P.dH + t * P.lddh * es, c);
        dh.to(db);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float slope;
        const float f = act<OP>(a[j], &slope);
        float du = d[j];
        if (P.gain) {
          const float u = two ? f * b[j] : f;
          dg[j >> 2][j & 3] += d[j] * (u * r);
          du = r * (d[j] * gain[j] - u * back);
        }
        if (OP == ROW_NORM) {
          da[j] = P.dH ? du + db[j] : du;
        } else {
          da[j] = (two ? du * b[j] : du) * slope;
          db[j] = du * f;
        }
      }
      if (P.gain) sums[c] = dg[0], sums[n + c] = dg[1];
      Vec8<F32> o;
      o.from(da);
      o.store((char*)P.dA + t * P.ldda * es, c);
      if (two) {
        o.from(db);
        o.store((char*)P.dB + t * P.lddb * es, c);
      }
    }
  }
  if (!P.gain) return;
  v4f* out = (v4f*)(P.part + (int64_t)blockIdx.x * P.K);
  for (int c = g; c < n; c += TPR) out[2 * c] = sums[c], out[2 * c + 1] = sums[n + c];
}

constexpr int64_t GRID_MAX = 1 << 20;                // blocks; rows beyond are taken in further rounds

template <bool F32, RowOp OP, int CH, int MAXT>
void run_fwd(const char* name, const FwdArgs& P, hipStream_t st) {
  SBN_LAUNCH(name, (kept_forward_kernel<F32, OP, CH, MAXT>), dim3((unsigned)(P.T < GRID_MAX ? P.T : GRID_MAX)),
             dim3((unsigned)threads_for(P.K / 8, CH)), 0, st, P);
}
// The norm goes by the plain norm's threads, so that its sums have the same order and its
// scales the same bits.  The activation takes up to 512 threads and more chunks, of which
// two blocks are on a unit (8192 x 11008, gated, normed and kept: 160 us; 704 threads, one
// block: 193), and above 1536 chunks reads twice (4096 x 16384: 123 us; four chunks held:
// 143), with 512 threads (256 / 512 / 768 / 1024: 128 / 123 / 124 / 123; 4096 x 20480 163 / 154
// / 156 / 154).  How many depends on K alone, so a row gives the same bits in any batch.
template <bool F32, RowOp OP>
void pick_fwd(const char* name, const FwdArgs& P, hipStream_t st) {
  const int n = P.K / 8;
  if (n <= 512) run_fwd<F32, OP, 1, 512>(name, P, st);
  else if (n <= 1024) run_fwd<F32, OP, 2, 512>(name, P, st);
  else if (n <= (OP == ROW_NORM ? 2048 : 1536)) run_fwd<F32, OP, OP == ROW_NORM ? 2 : 3, OP == ROW_NORM ? 1024 : 512>(name, P, st);
  else
    SBN_LAUNCH(name, (kept_forward_wide_kernel<F32, OP>), dim3((unsigned)(P.T < GRID_MAX ? P.T : GRID_MAX)),
               dim3((unsigned)(OP == ROW_NORM ? threads_for(n, 4) : 512)), 0, st, P);
}

// Threads of a gradient's block, and blocks with a row of partial sums of dgain each: as
// many as are on the machine at once (16 waves of a unit, one block of more than 8; of four
// chunks a thread, with 225 to 256 registers, 8 waves), but at least 8 rows a block where that
// leaves one a unit, since a block's partial costs as much traffic as two rows in 16 bits.
// (4096 x 14344 with a gain, bf16 and float32, one block a unit and two, with the sum of the
// partials: norm 89 and 101 us, 209 and 223; relu^2 107 and 118, 178 and 190; SiLU 133 and 143, 210 and 222.)
int bwd_chunks(int n) { return n <= 1024 ? 1 : n <= 1536 ? 2 : 4; }   // above 2048: of 1024 threads, in rounds
int bwd_blocks(int64_t T, int64_t K) {
  const int n = (int)(K / 8), waves = threads_for(n, bwd_chunks(n)) / 64, most = n > 1536 ? 256 : 256 * (16 / waves);
  int64_t g = T / 8 < 256 ? 256 : T / 8;
  if (g > most) g = most;
  return (int)(g < T ? g : T);
}

template <bool F32, RowOp OP, int CH, int MAXT>
void run_bwd(const char* name, const BwdArgs& P, hipStream_t st) {
  const dim3 threads((unsigned)threads_for(P.K / 8, CH));
  if (OP == ROW_NORM || P.gain)
    SBN_LAUNCH(name, (kept_backward_kernel<F32, OP, CH, MAXT, true>), dim3((unsigned)bwd_blocks(P.T, P.K)), threads, 0, st, P);
  else
    SBN_LAUNCH(name, (kept_backward_kernel<F32, OP, CH, MAXT, OP == ROW_NORM>),
               dim3((unsigned)(P.T < GRID_MAX ? P.T : GRID_MAX)), threads, 0, st, P);
}
template <bool F32, RowOp OP>
hipError_t run_bwd_wide(const char* name, const BwdArgs& P, hipStream_t st) {
  static OncePerDevice once;
  int device = 0;
  hipError_t e = hipGetDevice(&device);
  if (e == hipSuccess)
    e = once(device, [] {
      return hipFuncSetAttribute((const void*)kept_backward_wide_kernel<F32, OP>,
                                 hipFuncAttributeMaxDynamicSharedMemorySize, SBN_RMSNORM_MAX_K * (int)sizeof(float));
    });
  if (e != hipSuccess) return e;
  const int64_t blocks = P.gain ? bwd_blocks(P.T, P.K) : P.T < GRID_MAX ? P.T : GRID_MAX;
  SBN_LAUNCH(name, (kept_backward_wide_kernel<F32, OP>), dim3((unsigned)blocks), dim3(1024),
             P.gain ? (size_t)P.K * sizeof(float) : 0, st, P);
  return hipGetLastError();
}
// Above 1536 chunks float32 rows of the norm are read twice: held, 24 of their registers
// were spilled (600 x 14344: 28 us, held 38; 4096 x 14344 201 and 202).  Those of the activation are held
// all the same, with 2 (relu^2) and 8 (SiLU) spilled where there is a gain (4096 x 14344: 170 and 203 us,
// 5.0 and 4.2 TB/s; read twice 218 and 227; 600 x 14344 32 and 41, 34 and 37), and so are bf16 ones, which
// do not spill (norm 82, read twice 112).
template <bool F32, RowOp OP>
hipError_t pick_bwd(const char* name, const BwdArgs& P, hipStream_t st) {
  const int n = P.K / 8;
  if (n <= 512) run_bwd<F32, OP, 1, 512>(name, P, st);
  else if (n <= 1024) run_bwd<F32, OP, 1, 1024>(name, P, st);
  else if (n <= 1536) run_bwd<F32, OP, 2, 768>(name, P, st);
  else if constexpr (F32 && OP == ROW_NORM) return run_bwd_wide<F32, OP>(name, P, st);
  else if (n <= 2048) run_bwd<F32, OP, 4, 512>(name, P, st);
  else return run_bwd_wide<F32, OP>(name, P, st);
  return hipGetLastError();
}

template <RowOp OP>
hipError_t backward(const char* name, const BwdArgs& P, bool f32, float* dgain, hipStream_t st) {
  if (P.T > 0) {
    const hipError_t e = f32 ? pick_bwd<true, OP>(name, P, st) : pick_bwd<false, OP>(name, P, st);
    if (e != hipSuccess) return e;
  }
  return dgain ? launch_norm_dgain(P.part, bwd_blocks(P.T, P.K), P.K, dgain, st) : hipSuccess;
}

// Rows of a launch of the checkpoints' own kernels: their threads stay below 2^31.
int64_t slab_rows(int64_t lanes) { return ((int64_t(1) << 31) - (int64_t(1) << 24)) / lanes; }
unsigned slab_grid(int64_t threads) {
  const int64_t b = cdiv(threads, 256);
  return (unsigned)(b < 16384 ? b : 16384);
}

}  // namespace

size_t kept_bwd_ws_bytes(int64_t T, int64_t K) { return align256((size_t)bwd_blocks(T, K) * (size_t)K * sizeof(float)); }

hipError_t launch_keep8_encode(const void* X, int64_t ldx, bool f32, int64_t T, int64_t K, int8_t* codes, float* scales,
                               hipStream_t st) {
  const int64_t nb = cdiv(K, SBN_KEEP_BLOCK), lanes = nb * LANES, slab = slab_rows(lanes), es = f32 ? 4 : 2;
  for (int64_t t = 0; t < T; t += slab) {
    const int64_t rows = T - t < slab ? T - t : slab;
    const char* x = (const char*)X + t * ldx * es;
    const dim3 grid(slab_grid(rows * lanes));
    if (f32) SBN_LAUNCH("keep8_encode", keep8_encode_kernel<true>, grid, dim3(256), 0, st, x, ldx, (uint32_t)rows, (int)K, (uint32_t)lanes, codes + t * K, scales + t * nb);
    else SBN_LAUNCH("keep8_encode", keep8_encode_kernel<false>, grid, dim3(256), 0, st, x, ldx, (uint32_t)rows, (int)K, (uint32_t)lanes, codes + t * K, scales + t * nb);
  }
  return hipGetLastError();
}

hipError_t launch_keep8_decode(const int8_t* codes, const float* scales, int64_t T, int64_t K, void* Y, int64_t ldy,
                               bool f32, hipStream_t st) {
  const int64_t nb = cdiv(K, SBN_KEEP_BLOCK), slab = slab_rows(K / 8), es = f32 ? 4 : 2;
  for (int64_t t = 0; t < T; t += slab) {
    const int64_t rows = T - t < slab ? T - t : slab;
    char* y = (char*)Y + t * ldy * es;
    const dim3 grid(slab_grid(rows * (K / 8)));
    if (f32) SBN_LAUNCH("keep8_decode", keep8_decode_kernel<true>, grid, dim3(256), 0, st, codes + t * K, scales + t * nb, (uint32_t)rows, (int)K, y, ldy);
    else SBN_LAUNCH("keep8_decode", keep8_decode_kernel<false>, grid, dim3(256), 0, st, codes + t * K, scales + t * nb, (uint32_t)rows, (int)K, y, ldy);
  }
  return hipGetLastError();
}

hipError_t launch_rmsnorm_quant_keep(const void* X, int64_t ldx, const void* res, int64_t ldr, bool f32, const void* gain,
                                     bool gain_f32, int64_t T, int64_t K, float eps, void* H, int64_t ldh, int8_t* Xq,
                                     float* s_x, int8_t* codes, float* scales, hipStream_t st) {
  const FwdArgs P{X, res, gain, H, Xq, codes, nullptr, s_x, scales, nullptr, ldx, ldr, ldh, T, (int)K, eps, gain_f32};
  if (f32) pick_fwd<true, ROW_NORM>("rmsnorm_quant_keep", P, st);
  else pick_fwd<false, ROW_NORM>("rmsnorm_quant_keep", P, st);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_backward_kept(const void* dY, int64_t lddy, const void* dH, int64_t lddh, bool f32,
                                        const int8_t* codes, const float* scales, const void* gain, bool gain_f32,
                                        int64_t T, int64_t K, float eps, void* dX, int64_t lddx, float* dgain, void* ws,
                                        hipStream_t st) {
  const BwdArgs P{dY, dH, gain, codes, nullptr, scales, nullptr, dX, nullptr, (float*)ws, lddy, lddh, lddx, 0, T, (int)K,
                  eps, gain_f32};
  return backward<ROW_NORM>("rmsnorm_grad_kept", P, f32, dgain, st);
}

hipError_t launch_activation_quant(const void* A, int64_t lda, const void* B, int64_t ldb, bool f32, sbn_act act,
                                   const void* gain, bool gain_f32, int64_t T, int64_t K, float eps, int8_t* Xq,
                                   float* s_x, int8_t* codes_a, float* scales_a, int8_t* codes_b, float* scales_b,
                                   hipStream_t st) {
  const FwdArgs P{A, B, gain, nullptr, Xq, codes_a, codes_b, s_x, scales_a, scales_b, lda, ldb, 0, T, (int)K, eps, gain_f32};
  const char* name = "activation_quant";
  if (act == SBN_RELU2) {
    if (f32) pick_fwd<true, ROW_RELU2>(name, P, st);
    else pick_fwd<false, ROW_RELU2>(name, P, st);
  } else {
    if (f32) pick_fwd<true, ROW_SILU>(name, P, st);
    else pick_fwd<false, ROW_SILU>(name, P, st);
  }
  return hipGetLastError();
}

hipError_t launch_activation_backward(const void* dY, int64_t lddy, bool f32, const int8_t* codes_a,
                                      const float* scales_a, const int8_t* codes_b, const float* scales_b, sbn_act act,
                                      const void* gain, bool gain_f32, int64_t T, int64_t K, float eps, void* dA,
                                      int64_t ldda, void* dB, int64_t lddb, float* dgain, void* ws, hipStream_t st) {
  const BwdArgs P{dY, nullptr, gain, codes_a, codes_b, scales_a, scales_b, dA, dB, (float*)ws, lddy, 0, ldda, lddb, T,
                  (int)K, eps, gain_f32};
  const char* name = "activation_grad";
  return act == SBN_RELU2 ? backward<ROW_RELU2>(name, P, f32, dgain, st) : backward<ROW_SILU>(name, P, f32, dgain, st);
}

}  // namespace sbn
