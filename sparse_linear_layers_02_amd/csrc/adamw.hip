// AdamW over a table of tensors in one launch, states in 32 or in 8 bits.
//
//   m <- b1 m + (1-b1) g;  v <- b2 v + (1-b2) g^2
//   p <- p (1 - lr wd) - (lr / (1-b1^t)) m / (sqrt(v) / sqrt(1-b2^t) + eps)
//
// A block takes one chunk of one tensor (the map says which), a thread 8
// consecutive elements, so every stream moves in 8- and 16-byte accesses and
// the 32 lanes of half a wave hold exactly one block of 256 elements of an
// 8-bit state: its largest value is five lane exchanges away.
//
// 8-bit codes: m = s (c/127)|c/127|, v = s (c/255)^4 with s the block's largest
// value.  The code is the rint of a root, taken with the one-ulp root
// instruction: the estimate is off by at most 2 ulp below 256, under 2^-15.  If
// one of a thread's 8 estimates lies within 2^-14 of a half-integer, all 8 are
// taken again with correctly rounded roots, so the codes equal those of the
// correctly rounded formula.
//
// Products and sums are rounded one by one (no fused multiply-add): the result
// is that of the same formula in elementary float32 operations.
// Bound by memory traffic: 28 bytes an element with 32-bit parameters,
// gradients and states, 12 with bf16 parameters, float32 gradients and 8-bit
// states.  75.8 M elements, float32 with bf16 gradients and a bf16 copy (28
// bytes): 392 us, 5.4 TB/s; 135 M with 8-bit states (12 bytes): 318 to 360 us,
// up to 5.2 TB/s (1.11 GB fetched, 0.55 GB written); a state read back: 117 us,
// 5.8 TB/s.  A large copy reaches 4.9.
#include "train_internal.h"

#pragma clang fp contract(off)

namespace sbn {
namespace {

constexpr int QB = SBN_ADAMW_BLOCK;
constexpr float S_FLOOR = 0x1p-100f;                // a block whose largest value is smaller is all 0
constexpr float INV127 = 1.0f / 127.0f, INV255 = 1.0f / 255.0f;

__device__ inline float decode_m(int c, float s) {
  const float t = (float)c * INV127;
  return t * fabsf(t) * s;
}
__device__ inline float decode_v(int c, float s) {
  float t = (float)c * INV255;
  t = t * t;
  return t * t * s;
}

// Table entries hold plain pointers: into global memory, said so that the
// accesses are global ones (a flat access also waits in the LDS queue).
#define SBN_GLOBAL __attribute__((address_space(1)))
typedef SBN_GLOBAL const char gcchar;
typedef SBN_GLOBAL char gchar;
template <class T>
__device__ inline SBN_GLOBAL T* as_global(T* p) {
  return (SBN_GLOBAL T*)p;
}

// n (1..8) elements at p (16-byte aligned where n == 8); elements past n are 0
template <bool F32>
__device__ inline void load8(gcchar* p, int n, float* v) {
  if (F32) {
    SBN_GLOBAL const float* q = (SBN_GLOBAL const float*)p;
    if (n == 8) {
      *(v4f*)v = *(SBN_GLOBAL const v4f*)q;
      *(v4f*)(v + 4) = *(SBN_GLOBAL const v4f*)(q + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? q[i] : 0.0f;
    }
  } else {
    SBN_GLOBAL const uint16_t* q = (SBN_GLOBAL const uint16_t*)p;
    if (n == 8) {
      const v4i u = *(SBN_GLOBAL const v4i*)q;
      const uint32_t w[4] = {(uint32_t)u[0], (uint32_t)u[1], (uint32_t)u[2], (uint32_t)u[3]};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? bf16_to_f32(q[i]) : 0.0f;
    }
  }
}
template <bool F32>
__device__ inline void store8(gchar* p, int n, const float* v) {
  if (F32) {
    SBN_GLOBAL float* q = (SBN_GLOBAL float*)p;
    if (n == 8) {
      *(SBN_GLOBAL v4f*)q = *(const v4f*)v;
      *(SBN_GLOBAL v4f*)(q + 4) = *(const v4f*)(v + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) q[i] = v[i];
    }
  } else {
    SBN_GLOBAL uint16_t* q = (SBN_GLOBAL uint16_t*)p;
    if (n == 8) {
      *(SBN_GLOBAL v4i*)q = (v4i){(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3]),
                                  (int)pack_bf16x2(v[4], v[5]), (int)pack_bf16x2(v[6], v[7])};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) q[i] = (uint16_t)pack_bf16x2(v[i], 0.0f);   // as above, so that NaN stays NaN
    }
  }
}

// 8 codes of one byte
typedef int v2i __attribute__((ext_vector_type(2)));
__device__ inline uint2 load_codes(SBN_GLOBAL const uint8_t* p, int n) {
  if (n == 8) {
    const v2i w = *(SBN_GLOBAL const v2i*)p;
    return make_uint2((uint32_t)w[0], (uint32_t)w[1]);
  }
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}
__device__ inline void store_codes(SBN_GLOBAL uint8_t* p, int n, const int* c) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i >> 2] |= (uint32_t)(c[i] & 0xFF) << (8 * (i & 3));
  if (n == 8) {
    *(SBN_GLOBAL v2i*)p = (v2i){(int)w[0], (int)w[1]};
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
}
__device__ inline void unpack_codes(uint2 w, bool is_signed, int* c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = ((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xFFu;
    c[i] = is_signed ? (int)(int8_t)b : (int)b;
  }
}

// The larger of two magnitudes by their bits, where NaN is above Inf: a maximum
// of floats would drop a NaN.
struct MaxMagnitude {
  __device__ float operator()(float a, float b) const {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    return __uint_as_float(x > y ? x : y);
  }
};

// scale and codes of the 8 elements v of each lane (half a wave: one block).
// Lanes past the tensor hold zeros and take part in the maximum.  A NaN or Inf
// becomes the block's scale, and its values then decode to NaN or Inf.
template <bool SECOND>
__device__ inline float encode8(const float* v, int* c) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = MaxMagnitude{}(s, fabsf(v[i]));
  s = half_wave_all(s, MaxMagnitude{});
  if (s < S_FLOOR) s = 0.0f;
  const float inv = s > 0.0f ? 1.0f / s : 0.0f;
  float y[8], q[8], half = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = fminf(fabsf(v[i]) * inv, 1.0f);           // a number, also of Inf by Inf
    float r = __builtin_amdgcn_sqrtf(y[i]);
    if (SECOND) r = __builtin_amdgcn_sqrtf(r);
    q[i] = (SECOND ? 255.0f : 127.0f) * r;
    half = fmaxf(half, fabsf(q[i] - rintf(q[i])));
  }
  if (half > 0.5f - 0x1p-14f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = SECOND ? 255.0f * sqrtf(sqrtf(y[i])) : 127.0f * sqrtf(y[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = rintf(q[i]);
    // v > 0, not y > 0: the quotient may underflow
    c[i] = (int)(SECOND ? (v[i] > 0.0f && s > 0.0f ? fmaxf(r, 1.0f) : r) : copysignf(r, v[i]));
  }
  return s;
}

template <bool PF, bool GF, bool S8>
__global__ __launch_bounds__(256) void adamw_kernel(const sbn_adamw_entry* __restrict__ entries,
                                                    const int2* __restrict__ map, AdamWScalars S,
                                                    const float* __restrict__ dyn) {
  const int2 mp = map[blockIdx.x];
  const sbn_adamw_entry* E = entries + mp.x;
  const int64_t e = (int64_t)mp.y * ADAMW_CHUNK + threadIdx.x * 8;
  const int64_t left = E->n - e;
  const int n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
  float lr = S.lr, rate = S.rate, rbias2 = S.rbias2, gs = 1.0f;
  if (dyn) {
    lr = dyn[0];
    rate = lr / dyn[1];
    rbias2 = 1.0f / sqrtf(dyn[2]);
    gs = dyn[3];
  }
  const float keep = 1.0f - lr * E->weight_decay;

  float p[8], g[8], m[8], v[8];
  uint2 cm = make_uint2(0u, 0u), cv = cm;
  float sm = 0.0f, sv = 0.0f;
  if (n > 0) {
    load8<GF>(as_global((const char*)E->grad) + e * (GF ? 4 : 2), n, g);
    load8<PF>(as_global((const char*)E->p) + e * (PF ? 4 : 2), n, p);
    if (S8) {
      cm = load_codes(as_global((const uint8_t*)E->m) + e, n);
      cv = load_codes(as_global((const uint8_t*)E->v) + e, n);
      sm = as_global(E->m_scale)[e / QB];
      sv = as_global(E->v_scale)[e / QB];
    } else {
      load8<true>(as_global((const char*)E->m) + e * 4, n, m);
      load8<true>(as_global((const char*)E->v) + e * 4, n, v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = g[i] = m[i] = v[i] = 0.0f;
  }
  if (S8) {
    int c[8];
    unpack_codes(cm, true, c);
    if (sv == 0.0f) sm = 0.0f;                       // nothing to divide these m by
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = decode_m(c[i], sm);
    unpack_codes(cv, false, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = decode_v(c[i], sv);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float gi = g[i] * gs;
    m[i] = m[i] * S.beta1 + gi * S.one_minus_beta1;
    v[i] = v[i] * S.beta2 + (gi * gi) * S.one_minus_beta2;
    const float root = sqrtf(v[i]) * rbias2 + S.eps;
    p[i] = p[i] * keep - (m[i] * rate) / root;
  }
  if (S8) {
    int c[8];
    sm = encode8<false>(m, c);
    if (n > 0) store_codes(as_global((uint8_t*)E->m) + e, n, c);
    sv = encode8<true>(v, c);
    if (n > 0) store_codes(as_global((uint8_t*)E->v) + e, n, c);
    if (n > 0 && (threadIdx.x & 31) == 0) {
      as_global(E->m_scale)[e / QB] = sm;
      as_global(E->v_scale)[e / QB] = sv;
    }
  }
  if (n == 0) return;
  store8<PF>(as_global((char*)E->p) + e * (PF ? 4 : 2), n, p);
  if (PF && E->shadow) store8<false>(as_global((char*)E->shadow) + e * 2, n, p);
  if (!S8) {
    store8<true>(as_global((char*)E->m) + e * 4, n, m);
    store8<true>(as_global((char*)E->v) + e * 4, n, v);
  }
}

__global__ __launch_bounds__(256) void adamw_decode_kernel(const uint8_t* __restrict__ codes,
                                                           const float* __restrict__ scale, int64_t n, bool second,
                                                           float* __restrict__ out) {
  for (int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; e < n; e += (int64_t)gridDim.x * ADAMW_CHUNK) {
    const int k = n - e >= 8 ? 8 : (int)(n - e);
    const float s = scale[e / QB];
    int c[8];
    unpack_codes(load_codes(as_global(codes) + e, k), !second, c);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = second ? decode_v(c[i], s) : decode_m(c[i], s);
    store8<true>(as_global((char*)(out + e)), k, v);
  }
}

// rounds are the same for every lane of a wave: the maximum needs them all
__global__ __launch_bounds__(256) void adamw_encode_kernel(const float* __restrict__ x, int64_t n, bool second,
                                                           uint8_t* __restrict__ codes, float* __restrict__ scale) {
  for (int64_t e0 = (int64_t)blockIdx.x * ADAMW_CHUNK; e0 < n; e0 += (int64_t)gridDim.x * ADAMW_CHUNK) {
    const int64_t e = e0 + threadIdx.x * 8;
    const int k = n - e >= 8 ? 8 : n > e ? (int)(n - e) : 0;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (k > 0) load8<true>(as_global((const char*)(x + e)), k, v);
    int c[8];
    const float s = second ? encode8<true>(v, c) : encode8<false>(v, c);
    if (k > 0) {
      store_codes(as_global(codes) + e, k, c);
      if ((threadIdx.x & 31) == 0) scale[e / QB] = s;
    }
  }
}

dim3 stride_grid(int64_t n) {
  const int64_t b = cdiv(n, ADAMW_CHUNK);
  return dim3((unsigned)(b < (1 << 20) ? b : (1 << 20)));
}

template <bool PF, bool GF, bool S8>
void run(const sbn_adamw_entry* entries, const int2* map, int64_t blocks, const AdamWScalars& s, const float* dyn,
         hipStream_t st) {
  SBN_LAUNCH(S8 ? "adamw_8bit" : "adamw", (adamw_kernel<PF, GF, S8>), dim3((unsigned)blocks), dim3(256), 0, st, entries,
             map, s, dyn);
}

}  // namespace

hipError_t launch_adamw(const sbn_adamw_entry* entries, const int32_t* map, int64_t blocks, bool p_f32, bool g_f32,
                        bool state8, const AdamWScalars& s, const float* dyn, hipStream_t st) {
  // grids are limited to 2^32 threads: long tables take several launches
  constexpr int64_t PER = 1 << 23;
  for (int64_t b = 0; b < blocks; b += PER) {
    const int64_t nb = blocks - b < PER ? blocks - b : PER;
    const int2* mp = (const int2*)map + b;
    switch ((p_f32 ? 4 : 0) + (g_f32 ? 2 : 0) + (state8 ? 1 : 0)) {
      case 0: run<false, false, false>(entries, mp, nb, s, dyn, st); break;
      case 1: run<false, false, true>(entries, mp, nb, s, dyn, st); break;
      case 2: run<false, true, false>(entries, mp, nb, s, dyn, st); break;
      case 3: run<false, true, true>(entries, mp, nb, s, dyn, st); break;
      case 4: run<true, false, false>(entries, mp, nb, s, dyn, st); break;
      case 5: run<true, false, true>(entries, mp, nb, s, dyn, st); break;
      case 6: run<true, true, false>(entries, mp, nb, s, dyn, st); break;
      default: run<true, true, true>(entries, mp, nb, s, dyn, st); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_adamw_decode(const void* codes, const float* scale, int64_t n, bool second, float* out,
                               hipStream_t st) {
  SBN_LAUNCH("adamw_decode", adamw_decode_kernel, stride_grid(n), dim3(256), 0, st, (const uint8_t*)codes, scale, n,
             second, out);
  return hipGetLastError();
}

hipError_t launch_adamw_encode(const float* x, int64_t n, bool second, void* codes, float* scale, hipStream_t st) {
  SBN_LAUNCH("adamw_encode", adamw_encode_kernel, stride_grid(n), dim3(256), 0, st, x, n, second, (uint8_t*)codes,
             scale);
  return hipGetLastError();
}

}  // namespace sbn
