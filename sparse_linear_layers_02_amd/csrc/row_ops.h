// What the kernels that hold whole rows in registers share: 8 elements of a row,
// its int8 codes, and how many threads take a row.
#pragma once

#include "train_internal.h"

namespace sbn {

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

// the lowest bytes of 8 words
__device__ inline uint2 lowest_bytes(const float* q) {
  uint32_t o[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(q[4 * j + 1]), __float_as_uint(q[4 * j]), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(q[4 * j + 3]), __float_as_uint(q[4 * j + 2]), 0x0c0c0400u);
    o[j] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
  }
  return make_uint2(o[0], o[1]);
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
  return lowest_bytes(q);
}

// The same where u and a are bf16 values.  127 u / a is then a half-integer or at
// least 2^-9 off one if it is 64 to 128, half of that for each power of two below, while
// u rcp is off by under 2^-14 of that kind; rounded to 16 bits (steps of 2^-9 of that
// kind) a half-integer comes out as itself and nothing else as one.  (bf16 quotients
// are half-integers often enough that most waves took the division above: 90 million
// codes 55 us, with this 23.)
__device__ inline uint2 codes8_bf16(const float* u, float rcp) {
  constexpr float SHIFT = 12582912.0f;
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = __uint_as_float((__float_as_uint(u[j] * rcp) + 0x80u) & ~0xFFu) + SHIFT;
  return lowest_bytes(q);
}

// threads of a block for n chunks at CH a thread
inline int threads_for(int n, int ch) { return (int)round_up(cdiv(n, ch), 64); }
inline int chunks_for(int n) { return n <= 512 ? 1 : n <= 2048 ? 2 : 4; }

}  // namespace sbn
