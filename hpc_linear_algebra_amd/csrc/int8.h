// 8-bit integer codes: scale and code of an entry, and elements at any
// alignment (int8.hip, gated.hip, experts.hip).
#ifndef TLR_INT8_H
#define TLR_INT8_H

#include "codes8.h"

namespace tlr {

namespace {

constexpr float TOP_INT8 = 127.0f;

// The scale of entries whose largest magnitude has bits `a`.
__device__ __forceinline__ float int8_scale(uint32_t a) {
  const float s = fmaxf(__builtin_bit_cast(float, a) / TOP_INT8, SMALLEST_SCALE);
  return a >= 0x7f800000u ? __builtin_nanf("") : s;
}

// Four entries as codes rint(float(x / s)), ties to even, r = float(1 / s).  A
// quotient is at most 127 (1 + 2^-23) in magnitude.  Added to 1.5 2^23 it is rounded
// to an integer, which then stands in the sum's low bits in two's complement.
__device__ __forceinline__ uint32_t int8_codes4(float a, float b, float c, float d, float s, float r) {
  const float magic = 0x1.8p23f;
  const uint32_t p = __builtin_bit_cast(uint32_t, quotient(a, s, r) + magic), q = __builtin_bit_cast(uint32_t, quotient(b, s, r) + magic);
  const uint32_t u = __builtin_bit_cast(uint32_t, quotient(c, s, r) + magic), v = __builtin_bit_cast(uint32_t, quotient(d, s, r) + magic);
  const uint32_t lo = __builtin_amdgcn_perm(q, p, 0x0c0c0400u), hi = __builtin_amdgcn_perm(v, u, 0x04000c0cu);
  return lo | hi;
}

// Eight codes; zeros where the scale is a NaN.
__device__ __forceinline__ u2 int8_codes8(const float (&v)[8], float s, float r) {
  const uint32_t keep = s == s ? 0xffffffffu : 0u;
  return u2{int8_codes4(v[0], v[1], v[2], v[3], s, r) & keep, int8_codes4(v[4], v[5], v[6], v[7], s, r) & keep};
}

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(_Float16 x) { return (float)x; }
__device__ __forceinline__ float widen(__bf16 x) { return b2f(__builtin_bit_cast(uint16_t, x)); }

// 16 bytes at any alignment of 2 (the hardware takes them), past the caches if PAST.
typedef uint32_t u4_any __attribute__((ext_vector_type(4), aligned(2)));
template <bool PAST> __device__ __forceinline__ u4 get16(const void *p) {
  const u4_any *q = static_cast<const u4_any *>(p);
  if constexpr (PAST) return __builtin_nontemporal_load(q);
  else return *q;
}
template <bool PAST> __device__ __forceinline__ void put16(void *p, u4 v) {
  u4_any *q = static_cast<u4_any *>(p);
  if constexpr (PAST) __builtin_nontemporal_store((u4_any)v, q);
  else *q = v;
}

// Eight consecutive elements as they are.  WHOLE: all of them are there; otherwise
// zeros at or past `left`, element by element.  Several of them go under one branch on
// that: loads under a branch each wait for one another.
template <typename T> struct Eight {
  u4 w[sizeof(T) / 2];
  template <bool WHOLE, bool PAST = false> __device__ __forceinline__ void load(const T *p, int64_t left) {
    if constexpr (WHOLE) {
#pragma unroll
      for (int i = 0; i < (int)(sizeof(T) / 2); ++i) w[i] = get16<PAST>(reinterpret_cast<const char *>(p) + 16 * i);
    } else {
      T x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = e < left ? p[e] : (T)0.0f;
      __builtin_memcpy(w, x, sizeof x);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    T x[8];
    __builtin_memcpy(x, w, sizeof x);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = widen(x[e]);
  }
};

// Eight consecutive elements as floats; zeros at or past `left`.
template <typename T> __device__ __forceinline__ void get8(const T *p, int64_t left, float (&v)[8]) {
  Eight<T> x;
  if (left >= 8) x.template load<true>(p, left);
  else x.template load<false>(p, left);
  x.get(v);
}

// Eight floats rounded to consecutive elements, those before `left`.
template <bool PAST = false, typename T> __device__ __forceinline__ void put8(T *p, int64_t left, const float (&v)[8]) {
  if (left >= 8) {
    T x[8];
    u4 w[sizeof x / 16];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (T)v[e];
    __builtin_memcpy(w, x, sizeof x);
#pragma unroll
    for (int i = 0; i < (int)(sizeof x / 16); ++i) put16<PAST>(reinterpret_cast<char *>(p) + 16 * i, w[i]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) p[e] = (T)v[e];
  }
}

}  // namespace

}  // namespace tlr

#endif  // TLR_INT8_H
