// What the kernels on 8-bit codes share: elements to floats, magnitudes,
// correctly rounded quotients, and tiles of codes loaded straight into LDS
// (block.hip, int8.hip, gated.hip).
#ifndef TLR_CODES8_H
#define TLR_CODES8_H

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tlr {

namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int QB = 128;                   // columns of a block
constexpr float SMALLEST_SCALE = 0x1p-100f;

__device__ __forceinline__ float h2f(uint16_t x) { return (float)__builtin_bit_cast(_Float16, x); }
__device__ __forceinline__ float b2f(uint16_t x) { return __builtin_bit_cast(float, (uint32_t)x << 16); }

// Eight consecutive entries of a row as floats; entries at or past `left` are 0.
template <typename T> __device__ __forceinline__ void load8(const void *x, int64_t at, int64_t left, bool vec, float (&v)[8]);

template <> __device__ __forceinline__ void load8<float>(const void *x, int64_t at, int64_t left, bool vec, float (&v)[8]) {
  const float *p = static_cast<const float *>(x) + at;
  if (vec && left >= 8) {
    const f4 a = *reinterpret_cast<const f4 *>(p), b = *reinterpret_cast<const f4 *>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[4 + e] = b[e]; }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? p[e] : 0.0f;
  }
}

template <bool BF> __device__ __forceinline__ void load8_16(const void *x, int64_t at, int64_t left, bool vec, float (&v)[8]) {
  const uint16_t *p = static_cast<const uint16_t *>(x) + at;
  uint16_t h[8];
  if (vec && left >= 8) {
    *reinterpret_cast<u4 *>(h) = *reinterpret_cast<const u4 *>(p);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = e < left ? p[e] : (uint16_t)0;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = BF ? b2f(h[e]) : h2f(h[e]);
}
template <> __device__ __forceinline__ void load8<_Float16>(const void *x, int64_t at, int64_t left, bool vec, float (&v)[8]) {
  load8_16<false>(x, at, left, vec, v);
}
template <> __device__ __forceinline__ void load8<__bf16>(const void *x, int64_t at, int64_t left, bool vec, float (&v)[8]) {
  load8_16<true>(x, at, left, vec, v);
}

// Magnitudes are compared as the bits of |x|, which orders them as numbers and
// puts infinities and, above them, NaN on top.
__device__ __forceinline__ uint32_t mag(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

// Largest of 16 neighbouring lanes, in all of them (rotations within a DPP row).
__device__ __forceinline__ uint32_t max16(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x128, 0xf, 0xf, true));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x124, 0xf, 0xf, true));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x122, 0xf, 0xf, true));
  return max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x121, 0xf, 0xf, true));
}

// float(x / s) from r = float(1 / s): the residual of the first quotient is
// exact in one fma, and the corrected quotient is the correctly rounded one
// (Markstein's division step; 3 operations instead of about 10).
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
}

// ---- tiles of codes ------------------------------------------------------------------------------------

// 16 codes from column c of a row; codes at or past column k read as zero.
__device__ __forceinline__ u4 load16(const uint8_t *row, int c, int k) {
  u4 x = u4{0, 0, 0, 0};
  if (c < k) {
    x = *reinterpret_cast<const u4 *>(row + c);
    const int left = k - c;
    if (left < 16) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int bytes = left - 4 * w;
        x[w] = bytes >= 4 ? x[w] : bytes <= 0 ? 0u : x[w] & (0xffffffffu >> (32 - 8 * bytes));
      }
    }
  }
  return x;
}

// Buffer descriptor of `bytes` bytes: reads at or past them give zeros.
__device__ __forceinline__ u4 buffer(const void *p, int32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return u4{(uint32_t)a, (uint32_t)(a >> 32) & 0xffffu, (uint32_t)bytes, 0x00027000u};
}

// Loads from a lane's offset in a descriptor, moved by the uniform `by`, straight
// into LDS: lane l writes its 16 (4) bytes at lds + 16 (4) l.  Written out, with
// no register for a result, since the compiler, where it issues them, has LDS
// reads wait for them; the stage loop does the waiting.  The LDS address goes in
// m0, as an operand in that register: the compiler sets it.
__device__ __forceinline__ void to_lds16(u4 b, uint32_t at, uint32_t by, uint32_t lds) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" : : "{m0}"(lds), "v"(at), "s"(b), "s"(by) : "memory");
}
__device__ __forceinline__ void to_lds4(u4 b, uint32_t at, uint32_t lds) {
  asm volatile("s_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" : : "{m0}"(lds), "v"(at), "s"(b) : "memory");
}
typedef __attribute__((address_space(3))) uint8_t lds_byte;
__device__ __forceinline__ uint32_t lds_address(const uint8_t *p) { return (uint32_t)(uintptr_t)(lds_byte *)p; }

// LDS rows are a block's 128 codes, unpadded (the loads write 64 lanes x 16
// bytes in a row); chunk c of a row stands at chunk c ^ key, so that the 16
// rows which a fragment read takes at one chunk hit all 64 banks once.
__device__ __forceinline__ int a_key(int row) { return ((row >> 1) & 1) | ((row >> 3) & 3) << 1; }
__device__ __forceinline__ int b_key(int row) { return (row >> 1) & 7; }

// One operand's tile of ROWS rows: T threads fill a stage of ROWS x 128 codes,
// one 16-byte chunk each per step.
template <int ROWS, int T, bool IS_A> struct Panel {
  static constexpr int N = ROWS * 8 / T;
  static_assert(T % 256 == 0, "a step keeps the key");
  const uint8_t *base;      // first row of the tile (uniform)
  int32_t bytes;            // from there to the end of the last readable chunk
  int32_t step;             // from one step to the next
  uint32_t at;              // this thread's first chunk in column block 0
  u4 rows[N];               // descriptors of the rows from step i on: the steps share `at`
  template <typename Operand> __device__ __forceinline__ void init(const Operand &o, int r0, int k, int tid) {
    base = o.codes + (int64_t)r0 * o.ld;
    bytes = (min(ROWS, o.rows - r0) - 1) * (int32_t)o.ld + ((k + 15) & ~15);
    step = (T / 8) * (int32_t)o.ld;
    at = (uint32_t)(tid >> 3) * (uint32_t)o.ld + chunk(tid);
#pragma unroll
    for (int i = 0; i < N; ++i) rows[i] = buffer(base + i * step, max(bytes - i * step, 0));
  }
  static __device__ __forceinline__ int chunk(int tid) {
    return 16 * ((tid & 7) ^ (IS_A ? a_key(tid >> 3) : b_key(tid >> 3)));
  }
  // step i of a whole column block (rows past the operand's give zeros)
  __device__ __forceinline__ void load(int i, int kb, uint32_t lds, int wave) const {
    to_lds16(rows[i], at, kb * QB, lds + (i * T + wave * 64) * 16);
  }
  // the last column blocks (their descriptors end with the operand); zeros if there is none
  __device__ __forceinline__ void load_last(int kb, uint32_t lds, int wave, bool real) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int32_t o = kb * QB + i * step;
      to_lds16(buffer(base + o, real ? max(bytes - o, 0) : 0), at, 0, lds + (i * T + wave * 64) * 16);
    }
  }
  // zeros in a stage's columns from `left` on
  static __device__ __forceinline__ void cut(int left, uint8_t *lds, int tid) {
    left -= chunk(tid);
    if (left >= 16) return;
    u4 keep;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int n = left - 4 * w;
      keep[w] = n >= 4 ? 0xffffffffu : n <= 0 ? 0u : 0xffffffffu >> (32 - 8 * n);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<u4 *>(lds + (i * T + tid) * 16) &= keep;
  }
};

}  // namespace

}  // namespace tlr

#endif  // TLR_CODES8_H
