// Block-scaled 8-bit floating point: quantizer and matrix product for gfx950.
//
// A block-scaled matrix holds 8-bit codes (e4m3 or e5m2) whose rows are
// contiguous along the contraction, and one float scale per block of 128
// columns and 1 or 128 rows.  The product is
//   C[i,j] = alpha sum_q sA(i,q) sB(j,q) D_q[i,j] + beta C[i,j],
//   D_q[i,j] = sum of a[i,c] b[j,c] over the 128 columns c of block q,
// and the matrix instructions sum one D_q for 16 x 16 outputs from zero: the
// four results per lane are added into the accumulator with one float fma
// each, the two scales multiplied once per row and column.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "tlr_ops.h"

namespace tlr {

namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef int i8v __attribute__((ext_vector_type(8)));
typedef __bf16 b8v __attribute__((ext_vector_type(8)));

constexpr int QB = 128;                   // columns of a block
constexpr float TOP_E4M3 = 448.0f, TOP_E5M2 = 57344.0f;
constexpr float SMALLEST_SCALE = 0x1p-100f;

__device__ __forceinline__ float h2f(uint16_t x) { return (float)__builtin_bit_cast(_Float16, x); }
__device__ __forceinline__ float b2f(uint16_t x) { return __builtin_bit_cast(float, (uint32_t)x << 16); }

// ---- quantizer ---------------------------------------------------------------------------------------

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

// The scale of a block whose largest magnitude has bits `a`.
template <bool E5> __device__ __forceinline__ float scale_of(uint32_t a) {
  const float s = fmaxf(__builtin_bit_cast(float, a) / (E5 ? TOP_E5M2 : TOP_E4M3), SMALLEST_SCALE);
  return a >= 0x7f800000u ? __builtin_nanf("") : s;
}

// float(x / s) from r = float(1 / s): the residual of the first quotient is
// exact in one fma, and the corrected quotient is the correctly rounded one
// (Markstein's division step; 3 operations instead of about 10).
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
}

// Four quotients as four codes.
template <bool E5> __device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int w = 0;
  if (E5) {
    w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
  } else {
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  }
  return (uint32_t)w;
}

struct QuantArgs {
  const void *x;
  int64_t rows, k, ldx;
  uint8_t *codes;
  int64_t ldq;
  float *scales;
  int64_t lds;
  uint8_t *codes_t;
  int64_t ldq_t;
  float *scales_t;
  int64_t lds_t;
  int vec;              // rows of X 16-byte aligned
};

template <bool PAST, typename V> __device__ __forceinline__ void put(V *p, V v) {
  if constexpr (PAST) __builtin_nontemporal_store(v, p);
  else *p = v;
}


// Bytes of the eight codes in w that lie before column `left` (the rest zero).
__device__ __forceinline__ u2 cut8(u2 w, int64_t left) {
  if (left >= 8) return w;
  const uint64_t v = ((uint64_t)w[1] << 32 | w[0]) & (left <= 0 ? 0ull : (~0ull >> (64 - 8 * left)));
  return u2{(uint32_t)v, (uint32_t)(v >> 32)};
}

// One workgroup per 128 x 128 tile of X; thread (c, r) = (tid % 16, tid / 16)
// holds the 8 x 8 entries of rows 8r.. and columns 8c.. in registers, so that
// X is read once for both results.  Row maxima are 16-lane rotations, column
// maxima two lane exchanges and 4 x 128 words of LDS, the transposed codes
// (8 consecutive rows of a column are one 8-byte word) turn through LDS.
template <typename T, bool E5, int BLOCK, bool PAST>
__global__ __launch_bounds__(256) void quantize_kernel(QuantArgs a) {
  __shared__ uint32_t top[4][QB];
  __shared__ __attribute__((aligned(16))) uint8_t turn[QB][QB + 16];
  const int tid = threadIdx.x, c = tid & 15, r = tid >> 4, wave = tid >> 6;
  // Tiles row by row; where tiles share lines, each of the 8 XCDs (to which
  // workgroups go in turn) takes a contiguous part of them, so that such lines
  // meet in one L2.
  int cb, rb;
  {
    const int nx = (int)((a.k + QB - 1) / QB), all = gridDim.x, part = all >> 3, more = all & 7, x = blockIdx.x & 7;
    const int t = PAST ? (int)blockIdx.x : x * part + min(x, more) + (int)(blockIdx.x >> 3);
    rb = t / nx;
    cb = t - rb * nx;
  }
  const int64_t c0 = (int64_t)cb * QB, r0 = (int64_t)rb * QB;
  const int64_t col = c0 + 8 * c, row = r0 + 8 * r;

  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t left = row + i < a.rows ? a.k - col : 0;
    if (left > 0) load8<T>(a.x, (row + i) * a.ldx + col, left, a.vec, v[i]);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
  }

  float tile_s = 0.0f, tile_r = 0.0f;
  if constexpr (BLOCK == 128) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, mag(v[i][e]));
    m = max16(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if ((tid & 63) == 0) top[0][wave] = m;
    __syncthreads();
    m = max(max(top[0][0], top[0][1]), max(top[0][2], top[0][3]));
    tile_s = scale_of<E5>(m);
    tile_r = 1.0f / tile_s;
    if (tid == 0) {
      if (a.codes) a.scales[rb + cb * a.lds] = tile_s;
      if (a.codes_t) a.scales_t[cb + rb * a.lds_t] = tile_s;
    }
  }

  if (a.codes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s = tile_s, q = tile_r;
      if constexpr (BLOCK == 1) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, mag(v[i][e]));
        s = scale_of<E5>(max16(m));
        q = 1.0f / s;
        if (c == i && row + i < a.rows) a.scales[row + i + cb * a.lds] = s;
      }
      if (row + i < a.rows && col < ((a.k + 15) & ~(int64_t)15)) {
        u2 w;
        w[0] = codes4<E5>(quotient(v[i][0], s, q), quotient(v[i][1], s, q), quotient(v[i][2], s, q), quotient(v[i][3], s, q));
        w[1] = codes4<E5>(quotient(v[i][4], s, q), quotient(v[i][5], s, q), quotient(v[i][6], s, q), quotient(v[i][7], s, q));
        put<PAST>(reinterpret_cast<u2 *>(a.codes + (row + i) * a.ldq + col), cut8(w, a.k - col));
      }
    }
  }

  if (a.codes_t) {
    if constexpr (BLOCK == 1) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, mag(v[i][e]));
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        if ((tid & 63) < 16) top[wave][8 * c + e] = m;
      }
      __syncthreads();
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float s = tile_s, q = tile_r;
      if constexpr (BLOCK == 1) {
        const int x = 8 * c + e;
        s = scale_of<E5>(max(max(top[0][x], top[1][x]), max(top[2][x], top[3][x])));
        q = 1.0f / s;
        if (r == e && col + e < a.k) a.scales_t[col + e + rb * a.lds_t] = s;
      }
      u2 w;
      w[0] = codes4<E5>(quotient(v[0][e], s, q), quotient(v[1][e], s, q), quotient(v[2][e], s, q), quotient(v[3][e], s, q));
      w[1] = codes4<E5>(quotient(v[4][e], s, q), quotient(v[5][e], s, q), quotient(v[6][e], s, q), quotient(v[7][e], s, q));
      *reinterpret_cast<u2 *>(&turn[8 * c + e][8 * r]) = cut8(w, a.rows - row);
    }
    __syncthreads();
    // 128 rows of the result (columns of X), 8 vectors of 16 codes each
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = (tid >> 3) + 32 * i, y = 16 * (tid & 7);
      if (c0 + x < a.k && r0 + y < a.rows)
        put<PAST>(reinterpret_cast<u4 *>(a.codes_t + (c0 + x) * a.ldq_t + r0 + y), *reinterpret_cast<const u4 *>(&turn[x][y]));
    }
  }
}

template <typename T, bool E5>
void quantize_launch(const QuantArgs &a, int block, bool past, unsigned grid, hipStream_t st) {
  if (block == 1) {
    if (past) quantize_kernel<T, E5, 1, true><<<grid, 256, 0, st>>>(a);
    else quantize_kernel<T, E5, 1, false><<<grid, 256, 0, st>>>(a);
  } else {
    if (past) quantize_kernel<T, E5, 128, true><<<grid, 256, 0, st>>>(a);
    else quantize_kernel<T, E5, 128, false><<<grid, 256, 0, st>>>(a);
  }
}
template <typename T>
void quantize_launch(const QuantArgs &a, bool e5, int block, bool past, unsigned grid, hipStream_t st) {
  if (e5) quantize_launch<T, true>(a, block, past, grid, st);
  else quantize_launch<T, false>(a, block, past, grid, st);
}

// ---- product -----------------------------------------------------------------------------------------

struct Operand {
  const uint8_t *codes;
  const float *scales;
  int64_t ld, lds;
  int32_t rows, shift;      // shift: row block of row i is i >> shift (0 or 7)
};

struct GemmArgs {
  Operand a, b;
  int32_t m, n, k;
  float alpha, beta;
  void *c;
  int64_t ldc;
  int32_t dt;
};

// Two codes widened to bfloat16, exactly.
template <bool E5, bool HI> __device__ __forceinline__ uint32_t widen2(uint32_t w) {
  if (E5) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.0f, HI));
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}
template <bool E5> __device__ __forceinline__ b8v widen8(uint32_t w0, uint32_t w1) {
  return __builtin_bit_cast(b8v, u4{widen2<E5, false>(w0), widen2<E5, true>(w0), widen2<E5, false>(w1), widen2<E5, true>(w1)});
}

// One 16 x 16 x 128 block of products, summed from zero.  Lane l supplies 32
// codes of row l % 16 of A and of row l % 16 of B (the same columns of the
// block for both: any assignment of columns to lanes gives the same sum) and
// holds D[4 (l / 16) + v][l % 16] in element v.
//
// FAST: one 8-bit instruction.  Both 8-bit instructions (x128 and x32) line the
// products up with the largest one and drop what is below 2^-13 of its binary
// order (2^16 + 2^3 comes out whole, 2^16 + 2^2 as 2^16; 1.5e-5 relative
// Frobenius error on normal data).  Otherwise the codes are widened and the
// bfloat16 instructions add in float (9e-9 on the same data).  In registers
// only, the x128 instruction reaches 4.19 PFLOP/s on the whole chip.
__device__ __forceinline__ i8v join(u4 a, u4 b) {
  return __builtin_bit_cast(i8v, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// A fragment: the lane's 32 codes of a row, as the instructions take them.
template <bool E5, bool FAST> struct Fragment;
template <bool E5> struct Fragment<E5, true> {
  i8v x;
  Fragment() = default;
  __device__ __forceinline__ Fragment(i8v c) : x(c) {}
};
template <bool E5> struct Fragment<E5, false> {
  b8v x[4];
  Fragment() = default;
  __device__ __forceinline__ Fragment(i8v c)
      : x{widen8<E5>(c[0], c[1]), widen8<E5>(c[2], c[3]), widen8<E5>(c[4], c[5]), widen8<E5>(c[6], c[7])} {}
};
template <bool A5, bool B5> __device__ __forceinline__ f4 mma(const Fragment<A5, true> &a, const Fragment<B5, true> &b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.x, b.x, f4{0, 0, 0, 0}, A5 ? 1 : 0, B5 ? 1 : 0, 0, 0, 0, 0);
}
template <bool A5, bool B5> __device__ __forceinline__ f4 mma(const Fragment<A5, false> &a, const Fragment<B5, false> &b) {
  f4 d = f4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.x[i], b.x[i], d, 0, 0, 0);
  return d;
}

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

// alpha v + beta old in C's type, rounded once.
__device__ __forceinline__ void store_c(const GemmArgs &g, int i, int j, float v) {
  const int64_t at = (int64_t)j * g.ldc + i;
  v *= g.alpha;
  if (g.dt == TLR_F32) {
    float *p = static_cast<float *>(g.c) + at;
    *p = g.beta != 0.0f ? v + g.beta * *p : v;
  } else if (g.dt == TLR_F16) {
    _Float16 *p = static_cast<_Float16 *>(g.c) + at;
    *p = (_Float16)(g.beta != 0.0f ? v + g.beta * (float)*p : v);
  } else {
    __bf16 *p = static_cast<__bf16 *>(g.c) + at;
    *p = (__bf16)(g.beta != 0.0f ? v + g.beta * (float)*p : v);
  }
}

// Eight consecutive rows of a column from row i, all of them C's, as vectors of
// any alignment (2501 x 1111 x 1792 of odd columns: 14.7 us, element by element
// through LDS 15.7, 2560 x 1152 x 1792 of aligned ones 13.3).
__device__ __forceinline__ void store_c8(const GemmArgs &g, int i, int j, const float (&v)[8]) {
  const int64_t at = (int64_t)j * g.ldc + i;
  const bool add = g.beta != 0.0f;
  if (g.dt == TLR_F32) {
    float *p = static_cast<float *>(g.c) + at, x[8];
    if (add) __builtin_memcpy(x, p, 32);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = add ? v[e] * g.alpha + g.beta * x[e] : v[e] * g.alpha;
    __builtin_memcpy(p, x, 32);
  } else if (g.dt == TLR_F16) {
    _Float16 *p = static_cast<_Float16 *>(g.c) + at, x[8];
    if (add) __builtin_memcpy(x, p, 16);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (_Float16)(add ? v[e] * g.alpha + g.beta * (float)x[e] : v[e] * g.alpha);
    __builtin_memcpy(p, x, 16);
  } else {
    __bf16 *p = static_cast<__bf16 *>(g.c) + at, x[8];
    if (add) __builtin_memcpy(x, p, 16);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (__bf16)(add ? v[e] * g.alpha + g.beta * (float)x[e] : v[e] * g.alpha);
    __builtin_memcpy(p, x, 16);
  }
}

// Few columns or little work: a workgroup computes 16 rows of A against 16 rows
// of B, its eight waves taking every eighth block of the contraction; fragments
// come straight from global memory, UNROLL blocks in flight a wave, and the
// partial sums meet in LDS.  AB: A's blocks are 128 rows high.
template <bool A5, bool B5, bool FAST, bool AB>
__global__ __launch_bounds__(512, 4) void strip_kernel(GemmArgs g) {
  constexpr int W = 8, SA = AB ? 1 : 4, UNROLL = AB ? 4 : 2;      // 128 registers each way
  __shared__ float part[W][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int m0 = blockIdx.x * 16, n0 = blockIdx.y * 16;
  const uint8_t *arow = g.a.codes + (int64_t)min(m0 + r, g.m - 1) * g.a.ld + 16 * q;
  const int br = min(n0 + r, g.n - 1);
  const uint8_t *brow = g.b.codes + (int64_t)br * g.b.ld + 16 * q;
  const float *as[SA], *bs = g.b.scales + (br >> g.b.shift);
#pragma unroll
  for (int v = 0; v < SA; ++v) as[v] = g.a.scales + (AB ? m0 >> 7 : min(m0 + 4 * q + v, g.m - 1));

  f4 acc = f4{0, 0, 0, 0};
  struct Block {
    u4 a[2], b[2];
    float sa[SA], sb;
  };
  auto scales = [&](int kb, Block &x) {
#pragma unroll
    for (int v = 0; v < SA; ++v) x.sa[v] = as[v][kb * g.a.lds];
    x.sb = bs[kb * g.b.lds];
  };
  auto load = [&](int kb, Block &x) {
    const int64_t c = (int64_t)kb * QB;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x.a[h] = *reinterpret_cast<const u4 *>(arow + c + 64 * h);
      x.b[h] = *reinterpret_cast<const u4 *>(brow + c + 64 * h);
    }
    scales(kb, x);
  };
  auto add = [&](const Block &x) {
    const f4 d = mma<A5, B5>(Fragment<A5, FAST>(join(x.a[0], x.a[1])), Fragment<B5, FAST>(join(x.b[0], x.b[1])));
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = __builtin_fmaf(x.sa[AB ? 0 : v] * x.sb, d[v], acc[v]);
  };
  const int full = g.k / QB;
  int kb = wave;
  for (; kb + (UNROLL - 1) * W < full; kb += UNROLL * W) {
    Block x[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) load(kb + u * W, x[u]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) add(x[u]);
  }
  for (; kb < full; kb += W) {
    Block x;
    load(kb, x);
    add(x);
  }
  if (kb == full && g.k > full * QB) {          // the cut block
    Block x;
    const int64_t o = (int64_t)full * QB - 16 * q;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x.a[h] = load16(arow + o, 16 * q + 64 * h, g.k - full * QB);
      x.b[h] = load16(brow + o, 16 * q + 64 * h, g.k - full * QB);
    }
    scales(full, x);
    add(x);
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) part[wave][v][lane] = acc[v];
  __syncthreads();
  if (threadIdx.x < 256) {
    const int i = threadIdx.x & 15, j = threadIdx.x >> 4;      // row, column of the workgroup's block
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += part[w][i & 3][(i >> 2) * 16 + j];
    if (m0 + i < g.m && n0 + j < g.n) store_c(g, m0 + i, n0 + j, v);
  }
}

// ---- product, tiles ----------------------------------------------------------------------------------

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
  __device__ __forceinline__ void init(const Operand &o, int r0, int k, int tid) {
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

// C tiles of TM x TN, WM x WN waves, each RI x CJ tiles of 16 x 16.  AB: A's
// blocks are 128 rows high (a wave's rows lie in one of them).  KG 2: two such
// halves of waves take every other column block and add their sums at the end,
// which halves the barriers and lets waves be larger (fewer bytes from LDS); it
// pays from about 16 column blocks on.
//
// Two stages of KG column blocks each in LDS.  A wave goes through a stage row
// tile by row tile; with the last one's matrix instructions under way it waits
// for the next stage and reads its first fragments: one barrier a stage, and the
// matrix cores have work on both sides of it.  The stage after that is loaded
// into the buffer that is then used up, SPREAD pieces under each row tile's matrix
// instructions, or all at once (SPREAD 0), which a short stage needs: 8192^3 in
// 256 x 256 tiles 460 us with two pieces, 475 at once; 4096 x 4096 x 8192 exact in
// 128 x 128 tiles on four waves 243 with three, 259 at once; 2501 x 1111 x 1747 on
// eight waves 19.0 spread, 17.7 at once.
//
// What bounds 8192^3 (451 us, 2.4 PFLOP/s, 89% of the library's product without blocks):
// the matrix cores are busy 62% of the clocks.  Timing copies (at 460 us as built): matrix instructions
// and barriers alone 319 us, the scaled additions add 48, the loads 94 (alone they
// take 377; two, three or four stages of them in flight make no difference, nor do
// odd strides), the fragment reads from LDS 10.
template <bool A5, bool B5, bool FAST, bool AB, int TM, int TN, int WM, int WN, int KG, int SPREAD>
__global__ __launch_bounds__(64 * WM * WN * KG) __attribute__((amdgpu_waves_per_eu(2, 2))) void tile_kernel(GemmArgs g) {
  constexpr int T = 64 * WM * WN * KG, RI = TM / WM / 16, CJ = TN / WN / 16;
  static_assert(RI % 2 == 0 && (!AB || 128 % (TM / WM) == 0), "");
  // a column block: A's codes, B's codes, A's and B's scales; a stage: KG of them
  constexpr int SN = (TM + TN + T - 1) / T;                // scales a thread loads
  constexpr int AT_B = TM * QB, AT_S = (TM + TN) * QB, BLOCK = AT_S + SN * T * 4, STAGE = KG * BLOCK;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4, kg = wave / (WM * WN), wm = wave / WN % WM, wn = wave % WN;

  // tile of this workgroup: workgroups go to the 8 XCDs in turn; each XCD takes
  // a contiguous part of the tiles, which run down 8 row tiles at a time
  int mt, nt;
  {
    const int tm = (g.m + TM - 1) / TM, tn = (g.n + TN - 1) / TN, all = tm * tn;
    const int id = blockIdx.x, x = id & 7, part = all >> 3, more = all & 7;
    const int t = x * part + min(x, more) + (id >> 3);
    const int width = 8 * tn, band = t / width, h = min(8, tm - 8 * band), in = t - band * width;
    mt = 8 * band + in % h;
    nt = in / h;
  }
  const int m0 = mt * TM, n0 = nt * TN;
  Panel<TM, T, true> pa;
  Panel<TN, T, false> pb;
  pa.init(g.a, m0, g.k, tid);
  pb.init(g.b, n0, g.k, tid);
  // scales: TM + TN floats a stage, 64 a wave and step (the waves past them write zeros)
  const float *sbase[SN];
  int64_t sld[SN];
  int32_t sbytes[SN];
  uint32_t sat[SN];
#pragma unroll
  for (int i = 0; i < SN; ++i) {
    const int w = i * T + wave * 64;
    const bool isa = w < TM;
    const Operand &o = isa ? g.a : g.b;
    const int r0 = isa ? m0 : n0, first = r0 >> o.shift;
    sbase[i] = o.scales + first;
    sld[i] = o.lds;
    sbytes[i] = w < TM + TN ? 4 * (((min(r0 + (isa ? TM : TN), o.rows) - 1) >> o.shift) - first + 1) : 0;
    sat[i] = 4 * (((r0 + (isa ? w : w - TM) + lane) >> o.shift) - first);
  }
  auto load_scales = [&](int kb, uint32_t ls, bool real) {
#pragma unroll
    for (int i = 0; i < SN; ++i) to_lds4(buffer(sbase[i] + kb * sld[i], real ? sbytes[i] : 0), sat[i], ls + 4 * (i * T + wave * 64));
  };
  // The stage of column blocks kb, kb + 1, .., in LOADS pieces.
  constexpr int NA = Panel<TM, T, true>::N, PIECES = NA + Panel<TN, T, false>::N + 1, LOADS = KG * PIECES;
  auto load = [&](int piece, int kb, uint32_t to) {
    kb += piece / PIECES;
    to += piece / PIECES * BLOCK;
    piece %= PIECES;
    if (piece == 0) load_scales(kb, to + AT_S, true);
    else if (piece <= NA) pa.load(piece - 1, kb, to, wave);
    else pb.load(piece - 1 - NA, kb, to + AT_B, wave);
  };

  f4 acc[RI][CJ];
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int j = 0; j < CJ; ++j) acc[i][j] = f4{0, 0, 0, 0};

  // Fragment addresses.  Row tile i = 2h + p: lane r holds block row
  // 32 h + 8 (r / 4) + 4 p + r % 4, so that the two tiles of a pair leave 8
  // consecutive rows of C in one lane.
  const int ar = wm * (TM / WM) + 8 * (r >> 2) + (r & 3), br = wn * (TN / WN) + r;
  const int aat = ar * QB + 16 * (q ^ a_key(ar)), bat = AT_B + br * QB + 16 * (q ^ b_key(br));
  i8v x[2], b[CJ];            // of row tile i (mod 2) and of the stage's columns
  f4 sa[2];                   // scales of the lane's rows of row tile i (AB: in sb)
  float sb[CJ], sn[CJ];       // of its columns, and those of the next stage
  auto read_a = [&](const uint8_t *l, int i) {
    const int o = (i >> 1) * 32 * QB + (i & 1) * 4 * QB;
    x[i & 1] = join(*reinterpret_cast<const u4 *>(l + aat + o), *reinterpret_cast<const u4 *>(l + (aat ^ 64) + o));
  };
  auto read_sa = [&](const uint8_t *l, int i) {
    if constexpr (!AB)
      sa[i & 1] = *reinterpret_cast<const f4 *>(l + AT_S + 4 * (wm * (TM / WM) + (i >> 1) * 32 + 8 * q + 4 * (i & 1)));
  };
  auto read_b = [&](const uint8_t *l) {
#pragma unroll
    for (int j = 0; j < CJ; ++j) {
      b[j] = join(*reinterpret_cast<const u4 *>(l + bat + 16 * QB * j), *reinterpret_cast<const u4 *>(l + (bat ^ 64) + 16 * QB * j));
      sn[j] = *reinterpret_cast<const float *>(l + AT_S + 4 * (TM + br + 16 * j));
    }
    if constexpr (AB) {
      const float s = *reinterpret_cast<const float *>(l + AT_S + 4 * wm * (TM / WM));
#pragma unroll
      for (int j = 0; j < CJ; ++j) sn[j] *= s;
    }
  };
  auto add = [&](int i, const f4 (&d)[CJ]) {
#pragma unroll
    for (int j = 0; j < CJ; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(AB ? sb[j] : sa[i & 1][v] * sb[j], d[j][v], acc[i][j][v]);
  };
  auto meet = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // This workgroup's column blocks: all, or the part of grid y.  Stage 0 is its
  // last one to KG, the very last of which may be cut at column k; stage i > 0
  // is the KG from kb0 + (i - 1) KG on.
  const int blocks = (g.k + QB - 1) / QB;
  const int kb0 = (int)((int64_t)blocks * blockIdx.y / gridDim.y);
  const int mine = (int)((int64_t)blocks * (blockIdx.y + 1) / gridDim.y) - kb0;
  const int nb = (mine + KG - 1) / KG, last = mine - (nb - 1) * KG;      // stages; column blocks of stage 0
  const bool cut = (g.k & (QB - 1)) != 0 && kb0 + mine == blocks;
  const uint32_t base = lds_address(lds);
#pragma unroll
  for (int c = 0; c < KG; ++c) {
    const int kb = c < last ? kb0 + mine - last + c : 0;
    load_scales(kb, base + c * BLOCK + AT_S, c < last);
    pa.load_last(kb, base + c * BLOCK, wave, c < last);
    pb.load_last(kb, base + c * BLOCK + AT_B, wave, c < last);
  }
  auto load_all = [&](int kb, uint32_t to) {
#pragma unroll
    for (int c = 0; c < LOADS; ++c) load(c, kb, to);
  };
  if (SPREAD == 0 && nb > 1) {
    load_all(kb0, base + STAGE);
    constexpr int LEFT = LOADS + KG * (SN - 1);      // stage 1, still under way
    static_assert(LEFT < 16, "");
    __builtin_amdgcn_s_waitcnt(LEFT | 0xf << 8 | 7 << 4);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  } else {
    meet();
  }
  if (cut) {
    pa.cut(g.k & (QB - 1), lds + (last - 1) * BLOCK, tid);
    pb.cut(g.k & (QB - 1), lds + (last - 1) * BLOCK + AT_B, tid);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xf | 3 << 14 | 7 << 4);      // LDS only
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
  read_b(lds + kg * BLOCK);
  read_a(lds + kg * BLOCK, 0);
  f4 d[2][CJ];
  // All sums of a stage but the last row tile's, column block kb loaded meanwhile.
  auto row_tiles = [&](const uint8_t *l, auto live, int kb, uint32_t to) {
    static_assert(SPREAD == 0 || SPREAD * RI >= LOADS, "");
    Fragment<B5, FAST> bf[CJ];
#pragma unroll
    for (int j = 0; j < CJ; ++j) {
      sb[j] = sn[j];
      bf[j] = Fragment<B5, FAST>(b[j]);
    }
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      if (i + 1 < RI) read_a(l, i + 1);
      read_sa(l, i);
      const Fragment<A5, FAST> af(x[i & 1]);
#pragma unroll
      for (int j = 0; j < CJ; ++j) d[i & 1][j] = mma<A5, B5>(af, bf[j]);
      if constexpr (decltype(live)::value)
#pragma unroll
        for (int c = 0; c < SPREAD; ++c)
          if (i * SPREAD + c < LOADS) load(i * SPREAD + c, kb, to);
      if (i > 0) add(i - 1, d[(i - 1) & 1]);
      // here, not where the sums are next used: sunk there past the branches
      // below, they would keep every d in registers
      if (i > 0)
#pragma unroll
        for (int j = 0; j < CJ; ++j) asm volatile("" : "+v"(acc[i - 1][j]));
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int now = 0, next = STAGE;
  for (int stage = 0; stage < nb - 1; ++stage) {
    row_tiles(lds + now + kg * BLOCK, std::true_type{}, kb0 + stage * KG, base + next);
    meet();
    if (SPREAD == 0 && stage + 2 < nb) load_all(kb0 + (stage + 1) * KG, base + now);
    read_b(lds + next + kg * BLOCK);
    read_a(lds + next + kg * BLOCK, 0);
    add(RI - 1, d[1]);
    const int t = now;
    now = next;
    next = t;
  }
  row_tiles(lds + now + kg * BLOCK, std::false_type{}, 0, 0);
  add(RI - 1, d[1]);
  if constexpr (KG == 2) {                // the second half's sums to the first half
    static_assert(WM * WN * RI * CJ * 1024 <= 2 * STAGE, "");
    f4 *sums = reinterpret_cast<f4 *>(lds) + (wave % (WM * WN)) * RI * CJ * 64 + lane;
    __syncthreads();
    if (kg == 1)
#pragma unroll
      for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int j = 0; j < CJ; ++j) sums[(i * CJ + j) * 64] = acc[i][j];
    __syncthreads();
    if (kg == 1) return;
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
      for (int j = 0; j < CJ; ++j) acc[i][j] += sums[(i * CJ + j) * 64];
  }

  // lane (r, q): rows 32 h + 8 q .. + 7 of its columns
  if (gridDim.y > 1) g.c = static_cast<float *>(g.c) + (int64_t)blockIdx.y * g.m * g.n;      // a part's sums
  constexpr int ROWS = TM / WM;
  const int row0 = m0 + wm * ROWS, col0 = n0 + wn * (TN / WN);
#pragma unroll
  for (int j = 0; j < CJ; ++j) {
    const int col = col0 + 16 * j + r;
    if (col < g.n)
#pragma unroll
      for (int h = 0; h < RI / 2; ++h) {
        const int row = row0 + 32 * h + 8 * q;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = acc[2 * h + (e >> 2)][j][e & 3];
        if (row + 8 <= g.m) store_c8(g, row, col, v);
        else if (row < g.m)
#pragma unroll
          for (int e = 0; e < 7; ++e)
            if (row + e < g.m) store_c(g, row + e, col, v[e]);
      }
  }
}

// C = alpha (sum of PARTS m x n matrices of floats, in their order) + beta C: a
// thread takes 8 consecutive rows of a column.
template <int PARTS> __global__ __launch_bounds__(256) void parts_kernel(GemmArgs g, const float *part) {
  const int up = (g.m + 7) / 8;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int j = (int)(at / up), i = 8 * (int)(at - (int64_t)j * up);
  if (j >= g.n) return;
  const float *p = part + (int64_t)j * g.m + i;
  const int64_t step = (int64_t)g.m * g.n;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (i + 8 <= g.m) {
    float x[PARTS][8];
#pragma unroll
    for (int z = 0; z < PARTS; ++z) __builtin_memcpy(x[z], p + z * step, 32);
#pragma unroll
    for (int z = 0; z < PARTS; ++z)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += x[z][e];
    store_c8(g, i, j, v);
    return;
  }
  for (int e = 0; i + e < g.m; ++e) {
    float s = 0.0f;
    for (int z = 0; z < PARTS; ++z) s += p[z * step + e];
    store_c(g, i + e, j, s);
  }
}

// ---- which kernel -----------------------------------------------------------------------------------

enum Kind { STRIP, TILE_64, TILE_64K, TILE_128, TILE_128W, TILE_128K, TILE_256 };
struct Shape {
  int rows, cols, threads;  // of C and of the workgroup that computes them
  int halves;               // of its waves, which share the column blocks
};
constexpr Shape SHAPE[] = {{16, 16, 512, 1},   {128, 64, 512, 1},  {128, 64, 512, 2}, {128, 128, 256, 1},
                           {128, 128, 512, 1}, {128, 128, 512, 2}, {256, 256, 512, 1}};
struct Choice {
  Kind kind;
  int parts;                // of the contraction, with a launch that adds them if more than one
};

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A launch has less than 2^32 threads along x.  128 x 128 tiles of four waves fit
// whatever the others do, where a result has less than TILE_LIM of them.
constexpr int64_t THREAD_LIM = (int64_t)1 << 32, TILE_LIM = (int64_t)1 << 24;
int64_t workgroups(Kind kind, int64_t m, int64_t n) {
  return kind == STRIP ? cdiv(m, 16) : cdiv(m, SHAPE[kind].rows) * cdiv(n, SHAPE[kind].cols);      // along x
}
bool fits(Kind kind, int parts, int64_t m, int64_t n) {
  return workgroups(kind, m, n) * SHAPE[kind].threads < THREAD_LIM && (kind != STRIP || cdiv(n, 16) <= 65535) &&
         (parts == 1 || cdiv(m, 8) * n < THREAD_LIM - 256);
}

// The kernel with the least estimated time (us).  Each estimate is a fit to
// measured times (graph replays, 16-bit C with `fast`, float C of e4m3 and e5m2
// operands without).  Some of them, the kernel chosen first:
//   fast   512 x 20 x 512       strip 2.9, 128 x 64 tiles 4.6
//          8192 x 1 x 4096      strip 7.9, 128 x 64 tiles 20.0, four parts 11.2
//          1024 x 1024 x 1024   128 x 64 tiles 6.4, 128 x 128 8.4, strip 20.5
//          8192 x 64 x 8192     128 x 64 tiles in four parts 19.7, one 37.7, strip 60.2
//          2048 x 2048 x 512    128 x 128 on eight waves 7.3, on four 8.1, 256 x 256 13.3
//          2048 x 4096 x 2048   128 x 128 on four waves 23.3, on eight 27.2, 256 x 256 31.5
//          4096 x 4096 x 4096   256 x 256 tiles 63.0, 128 x 128 76.5
//          4096 x 512 x 4096    128 x 64 in two halves 18.0, whole 21.3, 128 x 128 23.5
//          2000 x 1000 x 8000   128 x 128 in two halves and two parts 32.7, whole in two parts 35.4
//          4096 x 1024 x 4096   128 x 128 in two halves 24.6, on eight waves 25.9
//   exact  1024 x 1024 x 1024   128 x 64 tiles 9.4, 128 x 128 13.2, strip 23.0
//          2048 x 2048 x 4096   128 x 128 in two halves 38.2, whole 43.0
//          4096 x 4096 x 8192   128 x 128 on four waves 247, on eight 295, 256 x 256 (not kept) 307
Choice choose(int64_t m, int64_t n, int64_t k, bool fast) {
  const double nb = (double)cdiv(k, QB);
  Choice best{TILE_128, 1};
  double least = 1e300;
  auto offer = [&](Kind kind, int parts, double t) {
    if (t < least && fits(kind, parts, m, n)) {
      least = t;
      best = Choice{kind, parts};
    }
  };
  // 4 KB a workgroup and block out of the caches
  offer(STRIP, 1, 2.8 + cdiv(m, 16) * cdiv(n, 16) * nb * (fast ? 0.00040 : 0.00048));
  // One workgroup a CU takes `one` a column block, two together `two`.
  auto tiles = [&](Kind kind, int tn, double one, double two, double first, double next) {
    for (const int parts : {1, 2, 4, 8}) {
      if (parts > 1 && nb < 4 * parts) break;
      const double t = (double)cdiv(m, 128) * (double)cdiv(n, tn) * parts;
      const double rounds = std::ceil(t / 512), rest = t - 512 * (rounds - 1);
      double us = first + (rounds - 1) * next + std::ceil(nb / parts) * ((rounds - 1) * two + (rest <= 256 ? one : two));
      if (parts > 1) us += 2.8 + parts * (0.1 + (double)m * (double)n * 2.1e-6);
      offer(kind, parts, us);
    }
  };
  if (fast) {
    tiles(TILE_64, 64, 0.57, 1.15, 3.2, 3.0);
    tiles(TILE_128W, 128, 0.69, 1.48, 3.9, 4.0);
    tiles(TILE_128, 128, 0.70, 1.10, 5.0, 5.0);
    tiles(TILE_64K, 64, 0.47, 0.96, 3.8, 3.0);
    tiles(TILE_128K, 128, 0.56, 1.25, 6.4, 5.5);
    const double rounds = std::ceil((double)cdiv(m, 256) * (double)cdiv(n, 256) / 256);
    offer(TILE_256, 1, 6.0 + (rounds - 1) * 4.0 + nb * rounds * 1.8);
  } else {
    tiles(TILE_64, 64, 0.75, 1.6, 3.5, 3.0);
    tiles(TILE_128W, 128, 1.2, 2.2, 4.0, 4.0);
    tiles(TILE_128, 128, 1.25, 1.85, 5.0, 5.0);
    tiles(TILE_64K, 64, 0.67, 1.32, 4.0, 3.0);
    tiles(TILE_128K, 128, 1.02, 2.04, 6.0, 6.0);
  }
  return best;
}

template <Kind KIND, bool A5, bool B5, bool FAST, int WM, int WN, int SPREAD>
void tile_launch(const GemmArgs &g, int parts, float *ws, hipStream_t st) {
  constexpr int TM = SHAPE[KIND].rows, TN = SHAPE[KIND].cols, KG = SHAPE[KIND].halves;
  static_assert(SHAPE[KIND].threads == 64 * WM * WN * KG, "");
  const dim3 grid((unsigned)workgroups(KIND, g.m, g.n), (unsigned)parts);
  GemmArgs h = g;
  if (parts > 1) {
    h.alpha = 1.0f;
    h.beta = 0.0f;
    h.c = ws;
    h.ldc = g.m;
    h.dt = TLR_F32;
  }
  if (g.a.shift) tile_kernel<A5, B5, FAST, true, TM, TN, WM, WN, KG, SPREAD><<<grid, 64 * WM * WN * KG, 0, st>>>(h);
  else tile_kernel<A5, B5, FAST, false, TM, TN, WM, WN, KG, SPREAD><<<grid, 64 * WM * WN * KG, 0, st>>>(h);
  if (parts == 1) return;
  const unsigned sum = (unsigned)cdiv(cdiv(g.m, 8) * g.n, 256);
  if (parts == 2) parts_kernel<2><<<sum, 256, 0, st>>>(g, ws);
  else if (parts == 4) parts_kernel<4><<<sum, 256, 0, st>>>(g, ws);
  else parts_kernel<8><<<sum, 256, 0, st>>>(g, ws);
}

template <bool A5, bool B5, bool FAST> void strip_launch(const GemmArgs &g, hipStream_t st) {
  const dim3 grid((unsigned)workgroups(STRIP, g.m, g.n), (unsigned)cdiv(g.n, 16));
  if (g.a.shift) strip_kernel<A5, B5, FAST, true><<<grid, 512, 0, st>>>(g);
  else strip_kernel<A5, B5, FAST, false><<<grid, 512, 0, st>>>(g);
}

template <bool A5, bool B5, bool FAST> void gemm_launch(const GemmArgs &g, const Choice &c, float *ws, hipStream_t st) {
  switch (c.kind) {
    case STRIP: return strip_launch<A5, B5, FAST>(g, st);
    case TILE_64: return tile_launch<TILE_64, A5, B5, FAST, 4, 2, 0>(g, c.parts, ws, st);
    case TILE_64K: return tile_launch<TILE_64K, A5, B5, FAST, 2, 2, 0>(g, c.parts, ws, st);
    case TILE_128: return tile_launch<TILE_128, A5, B5, FAST, 2, 2, 3>(g, c.parts, ws, st);
    case TILE_128W: return tile_launch<TILE_128W, A5, B5, FAST, 2, 4, 0>(g, c.parts, ws, st);
    case TILE_128K: return tile_launch<TILE_128K, A5, B5, FAST, 2, 2, FAST ? 0 : 3>(g, c.parts, ws, st);
    case TILE_256:
      if constexpr (FAST) return tile_launch<TILE_256, A5, B5, FAST, 2, 4, 2>(g, c.parts, ws, st);
  }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

tlr_status launched(const char *what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TLR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
  return TLR_OK;
}

constexpr int64_t SIZE_LIM = 0x7fffffff, PRODUCT_LIM = SIZE_LIM - 511, LD_LIM = (int64_t)1 << 22;

// Sizes of a product; a tile's rows past the end are still an int.
tlr_status check_sizes(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || n < 0 || k < 0 || m > PRODUCT_LIM || n > PRODUCT_LIM || k > SIZE_LIM)
    return fail(TLR_ERR_INVALID_ARG, "block_gemm: size out of range");
  if (cdiv(m, 128) * cdiv(n, 128) >= TILE_LIM) return fail(TLR_ERR_INVALID_ARG, "block_gemm: too many tiles for a launch");
  return TLR_OK;
}

// Workspace of a product in parts.
size_t parts_bytes(const Choice &c, int64_t m, int64_t n) { return c.parts > 1 ? sizeof(float) * (size_t)c.parts * m * n : 0; }

// Checks one result of the quantizer: rows x k codes with blocks of `block` rows.
tlr_status check_result(const char *name, int block, int64_t rows, int64_t k, const void *codes, int64_t ld,
                        const float *scales, int64_t lds) {
  const std::string w = std::string("block_quantize: ") + name;
  if (!scales) return fail(TLR_ERR_INVALID_ARG, w + ": null scales");
  if (!aligned(codes, 16) || ld % 16 != 0) return fail(TLR_ERR_INVALID_ARG, w + ": codes and their rows must be 16-byte aligned");
  if (!aligned(scales, 4)) return fail(TLR_ERR_INVALID_ARG, w + ": misaligned scales");
  if (ld < k) return fail(TLR_ERR_INVALID_ARG, w + ": leading dimension too small");
  if (lds < (block == 1 ? rows : (rows + QB - 1) / QB)) return fail(TLR_ERR_INVALID_ARG, w + ": scale leading dimension too small");
  return TLR_OK;
}

tlr_status check_operand(const char *name, const tlr_block_matrix *x, int64_t rows, int64_t k, Operand *o) {
  const std::string w = std::string("block_gemm: ") + name;
  if (!x || !x->codes || !x->scales) return fail(TLR_ERR_INVALID_ARG, w + ": null matrix, codes or scales");
  if (x->fmt != TLR_E4M3 && x->fmt != TLR_E5M2) return fail(TLR_ERR_INVALID_ARG, w + ": format must be TLR_E4M3 or TLR_E5M2");
  if (x->block != 1 && x->block != QB) return fail(TLR_ERR_INVALID_ARG, w + ": blocks are 1 or 128 rows high");
  if (x->ld % 16 != 0 || !aligned(x->codes, 16)) return fail(TLR_ERR_INVALID_ARG, w + ": codes and their rows must be 16-byte aligned");
  if (x->ld < k || x->ld >= LD_LIM) return fail(TLR_ERR_INVALID_ARG, w + ": leading dimension out of range");
  if (!aligned(x->scales, 4)) return fail(TLR_ERR_INVALID_ARG, w + ": misaligned scales");
  if (x->lds < (x->block == 1 ? rows : (rows + QB - 1) / QB) || x->lds > SIZE_LIM)
    return fail(TLR_ERR_INVALID_ARG, w + ": scale leading dimension out of range");
  o->codes = static_cast<const uint8_t *>(x->codes);
  o->scales = x->scales;
  o->ld = x->ld;
  o->lds = x->lds;
  o->rows = (int32_t)rows;
  o->shift = x->block == 1 ? 0 : 7;
  return TLR_OK;
}

}  // namespace

tlr_status block_quantize(tlr_dtype dt, tlr_dtype fmt, int32_t block, int64_t rows, int64_t k, const void *X,
                          int64_t ldx, void *codes, int64_t ldq, float *scales, int64_t lds, void *codes_t,
                          int64_t ldq_t, float *scales_t, int64_t lds_t, void *stream) {
  if (dt == TLR_F64) return fail(TLR_ERR_UNSUPPORTED, "block_quantize: TLR_F64 is not provided");
  if (dt != TLR_F32 && dt != TLR_F16 && dt != TLR_BF16) return fail(TLR_ERR_INVALID_ARG, "block_quantize: bad dtype");
  if (fmt != TLR_E4M3 && fmt != TLR_E5M2) return fail(TLR_ERR_INVALID_ARG, "block_quantize: format must be TLR_E4M3 or TLR_E5M2");
  if (block != 1 && block != QB) return fail(TLR_ERR_INVALID_ARG, "block_quantize: blocks are 1 or 128 rows high");
  if (rows < 0 || k < 0 || rows > SIZE_LIM || k > SIZE_LIM) return fail(TLR_ERR_INVALID_ARG, "block_quantize: size out of range");
  if ((rows + QB - 1) / QB > 65535) return fail(TLR_ERR_INVALID_ARG, "block_quantize: too many rows");
  if (((rows + QB - 1) / QB) * ((k + QB - 1) / QB) >= TILE_LIM) return fail(TLR_ERR_INVALID_ARG, "block_quantize: too many tiles");
  if (ldx < std::max<int64_t>(1, k)) return fail(TLR_ERR_INVALID_ARG, "block_quantize: leading dimension of X too small");
  if (rows == 0 || k == 0) return TLR_OK;
  if (!codes && !codes_t) return fail(TLR_ERR_INVALID_ARG, "block_quantize: no result wanted");
  if (codes) {
    const tlr_status st = check_result("codes", block, rows, k, codes, ldq, scales, lds);
    if (st != TLR_OK) return st;
  }
  if (codes_t) {
    const tlr_status st = check_result("codes_t", block, k, rows, codes_t, ldq_t, scales_t, lds_t);
    if (st != TLR_OK) return st;
  }
  const int es = dt == TLR_F32 ? 4 : 2;
  if (!X || !aligned(X, es)) return fail(TLR_ERR_INVALID_ARG, "block_quantize: null or misaligned X");
  QuantArgs a{X, rows, k, ldx, static_cast<uint8_t *>(codes), ldq, scales, lds,
              static_cast<uint8_t *>(codes_t), ldq_t, scales_t, lds_t, aligned(X, 16) && ldx * es % 16 == 0};
  // 8192 x 4096 bf16 both ways, whole lines: 28.6 us past the caches, 31.7
  // through them, 32.4 with the XCDs' parts; 5000 x 4136 float, split lines: 22.5
  // with the XCDs' parts, 25.3 without, 34.3 past the caches without.  Results
  // that fit into the caches are left there for their reader.
  auto lines = [](const void *p, int64_t ld) { return !p || (aligned(p, 128) && ld % 128 == 0); };
  const bool past = rows * k >= (int64_t)1 << 24 && lines(codes, ldq) && lines(codes_t, ldq_t);
  const unsigned grid = (unsigned)(((k + QB - 1) / QB) * ((rows + QB - 1) / QB));
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool e5 = fmt == TLR_E5M2;
  if (dt == TLR_F32) quantize_launch<float>(a, e5, block, past, grid, st);
  else if (dt == TLR_F16) quantize_launch<_Float16>(a, e5, block, past, grid, st);
  else quantize_launch<__bf16>(a, e5, block, past, grid, st);
  return launched("block_quantize");
}

tlr_status block_gemm_workspace(int64_t m, int64_t n, int64_t k, size_t *bytes) {
  if (!bytes) return fail(TLR_ERR_INVALID_ARG, "block_gemm_workspace_bytes: null output");
  const tlr_status st = check_sizes(m, n, k);
  if (st != TLR_OK) return st;
  *bytes = 0;
  if (m > 0 && n > 0 && k > 0)
    for (const bool fast : {false, true}) *bytes = std::max(*bytes, parts_bytes(choose(m, n, k, fast), m, n));
  return TLR_OK;
}

tlr_status block_gemm_plan(int64_t m, int64_t n, int64_t k, uint32_t flags, tlr_block_gemm_choice *out) {
  if (!out) return fail(TLR_ERR_INVALID_ARG, "block_gemm_plan: null output");
  if (flags & ~TLR_BLOCK_FAST) return fail(TLR_ERR_INVALID_ARG, "block_gemm_plan: unknown flags");
  const tlr_status st = check_sizes(m, n, k);
  if (st != TLR_OK) return st;
  *out = tlr_block_gemm_choice{};
  if (m == 0 || n == 0 || k == 0) return TLR_OK;
  const Choice c = choose(m, n, k, (flags & TLR_BLOCK_FAST) != 0);
  const Shape &s = SHAPE[c.kind];
  const int64_t x = workgroups(c.kind, m, n), y = c.kind == STRIP ? cdiv(n, 16) : 1;
  *out = tlr_block_gemm_choice{s.rows, s.cols, s.threads, s.halves, c.parts, 0, x, y, parts_bytes(c, m, n)};
  return TLR_OK;
}

tlr_status block_gemm(tlr_dtype dt, int64_t m, int64_t n, int64_t k, double alpha, const tlr_block_matrix *A,
                      const tlr_block_matrix *B, double beta, void *C, int64_t ldc, uint32_t flags, void *ws,
                      size_t ws_bytes, void *stream) {
  if (dt == TLR_F64) return fail(TLR_ERR_UNSUPPORTED, "block_gemm: C of type TLR_F64 is not provided");
  if (dt != TLR_F32 && dt != TLR_F16 && dt != TLR_BF16) return fail(TLR_ERR_INVALID_ARG, "block_gemm: bad dtype of C");
  if (flags & ~TLR_BLOCK_FAST) return fail(TLR_ERR_INVALID_ARG, "block_gemm: unknown flags");
  tlr_status st = check_sizes(m, n, k);
  if (st != TLR_OK) return st;
  if (ldc < std::max<int64_t>(1, m) || ldc > SIZE_LIM) return fail(TLR_ERR_INVALID_ARG, "block_gemm: ldc out of range");
  if (m == 0 || n == 0) return TLR_OK;
  GemmArgs g{};
  const bool product = k > 0 && alpha != 0.0;
  const Choice choice = product ? choose(m, n, k, (flags & TLR_BLOCK_FAST) != 0) : Choice{STRIP, 1};
  const size_t need = parts_bytes(choice, m, n);
  if (need > 0 && (!ws || !aligned(ws, 256))) return fail(TLR_ERR_INVALID_ARG, "block_gemm: null or misaligned workspace");
  if (ws_bytes < need) return fail(TLR_ERR_WORKSPACE, "block_gemm: workspace too small");
  if (product) {
    if ((st = check_operand("A", A, m, k, &g.a)) != TLR_OK) return st;
    if ((st = check_operand("B", B, n, k, &g.b)) != TLR_OK) return st;
  }
  if (!C || !aligned(C, dt == TLR_F32 ? 4 : 2)) return fail(TLR_ERR_INVALID_ARG, "block_gemm: null or misaligned C");
  if (!product) {
    if (beta == 1.0) return TLR_OK;
    const int e = launch_scale(dt, C, m, n, ldc, beta, stream);
    if (e) return fail(TLR_ERR_HIP, std::string("block_gemm: scale launch: ") + hipGetErrorString((hipError_t)e));
    return TLR_OK;
  }
  g.m = (int32_t)m;
  g.n = (int32_t)n;
  g.k = (int32_t)k;
  g.alpha = (float)alpha;
  g.beta = (float)beta;
  g.c = C;
  g.ldc = ldc;
  g.dt = dt;
  hipStream_t hs = static_cast<hipStream_t>(stream);
  float *part = static_cast<float *>(ws);
  const bool a5 = A->fmt == TLR_E5M2, b5 = B->fmt == TLR_E5M2;
  if (flags & TLR_BLOCK_FAST) {
    if (a5) b5 ? gemm_launch<true, true, true>(g, choice, part, hs) : gemm_launch<true, false, true>(g, choice, part, hs);
    else b5 ? gemm_launch<false, true, true>(g, choice, part, hs) : gemm_launch<false, false, true>(g, choice, part, hs);
  } else {
    if (a5) b5 ? gemm_launch<true, true, false>(g, choice, part, hs) : gemm_launch<true, false, false>(g, choice, part, hs);
    else b5 ? gemm_launch<false, true, false>(g, choice, part, hs) : gemm_launch<false, false, false>(g, choice, part, hs);
  }
  return launched("block_gemm");
}

}  // namespace tlr
