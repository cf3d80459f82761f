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
#include <string>

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
template <typename T, bool E5, int BLOCK>
__global__ __launch_bounds__(256) void quantize_kernel(QuantArgs a) {
  __shared__ uint32_t top[4][QB];
  __shared__ __attribute__((aligned(16))) uint8_t turn[QB][QB + 16];
  const int tid = threadIdx.x, c = tid & 15, r = tid >> 4, wave = tid >> 6;
  const int64_t c0 = (int64_t)blockIdx.x * QB, r0 = (int64_t)blockIdx.y * QB;
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
      if (a.codes) a.scales[blockIdx.y + blockIdx.x * a.lds] = tile_s;
      if (a.codes_t) a.scales_t[blockIdx.x + blockIdx.y * a.lds_t] = tile_s;
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
        if (c == i && row + i < a.rows) a.scales[row + i + blockIdx.x * a.lds] = s;
      }
      if (row + i < a.rows && col < ((a.k + 15) & ~(int64_t)15)) {
        u2 w;
        w[0] = codes4<E5>(quotient(v[i][0], s, q), quotient(v[i][1], s, q), quotient(v[i][2], s, q), quotient(v[i][3], s, q));
        w[1] = codes4<E5>(quotient(v[i][4], s, q), quotient(v[i][5], s, q), quotient(v[i][6], s, q), quotient(v[i][7], s, q));
        *reinterpret_cast<u2 *>(a.codes + (row + i) * a.ldq + col) = cut8(w, a.k - col);
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
        if (r == e && col + e < a.k) a.scales_t[col + e + blockIdx.y * a.lds_t] = s;
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
        *reinterpret_cast<u4 *>(a.codes_t + (c0 + x) * a.ldq_t + r0 + y) = *reinterpret_cast<const u4 *>(&turn[x][y]);
    }
  }
}

template <typename T>
void quantize_launch(const QuantArgs &a, bool e5, int block, dim3 grid, hipStream_t st) {
  if (e5) {
    if (block == 1) quantize_kernel<T, true, 1><<<grid, 256, 0, st>>>(a);
    else quantize_kernel<T, true, 128><<<grid, 256, 0, st>>>(a);
  } else {
    if (block == 1) quantize_kernel<T, false, 1><<<grid, 256, 0, st>>>(a);
    else quantize_kernel<T, false, 128><<<grid, 256, 0, st>>>(a);
  }
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
  int32_t vec;              // columns of C 16-byte aligned
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
template <bool A5, bool B5, bool FAST> __device__ __forceinline__ f4 mma(u4 a0, u4 a1, u4 b0, u4 b1) {
  f4 d = f4{0, 0, 0, 0};
  if constexpr (FAST) {
    const i8v a = __builtin_bit_cast(i8v, __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7));
    const i8v b = __builtin_bit_cast(i8v, __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7));
    d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, d, A5 ? 1 : 0, B5 ? 1 : 0, 0, 0, 0, 0);
  } else {
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<A5>(a0[0], a0[1]), widen8<B5>(b0[0], b0[1]), d, 0, 0, 0);
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<A5>(a0[2], a0[3]), widen8<B5>(b0[2], b0[3]), d, 0, 0, 0);
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<A5>(a1[0], a1[1]), widen8<B5>(b1[0], b1[1]), d, 0, 0, 0);
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<A5>(a1[2], a1[3]), widen8<B5>(b1[2], b1[3]), d, 0, 0, 0);
  }
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

// Eight consecutive rows of a column from row i.
__device__ __forceinline__ void store_c8(const GemmArgs &g, int i, int j, const float (&v)[8]) {
  if (!g.vec || i + 8 > g.m) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i + e < g.m) store_c(g, i + e, j, v[e]);
    return;
  }
  const int64_t at = (int64_t)j * g.ldc + i;
  float x[8];
  if (g.dt == TLR_F32) {
    f4 *p = reinterpret_cast<f4 *>(static_cast<float *>(g.c) + at);
    f4 lo = f4{0, 0, 0, 0}, hi = f4{0, 0, 0, 0};
    if (g.beta != 0.0f) { lo = p[0]; hi = p[1]; }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = g.beta != 0.0f ? v[e] * g.alpha + g.beta * (e < 4 ? lo[e & 3] : hi[e & 3]) : v[e] * g.alpha;
    p[0] = f4{x[0], x[1], x[2], x[3]};
    p[1] = f4{x[4], x[5], x[6], x[7]};
    return;
  }
  u4 *p = reinterpret_cast<u4 *>(static_cast<uint16_t *>(g.c) + at);
  u4 old = u4{0, 0, 0, 0};
  if (g.beta != 0.0f) old = *p;
  if (g.dt == TLR_F16) {
    typedef _Float16 h8 __attribute__((ext_vector_type(8)));
    const h8 o = __builtin_bit_cast(h8, old);
    h8 y;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (_Float16)(g.beta != 0.0f ? v[e] * g.alpha + g.beta * (float)o[e] : v[e] * g.alpha);
    *p = __builtin_bit_cast(u4, y);
  } else {
    const b8v o = __builtin_bit_cast(b8v, old);
    b8v y;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (__bf16)(g.beta != 0.0f ? v[e] * g.alpha + g.beta * (float)o[e] : v[e] * g.alpha);
    *p = __builtin_bit_cast(u4, y);
  }
}

// Few columns: a workgroup computes 16 rows of A against NJ x 16 rows of B, its
// eight waves taking every eighth block of the contraction; fragments come
// straight from global memory and the partial sums meet in LDS.
template <bool A5, bool B5, bool FAST, int NJ>
__global__ __launch_bounds__(512) void strip_kernel(GemmArgs g) {
  constexpr int W = 8;
  __shared__ float part[W][NJ][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int m0 = blockIdx.x * 16, n0 = blockIdx.y * 16 * NJ;
  const int ar = min(m0 + r, g.m - 1);
  const uint8_t *arow = g.a.codes + (int64_t)ar * g.a.ld;
  const uint8_t *brow[NJ];
  const float *bs[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int br = min(n0 + 16 * j + r, g.n - 1);
    brow[j] = g.b.codes + (int64_t)br * g.b.ld;
    bs[j] = g.b.scales + (br >> g.b.shift);
  }
  const float *as[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) as[v] = g.a.scales + (min(m0 + 4 * q + v, g.m - 1) >> g.a.shift);

  f4 acc[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[j] = f4{0, 0, 0, 0};
  const int nb = (g.k + QB - 1) / QB;
  for (int kb = wave; kb < nb; kb += W) {
    const int c = kb * QB + 16 * q;
    const u4 a0 = load16(arow, c, g.k), a1 = load16(arow, c + 64, g.k);
    float sa[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) sa[v] = as[v][kb * g.a.lds];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const u4 b0 = load16(brow[j], c, g.k), b1 = load16(brow[j], c + 64, g.k);
      const float sb = bs[j][kb * g.b.lds];
      const f4 d = mma<A5, B5, FAST>(a0, a1, b0, b1);
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[j][v] = __builtin_fmaf(sa[v] * sb, d[v], acc[j][v]);
    }
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) part[wave][j][v][lane] = acc[j][v];
  __syncthreads();
  for (int x = threadIdx.x; x < NJ * 256; x += 512) {
    const int i = x & 15, j = x >> 4;      // row, column of the workgroup's block
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += part[w][j >> 4][i & 3][(i >> 2) * 16 + (j & 15)];
    if (m0 + i < g.m && n0 + j < g.n) store_c(g, m0 + i, n0 + j, v);
  }
}

// ---- product, tiles ----------------------------------------------------------------------------------

// Loads through a buffer descriptor: lanes at or past its size write zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *p, int32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, bytes, 0x00027000);
}
typedef __attribute__((address_space(3))) void *lds_ptr;
__device__ __forceinline__ void to_lds16(__amdgpu_buffer_rsrc_t b, uint32_t at, void *lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_ptr)lds, 16, at, 0, 0, 0);
}
__device__ __forceinline__ void to_lds4(__amdgpu_buffer_rsrc_t b, uint32_t at, void *lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_ptr)lds, 4, at, 0, 0, 0);
}

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
  __device__ __forceinline__ void init(const Operand &o, int r0, int k, int tid) {
    base = o.codes + (int64_t)r0 * o.ld;
    bytes = (min(ROWS, o.rows - r0) - 1) * (int32_t)o.ld + ((k + 15) & ~15);
    step = (T / 8) * (int32_t)o.ld;
    at = (uint32_t)(tid >> 3) * (uint32_t)o.ld + chunk(tid);
  }
  static __device__ __forceinline__ int chunk(int tid) {
    return 16 * ((tid & 7) ^ (IS_A ? a_key(tid >> 3) : b_key(tid >> 3)));
  }
  // a descriptor of the rows from step i on: the steps share one address register
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(int kb, int i) const {
    const int32_t o = kb * QB + i * step;
    return buffer(base + o, max(bytes - o, 0));
  }
  __device__ __forceinline__ void load(int kb, uint8_t *lds, int wave) const {
#pragma unroll
    for (int i = 0; i < N; ++i) to_lds16(rows(kb, i), at, lds + (i * T + wave * 64) * 16);
  }
  // the last column block, whose columns from `left` on read as zero
  __device__ __forceinline__ void load_cut(int kb, int left, uint8_t *lds, int tid) const {
    u4 x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(rows(kb, i), at, 0, 0));
    u4 keep;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int n = left - chunk(tid) - 4 * w;
      keep[w] = n >= 4 ? 0xffffffffu : n <= 0 ? 0u : 0xffffffffu >> (32 - 8 * n);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<u4 *>(lds + (i * T + tid) * 16) = x[i] & keep;
  }
};

// C tiles of TM x TN, WM x WN waves.  AB: A's blocks are 128 rows high (a wave's
// rows lie in one of them, or in two halves).
template <bool A5, bool B5, bool FAST, bool AB, int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2))) void tile_kernel(GemmArgs g) {
  constexpr int T = 64 * WM * WN, RI = TM / WM / 16, CJ = TN / WN / 16;
  __shared__ __attribute__((aligned(16))) uint8_t a0[TM * QB], a1[TM * QB], b0[TN * QB], b1[TN * QB];
  __shared__ __attribute__((aligned(16))) float s0[TM + TN], s1[TM + TN];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4, wm = wave / WN, wn = wave % WN;

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
  // scales: TM + TN floats a stage, 64 a wave and step
  constexpr int SN = (TM + TN) / T;
  static_assert((TM + TN) % T == 0 && TM % 64 == 0, "");
  auto load_scales = [&](int kb, float *ls) {
#pragma unroll
    for (int i = 0; i < SN; ++i) {
      const int w = i * T + wave * 64;
      const bool isa = w < TM;
      const Operand &o = isa ? g.a : g.b;
      const int r0 = isa ? m0 : n0, at = (isa ? w : w - TM) + lane;
      const int first = r0 >> o.shift, n = ((min(r0 + (isa ? TM : TN), o.rows) - 1) >> o.shift) - first + 1;
      to_lds4(buffer(o.scales + kb * o.lds + first, 4 * n), 4 * (((r0 + at) >> o.shift) - first), ls + w);
    }
  };
  auto load = [&](int kb, uint8_t *la, uint8_t *lb, float *ls) {
    load_scales(kb, ls);
    pa.load(kb, la, wave);
    pb.load(kb, lb, wave);
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
  const int aat = ar * QB + 16 * (q ^ a_key(ar)), bat = br * QB + 16 * (q ^ b_key(br));

  auto compute = [&](const uint8_t *la, const uint8_t *lb, const float *ls) {
    u4 bf[CJ][2];
    float sb[CJ];
#pragma unroll
    for (int j = 0; j < CJ; ++j) {
      bf[j][0] = *reinterpret_cast<const u4 *>(lb + bat + 16 * QB * j);
      bf[j][1] = *reinterpret_cast<const u4 *>(lb + (bat ^ 64) + 16 * QB * j);
      sb[j] = ls[TM + br + 16 * j];
    }
    if constexpr (AB) {
      const float s = ls[wm * (TM / WM)];
#pragma unroll
      for (int j = 0; j < CJ; ++j) sb[j] *= s;
    }
    // Row tile by row tile: the next one's fragment is read and the last one's
    // results are added while the matrix instructions of this one run.
    auto frag = [&](int i, u4 (&x)[2]) {
      const int o = (i >> 1) * 32 * QB + (i & 1) * 4 * QB;
      x[0] = *reinterpret_cast<const u4 *>(la + aat + o);
      x[1] = *reinterpret_cast<const u4 *>(la + (aat ^ 64) + o);
    };
    auto add = [&](int i, const f4 (&d)[CJ]) {
      f4 sa;
      if constexpr (!AB) sa = *reinterpret_cast<const f4 *>(ls + wm * (TM / WM) + (i >> 1) * 32 + 8 * q + 4 * (i & 1));
#pragma unroll
      for (int j = 0; j < CJ; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(AB ? sb[j] : sa[v] * sb[j], d[j][v], acc[i][j][v]);
    };
    u4 x[2][2];
    f4 d[2][CJ];
    frag(0, x[0]);
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      if (i + 1 < RI) frag(i + 1, x[(i + 1) & 1]);
#pragma unroll
      for (int j = 0; j < CJ; ++j) d[i & 1][j] = mma<A5, B5, FAST>(x[i & 1][0], x[i & 1][1], bf[j][0], bf[j][1]);
      if (i > 0) add(i - 1, d[(i - 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
    add(RI - 1, d[(RI - 1) & 1]);
  };
  auto meet = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // Stage 0 is the last column block, which may be cut at column k; stage i > 0
  // is column block i - 1.  Stages alternate between the buffers, the last one
  // is in the second.
  const int nb = (g.k + QB - 1) / QB;
  bool second = nb & 1;
  load_scales(nb - 1, second ? s1 : s0);
  if (g.k & (QB - 1)) {
    pa.load_cut(nb - 1, g.k & (QB - 1), second ? a1 : a0, tid);
    pb.load_cut(nb - 1, g.k & (QB - 1), second ? b1 : b0, tid);
  } else {
    pa.load(nb - 1, second ? a1 : a0, wave);
    pb.load(nb - 1, second ? b1 : b0, wave);
  }
  meet();
  int kb = 0;               // column block of the next stage to load
  do {
    if (!second) {
      load(kb++, a1, b1, s1);
      compute(a0, b0, s0);
      meet();
    }
    second = false;
    if (kb < nb - 1) load(kb, a0, b0, s0);
    compute(a1, b1, s1);
    meet();
  } while (kb++ < nb - 1);

  // lane (r, q): rows 32 h + 8 q .. + 7 of its columns
#pragma unroll
  for (int j = 0; j < CJ; ++j) {
    const int col = n0 + wn * (TN / WN) + 16 * j + r;
    if (col < g.n)
#pragma unroll
      for (int h = 0; h < RI / 2; ++h) {
        const int row = m0 + wm * (TM / WM) + 32 * h + 8 * q;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = acc[2 * h + (e >> 2)][j][e & 3];
        store_c8(g, row, col, v);
      }
  }
}

template <bool A5, bool B5, bool FAST, int TM, int TN, int WM, int WN> void tile_launch(const GemmArgs &g, hipStream_t st) {
  const unsigned grid = (unsigned)((g.m + TM - 1) / TM) * (unsigned)((g.n + TN - 1) / TN);
  if (g.a.shift) tile_kernel<A5, B5, FAST, true, TM, TN, WM, WN><<<grid, 64 * WM * WN, 0, st>>>(g);
  else tile_kernel<A5, B5, FAST, false, TM, TN, WM, WN><<<grid, 64 * WM * WN, 0, st>>>(g);
}

template <bool A5, bool B5, bool FAST> void gemm_launch(const GemmArgs &g, hipStream_t st) {
  const unsigned gx = (unsigned)((g.m + 15) / 16);
  if (g.n <= 16) strip_kernel<A5, B5, FAST, 1><<<dim3(gx, 1), 512, 0, st>>>(g);
  else if (g.n <= 32) strip_kernel<A5, B5, FAST, 2><<<dim3(gx, 1), 512, 0, st>>>(g);
  else if (g.n <= 64) strip_kernel<A5, B5, FAST, 4><<<dim3(gx, (g.n + 63) / 64), 512, 0, st>>>(g);
  else if ((int64_t)((g.m + 255) / 256) * ((g.n + 255) / 256) >= 192) tile_launch<A5, B5, FAST, 256, 256, 2, 4>(g, st);
  else tile_launch<A5, B5, FAST, 128, 128, 2, 2>(g, st);
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

tlr_status launched(const char *what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TLR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
  return TLR_OK;
}

constexpr int64_t SIZE_LIM = 0x7fffffff, LD_LIM = (int64_t)1 << 22;

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
  const dim3 grid((unsigned)((k + QB - 1) / QB), (unsigned)((rows + QB - 1) / QB));
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool e5 = fmt == TLR_E5M2;
  if (dt == TLR_F32) quantize_launch<float>(a, e5, block, grid, st);
  else if (dt == TLR_F16) quantize_launch<_Float16>(a, e5, block, grid, st);
  else quantize_launch<__bf16>(a, e5, block, grid, st);
  return launched("block_quantize");
}

tlr_status block_gemm_workspace(int64_t m, int64_t n, int64_t k, size_t *bytes) {
  if (!bytes) return fail(TLR_ERR_INVALID_ARG, "block_gemm_workspace_bytes: null output");
  if (m < 0 || n < 0 || k < 0 || m > SIZE_LIM || n > SIZE_LIM || k > SIZE_LIM)
    return fail(TLR_ERR_INVALID_ARG, "block_gemm_workspace_bytes: size out of range");
  *bytes = 0;
  return TLR_OK;
}

tlr_status block_gemm(tlr_dtype dt, int64_t m, int64_t n, int64_t k, double alpha, const tlr_block_matrix *A,
                      const tlr_block_matrix *B, double beta, void *C, int64_t ldc, uint32_t flags, void *ws,
                      size_t ws_bytes, void *stream) {
  if (dt == TLR_F64) return fail(TLR_ERR_UNSUPPORTED, "block_gemm: C of type TLR_F64 is not provided");
  if (dt != TLR_F32 && dt != TLR_F16 && dt != TLR_BF16) return fail(TLR_ERR_INVALID_ARG, "block_gemm: bad dtype of C");
  if (flags & ~TLR_BLOCK_FAST) return fail(TLR_ERR_INVALID_ARG, "block_gemm: unknown flags");
  size_t need = 0;
  tlr_status st = block_gemm_workspace(m, n, k, &need);
  if (st != TLR_OK) return st;
  if (ldc < std::max<int64_t>(1, m) || ldc > SIZE_LIM) return fail(TLR_ERR_INVALID_ARG, "block_gemm: ldc out of range");
  if (m == 0 || n == 0) return TLR_OK;
  if (need > 0 && (!ws || !aligned(ws, 256))) return fail(TLR_ERR_INVALID_ARG, "block_gemm: null or misaligned workspace");
  if (ws_bytes < need) return fail(TLR_ERR_WORKSPACE, "block_gemm: workspace too small");
  GemmArgs g{};
  const bool product = k > 0 && alpha != 0.0;
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
  g.vec = aligned(C, 16) && ldc * (dt == TLR_F32 ? 4 : 2) % 16 == 0;
  hipStream_t hs = static_cast<hipStream_t>(stream);
  const bool a5 = A->fmt == TLR_E5M2, b5 = B->fmt == TLR_E5M2;
  if (flags & TLR_BLOCK_FAST) {
    if (a5) b5 ? gemm_launch<true, true, true>(g, hs) : gemm_launch<true, false, true>(g, hs);
    else b5 ? gemm_launch<false, true, true>(g, hs) : gemm_launch<false, false, true>(g, hs);
  } else {
    if (a5) b5 ? gemm_launch<true, true, false>(g, hs) : gemm_launch<true, false, false>(g, hs);
    else b5 ? gemm_launch<false, true, false>(g, hs) : gemm_launch<false, false, false>(g, hs);
  }
  return launched("block_gemm");
}

}  // namespace tlr
