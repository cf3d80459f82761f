// 8-bit integers with a float scale for each row: quantizer and matrix product
// for gfx950.
//
//   C[i,j] = sA(i) sB(j) sum_c a[i,c] b[j,c]
// The sum is one of 32-bit integers and exact, whatever its order, for up to
// 131071 columns; it is converted to float, multiplied by the scale of its column
// (a token) and then of its row (a channel), and rounded to C's type once.
// Grouped, the rows of B are cut into consecutive groups, each with an A of its own
// (a weight for each expert).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "int8.h"
#include "tlr_ops.h"

namespace tlr {

namespace {

typedef int i4 __attribute__((ext_vector_type(4)));

constexpr int MOST_GROUPS = 1024;

// ---- quantizer ---------------------------------------------------------------------------------------

struct RowQuantArgs {
  const void *x;
  int64_t rows, x_rows, ldx, ldq;
  const int32_t *index;
  uint8_t *codes;
  float *scales;
  int32_t k;
};

__device__ __forceinline__ uint32_t max64(uint32_t x) {
  x = max16(x);
  x = max(x, (uint32_t)__shfl_xor((int)x, 16));
  return max(x, (uint32_t)__shfl_xor((int)x, 32));
}

// A row is read once into the registers of W waves, U vectors of 8 entries a lane
// (U 0: too long for them, read twice).  One wave: four rows a workgroup.
template <typename T, int W, int U, bool PAST> __global__ __launch_bounds__(256) void row_quantize_kernel(RowQuantArgs a) {
  __shared__ uint32_t top[4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int STEP = W * 512;
  const int at = W == 1 ? lane * 8 : threadIdx.x * 8, up = (a.k + 15) & ~15;
  for (int64_t r = W == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x; r < a.rows; r += (int64_t)gridDim.x * (W == 1 ? 4 : 1)) {
    const int64_t from = a.index ? a.index[r] : r;
    const bool none = from < 0 || from >= a.x_rows;       // a row of zeros
    const T *x = static_cast<const T *>(a.x) + (none ? 0 : from * a.ldx);
    const int k = none ? 0 : a.k;
    float v[U > 0 ? U : 1][8];
    uint32_t m = 0;
    if constexpr (U > 0) {
      Eight<T> in[U];
      if (k >= 8) {             // all loads at once, from the row's end where there is nothing else
#pragma unroll
        for (int u = 0; u < U; ++u) in[u].template load<true>(x + min(at + u * STEP, k - 8), 8);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int left = k - at - u * STEP;
        if (left <= 0) in[u] = Eight<T>{};
        else if (left < 8) in[u].template load<false>(x + at + u * STEP, left);
        in[u].get(v[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, mag(v[u][e]));
    } else {
      for (int c = at; c < k; c += STEP) {
        get8(x + c, k - c, v[0]);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, mag(v[0][e]));
      }
    }
    m = max64(m);
    if constexpr (W > 1) {
      __syncthreads();
      if (lane == 0) top[wave] = m;
      __syncthreads();
      m = max(max(top[0], top[1]), max(top[2], top[3]));
    }
    const float s = int8_scale(m), q = 1.0f / s;
    if (at == 0) a.scales[r] = s;
    uint8_t *out = a.codes + r * a.ldq;
    if constexpr (U > 0) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (at + u * STEP < up) {
          u2 *to = reinterpret_cast<u2 *>(out + at + u * STEP);
          const u2 w = int8_codes8(v[u], s, q);
          if constexpr (PAST) __builtin_nontemporal_store(w, to);
          else *to = w;
        }
    } else {
      for (int c = at; c < up; c += STEP) {
        get8(x + c, k - c, v[0]);
        *reinterpret_cast<u2 *>(out + c) = int8_codes8(v[0], s, q);
      }
    }
  }
}

// Results that fit into the caches are left there for their reader (8192 x 2048 past
// them 8.4 us, through them 9.9; 32768 x 2048 28.7 and 30.0).  A few rows of up to 2048
// entries go to a workgroup each (96: 2.6 us, a wave each 2.8).
template <typename T, bool PAST> void row_quantize_launch(const RowQuantArgs &a, hipStream_t st) {
  const unsigned one = (unsigned)std::min<int64_t>((a.rows + 3) / 4, 1 << 22), all = (unsigned)std::min<int64_t>(a.rows, 1 << 22);
  if (a.k <= 512) row_quantize_kernel<T, 1, 1, PAST><<<one, 256, 0, st>>>(a);
  else if (a.k <= 2048 && a.rows < 512) row_quantize_kernel<T, 4, 1, false><<<all, 256, 0, st>>>(a);
  else if (a.k <= 2048) row_quantize_kernel<T, 1, 4, PAST><<<one, 256, 0, st>>>(a);
  else if (a.k <= 4096) row_quantize_kernel<T, 4, 2, PAST><<<all, 256, 0, st>>>(a);
  else if (a.k <= 8192) row_quantize_kernel<T, 4, 4, PAST><<<all, 256, 0, st>>>(a);
  else row_quantize_kernel<T, 4, 0, false><<<all, 256, 0, st>>>(a);
}
template <typename T> void row_quantize_launch(const RowQuantArgs &a, hipStream_t st) {
  if (a.rows * a.k >= (int64_t)1 << 24) row_quantize_launch<T, true>(a, st);
  else row_quantize_launch<T, false>(a, st);
}

// ---- product -----------------------------------------------------------------------------------------

struct Operand {
  const uint8_t *codes;
  const float *scales;
  int64_t ld;
  int32_t rows;
};

struct RowGemmArgs {
  Operand a, b;
  int32_t m, n, k;
  void *c;
  int64_t ldc;
  int32_t dt;
  // groups of B's rows (offsets null: one of all rows, with A)
  const int32_t *offsets;
  int64_t code_step, scale_step;        // from one group's A to the next
  int32_t groups, clear;                // clear: rows of no group become zeros
};

// The rows of B that a workgroup takes, and what belongs to them.
struct Rows {
  int first, end;           // end: of the group
  int group;                // -1: nothing to do; `groups`: zeros
};

__device__ __forceinline__ int scan64(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(x, d);
    if (lane >= d) x += v;
  }
  return x;
}

// Pieces of TN rows, counted through the groups, those of the rows behind the last group
// and before the first (to be zeroed) at the end.  A lane has one of 64 groups; with more
// of them they are gone through again to find a piece.  Offsets out of order or range give
// empty or shorter groups.
template <int TN> struct Pieces {
  const RowGemmArgs &g;
  int lane, lo, hi, mine, upto;         // of the lane's group in the 64 looked at last
  int in_groups, behind, front, in_behind, total;        // in_groups, in_behind: pieces
  __device__ __forceinline__ void look(int e0, int before) {
    const int e = e0 + lane;
    lo = e < g.groups ? min(max(g.offsets[e], 0), g.n) : 0;
    hi = e < g.groups ? max(lo, min(max(g.offsets[e + 1], 0), g.n)) : 0;
    mine = (hi - lo + TN - 1) / TN;
    upto = before + scan64(mine, lane);
  }
  __device__ __forceinline__ Pieces(const RowGemmArgs &args) : g(args), lane(threadIdx.x & 63) {
    behind = g.clear ? min(max(g.offsets[g.groups], 0), g.n) : g.n;
    front = g.clear ? min(max(g.offsets[0], 0), g.n) : 0;
    in_groups = 0;
    for (int e0 = 0; e0 < g.groups; e0 += 64) {
      look(e0, in_groups);
      in_groups = __builtin_amdgcn_readlane(upto, 63);
    }
    in_behind = (g.n - behind + TN - 1) / TN;
    total = in_groups + in_behind + (front + TN - 1) / TN;
  }
  __device__ __forceinline__ Rows find(int at) {
    if (at >= in_groups) {
      const bool last = at - in_groups < in_behind;
      const int from = last ? behind : 0, end = last ? g.n : front, first = from + (at - in_groups - (last ? 0 : in_behind)) * TN;
      return first >= from && first < end ? Rows{first, end, g.groups} : Rows{0, 0, -1};
    }
    int e0 = 0, before = 0;
    if (g.groups > 64) look(0, 0);
    while (true) {
      const uint64_t past = __ballot(at < upto);
      if (past) {
        const int l = __builtin_ctzll(past);
        const int start = __builtin_amdgcn_readlane(upto - mine, l), from = __builtin_amdgcn_readlane(lo, l), end = __builtin_amdgcn_readlane(hi, l);
        const int first = from + (at - start) * TN;
        // always so, unless groups that overlap have more pieces than an int counts
        return first >= from && first < end ? Rows{first, end, e0 + l} : Rows{0, 0, -1};
      }
      before = __builtin_amdgcn_readlane(upto, 63);
      e0 += 64;
      if (e0 >= g.groups) return Rows{0, 0, -1};
      look(e0, before);
    }
  }
};

template <int TN> struct Whole {
  int total;
  __device__ __forceinline__ Whole(const RowGemmArgs &g) : total((g.n + TN - 1) / TN) {}
};

// A's codes and scales for a group.
__device__ __forceinline__ void take_group(RowGemmArgs &g, const Rows &r) {
  g.a.codes += r.group * g.code_step;
  g.a.scales += r.group * g.scale_step;
  g.b.rows = r.end;
  g.n = r.end;
}

__device__ __forceinline__ void store_one(const RowGemmArgs &g, int i, int j, float v) {
  const int64_t at = (int64_t)j * g.ldc + i;
  if (g.dt == TLR_F32) static_cast<float *>(g.c)[at] = v;
  else if (g.dt == TLR_F16) static_cast<_Float16 *>(g.c)[at] = (_Float16)v;
  else static_cast<__bf16 *>(g.c)[at] = (__bf16)v;
}

// Eight consecutive rows of a column of C from row i on, those that C has.
__device__ __forceinline__ void store8(const RowGemmArgs &g, int i, int j, const float (&v)[8]) {
  const int64_t at = (int64_t)j * g.ldc + i;
  if (g.dt == TLR_F32) put8(static_cast<float *>(g.c) + at, g.m - i, v);
  else if (g.dt == TLR_F16) put8(static_cast<_Float16 *>(g.c) + at, g.m - i, v);
  else put8(static_cast<__bf16 *>(g.c) + at, g.m - i, v);
}

// Eight consecutive sums of a column, those before `left`.
__device__ __forceinline__ void put_sums(int *p, int left, const int (&v)[8]) {
  if (left >= 8) __builtin_memcpy(p, v, 32);
  else
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) p[e] = v[e];
}

// Few columns or little work: a workgroup computes 16 rows of A against 16 NJ rows of
// B, its eight waves taking every eighth block of 128 columns; fragments come straight
// from global memory, UNROLL blocks of a wave at once (whole or not: those behind the
// last are zeros), and the partial sums meet in LDS.
template <bool GROUPED, int NJ> __global__ __launch_bounds__(512, 4) void strip_kernel(RowGemmArgs g) {
  constexpr int W = 8, UNROLL = 2, TN = 16 * NJ;
  __shared__ int part[W][4 * NJ][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int m0 = blockIdx.x * 16;
  int n0 = blockIdx.y * TN;
  bool zero = false;
  if constexpr (GROUPED) {
    const Rows rows = Pieces<TN>(g).find(blockIdx.y);
    if (rows.group < 0) return;
    n0 = rows.first;
    zero = rows.group == g.groups;
    take_group(g, zero ? Rows{rows.first, rows.end, 0} : rows);
  }
  const uint8_t *arow = g.a.codes + (int64_t)min(m0 + r, g.m - 1) * g.a.ld + 16 * q;
  const uint8_t *brow[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) brow[j] = g.b.codes + (int64_t)min(n0 + 16 * j + r, g.n - 1) * g.b.ld + 16 * q;
  i4 acc[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[j] = i4{0, 0, 0, 0};
  const int full = zero ? 0 : g.k / QB, blocks = zero ? 0 : (g.k + QB - 1) / QB;
  for (int kb = wave; kb < blocks; kb += UNROLL * W) {
    u4 a[UNROLL][2], b[UNROLL][NJ][2];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int at = kb + u * W;
      const int64_t c = (int64_t)at * QB;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (at < full) {
          a[u][h] = *reinterpret_cast<const u4 *>(arow + c + 64 * h);
#pragma unroll
          for (int j = 0; j < NJ; ++j) b[u][j][h] = *reinterpret_cast<const u4 *>(brow[j] + c + 64 * h);
        } else {
          // the cut block: zeros from column k on in one operand are enough
          const bool cut = at < blocks && 16 * q + 64 * h < g.k - full * QB;
          a[u][h] = at < blocks ? load16(arow + c - 16 * q, 16 * q + 64 * h, g.k - full * QB) : u4{0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < NJ; ++j) b[u][j][h] = cut ? *reinterpret_cast<const u4 *>(brow[j] + c + 64 * h) : u4{0, 0, 0, 0};
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i4, a[u][h]), __builtin_bit_cast(i4, b[u][j][h]), acc[j], 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) part[wave][4 * j + v][lane] = acc[j][v];
  __syncthreads();
#pragma unroll
  for (int j0 = 0; j0 < NJ; j0 += 2) {
    const int i = threadIdx.x & 15, j = j0 + (threadIdx.x >> 8), c = threadIdx.x >> 4 & 15;      // row, strip and column of the workgroup's block
    if (j < NJ) {
      int v = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) v += part[w][4 * j + (i & 3)][(i >> 2) * 16 + c];
      const int col = n0 + 16 * j + c;
      if (m0 + i < g.m && col < g.n) store_one(g, m0 + i, col, zero ? 0.0f : (float)v * g.b.scales[col] * g.a.scales[m0 + i]);
    }
  }
}

// A few tokens, quantized by every workgroup for itself: codes and scales stand in LDS,
// and the strip's product follows, its first weights under way while x is read.  One
// launch where quantizer and product are two: 8192 x 1 x 4096 7.0 us, 9.5 (the product
// alone 6.8); 8192 x 4 x 4096 10.0, 10.4; 4096 x 8 x 2048 5.5, 6.2.
constexpr int FEW_TOKENS = 8, FEW = 16384;       // tokens, and entries of all of them
__host__ __device__ constexpr int few_waves(int64_t n) { return n == 1 ? 8 : n == 2 ? 4 : n <= 4 ? 2 : 1; }     // for each token
template <typename T> __global__ __launch_bounds__(512, 4) void few_kernel(RowGemmArgs g, const void *xp, int64_t ldx) {
  constexpr int W = 8, AHEAD = 4, MOST = FEW_TOKENS;       // eight waves, as many as tokens at most
  __shared__ __attribute__((aligned(16))) uint8_t codes[FEW + MOST * QB];
  __shared__ int part[W][4][64];
  __shared__ uint32_t top[W];
  __shared__ float scale[MOST];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4, m0 = blockIdx.x * 16;
  const uint8_t *arow = g.a.codes + (int64_t)min(m0 + r, g.m - 1) * g.a.ld + 16 * q;
  const int blocks = (g.k + QB - 1) / QB, full = g.k / QB, ld = blocks * QB;      // rows of whole blocks in LDS, zeros behind column k
  u4 ahead[AHEAD][2];
#pragma unroll
  for (int u = 0; u < AHEAD; ++u)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int kb = wave + u * W;
      ahead[u][h] = kb < full ? *reinterpret_cast<const u4 *>(arow + kb * QB + 64 * h) : u4{0, 0, 0, 0};
    }
  // the waves share the tokens: eight, four, two or one of them for each
  const int waves = few_waves(g.n), j = wave / waves, step = 512 * waves, at = 512 * (wave % waves) + 8 * lane;
  const T *x = static_cast<const T *>(xp) + min(j, g.n - 1) * ldx;
  float v[8];
  if (j < g.n) {
    uint32_t m = 0;
    for (int c = at; c < g.k; c += step) {
      get8(x + c, g.k - c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, mag(v[e]));
    }
    m = max64(m);
    if (lane == 0) top[wave] = m;
  }
  __syncthreads();
  if (j < g.n) {
    uint32_t m = top[wave];
    for (int w = 0; w < waves; ++w) m = max(m, top[j * waves + w]);
    const float s = int8_scale(m), inverse = 1.0f / s;
    if (at == 0) scale[j] = s;
    for (int c = at; c < ld; c += step) {
      if (ld > step || c >= g.k) get8(x + min(c, g.k), g.k - c, v);
      *reinterpret_cast<u2 *>(codes + j * ld + c) = int8_codes8(v, s, inverse);
    }
  }
  __syncthreads();
  i4 acc = i4{0, 0, 0, 0};
  const uint8_t *brow = codes + min(r, g.n - 1) * ld + 16 * q;
  auto add = [&](int kb, const u4 (&x)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i4, x[h]), *reinterpret_cast<const i4 *>(brow + kb * QB + 64 * h), acc, 0, 0, 0);
  };
#pragma unroll
  for (int u = 0; u < AHEAD; ++u)
    if (wave + u * W < full) add(wave + u * W, ahead[u]);
  int kb = wave + AHEAD * W;
  for (; kb + (AHEAD - 1) * W < full; kb += AHEAD * W) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) ahead[u][h] = *reinterpret_cast<const u4 *>(arow + (kb + u * W) * QB + 64 * h);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) add(kb + u * W, ahead[u]);
  }
  for (; kb < full; kb += W) {
#pragma unroll
    for (int h = 0; h < 2; ++h) ahead[0][h] = *reinterpret_cast<const u4 *>(arow + kb * QB + 64 * h);
    add(kb, ahead[0]);
  }
  if (full < blocks && wave == full % W) {                // the cut block
#pragma unroll
    for (int h = 0; h < 2; ++h) ahead[0][h] = load16(arow + full * QB - 16 * q, 16 * q + 64 * h, g.k - full * QB);
    add(full, ahead[0]);
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) part[wave][v][lane] = acc[v];
  __syncthreads();
  if (tid < 256) {
    const int i = tid & 15, j = tid >> 4;
    int v = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) v += part[w][i & 3][(i >> 2) * 16 + j];
    if (m0 + i < g.m && j < g.n) store_one(g, m0 + i, j, (float)v * scale[j] * g.a.scales[m0 + i]);
  }
}

// All waves of a workgroup, once this one has no LDS access under way; its loads go on.
__device__ __forceinline__ void meet_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xf | 3 << 14 | 7 << 4);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A wave's sums, scaled, to C from row m0 and column n0 on, up to column `end`.  They go
// through 2 KB of LDS that only this wave uses, 16 columns of 128 bytes at a time, so that
// no wave waits for another: a wave's accesses to LDS stay in their order.  STORES of
// them, where all of the entries exist.
template <typename E, int RI, int CJ, bool PAST> struct WaveStore {
  static constexpr int HS = 4 / sizeof(E), STORES = RI * CJ * (int)sizeof(E) / 4;      // pairs of row tiles at a time
  static __device__ __forceinline__ void run(const RowGemmArgs &g, const i4 (&acc)[RI][CJ], uint8_t *slice, const float *row_scales,
                                             const float *column_scales, int m0, int n0, int end, int lane) {
    const int r = lane & 15, q = lane >> 4;
    static_assert(RI % (2 * HS) == 0, "");
#pragma unroll
    for (int h0 = 0; h0 < RI / 2; h0 += HS) {
      float sa[HS][8];
#pragma unroll
      for (int h = 0; h < HS; ++h) __builtin_memcpy(sa[h], __builtin_assume_aligned(row_scales + 32 * (h0 + h) + 8 * q, 16), sizeof sa[h]);
#pragma unroll
      for (int j = 0; j < CJ; ++j) {
        const float sb = column_scales[16 * j + r];
#pragma unroll
        for (int h = 0; h < HS; ++h) {
          E v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = (E)((float)acc[2 * (h0 + h) + (e >> 2)][j][e & 3] * sb * sa[h][e]);
          u4 w[sizeof v / 16];
          __builtin_memcpy(w, v, sizeof v);
#pragma unroll
          for (int p = 0; p < (int)(sizeof v / 16); ++p)
            *reinterpret_cast<u4 *>(slice + r * 128 + 16 * (((4 * h + q) * (int)(sizeof v / 16) + p) ^ (r & 7))) = w[p];
        }
        asm volatile("" ::: "memory");
        u4 w[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int at = 8 * t + (lane >> 3);
          w[t] = *reinterpret_cast<const u4 *>(slice + at * 128 + 16 * ((lane & 7) ^ (at & 7)));
        }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          constexpr int N = 16 / sizeof(E);
          const int col = n0 + 16 * j + 8 * t + (lane >> 3), row = m0 + 32 * h0 + N * (lane & 7);
          if (col < end && row < g.m) {
            E *to = static_cast<E *>(g.c) + (int64_t)col * g.ldc + row;
            if (row + N <= g.m) {
              put16<PAST>(to, w[t]);
            } else {
              E v[N];
              __builtin_memcpy(v, &w[t], 16);
#pragma unroll
              for (int e = 0; e < N - 1; ++e)
                if (row + e < g.m) to[e] = v[e];
            }
          }
        }
      }
    }
  }
};

// C tiles of TM x TN, WM x WN waves, each RI x CJ tiles of 16 x 16; blocks of 128
// columns pass through a ring of NS stages in LDS.  A wave goes through a stage row tile
// by row tile; with the last one's matrix instructions under way it waits for the next
// stage and reads its first fragments: one barrier a stage, and the matrix cores have
// work on both sides of it.  The buffer that is then used up takes the stage NS further
// on.  A short stage is computed faster than its loads arrive: with three of them
// 2000 x 1000 x 8000 in 128 x 64 tiles takes 27.6 us, with two 42, with four 27.7;
// 2501 x 1111 x 1747 in 128 x 128 on eight waves 13.6, 15.0, 13.8.  128 x 128 on four
// waves keep two, so that two workgroups fit a CU: 2048 x 4096 x 2048 22, with three 34.
template <bool GROUPED, int TM, int TN, int WM, int WN, int NS>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2))) void tile_kernel(RowGemmArgs g) {
  constexpr int T = 64 * WM * WN, RI = TM / WM / 16, CJ = TN / WN / 16;
  static_assert(RI % 2 == 0, "");
  constexpr int AT_B = TM * QB, STAGE = (TM + TN) * QB;
  __shared__ __attribute__((aligned(16))) uint8_t lds[NS * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4, wm = wave / WN, wn = wave % WN;

  // tile of this workgroup: workgroups go to the 8 XCDs in turn; each XCD takes
  // a contiguous part of the tiles, which run down 8 row tiles at a time
  int mt, nt, n0;
  bool zero = false;
  {
    std::conditional_t<GROUPED, Pieces<TN>, Whole<TN>> pieces(g);
    const int tm = (g.m + TM - 1) / TM, tn = pieces.total, all = tm * tn;
    const int id = blockIdx.x, x = id & 7, part = all >> 3, more = all & 7;
    if (GROUPED && (id >> 3) >= part + (x < more)) return;
    const int t = x * part + min(x, more) + (id >> 3);
    const int width = 8 * tn, band = t / width, h = min(8, tm - 8 * band), in = t - band * width;
    mt = 8 * band + in % h;
    nt = in / h;
    n0 = nt * TN;
    if constexpr (GROUPED) {
      const Rows rows = pieces.find(nt);
      if (rows.group < 0 || mt < 0 || mt >= tm) return;      // the latter as in find
      n0 = rows.first;
      zero = rows.group == g.groups;
      take_group(g, zero ? Rows{rows.first, rows.end, 0} : rows);
    }
  }
  const int m0 = mt * TM;
  Panel<TM, T, true> pa;
  Panel<TN, T, false> pb;
  pa.init(g.a, m0, g.k, tid);
  pb.init(g.b, n0, g.k, tid);
  // The stage of block kb, in LOADS pieces.
  constexpr int NA = Panel<TM, T, true>::N, LOADS = NA + Panel<TN, T, false>::N;
  auto load = [&](int piece, int kb, uint32_t to) {
    if (piece < NA) pa.load(piece, kb, to, wave);
    else pb.load(piece - NA, kb, to + AT_B, wave);
  };
  auto load_all = [&](int kb, uint32_t to) {
#pragma unroll
    for (int c = 0; c < LOADS; ++c) load(c, kb, to);
  };

  i4 acc[RI][CJ];
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int j = 0; j < CJ; ++j) acc[i][j] = i4{0, 0, 0, 0};

  // Fragment addresses.  Row tile i = 2h + p: lane r holds block row
  // 32 h + 8 (r / 4) + 4 p + r % 4, so that the two tiles of a pair leave 8
  // consecutive rows of C in one lane.
  const int ar = wm * (TM / WM) + 8 * (r >> 2) + (r & 3), br = wn * (TN / WN) + r;
  const int aat = ar * QB + 16 * (q ^ a_key(ar)), bat = AT_B + br * QB + 16 * (q ^ b_key(br));
  i4 x[2][2], b[CJ][2];       // of row tile i (mod 2) and of the stage's columns
  auto read_a = [&](const uint8_t *l, int i) {
    const int o = (i >> 1) * 32 * QB + (i & 1) * 4 * QB;
    x[i & 1][0] = *reinterpret_cast<const i4 *>(l + aat + o);
    x[i & 1][1] = *reinterpret_cast<const i4 *>(l + (aat ^ 64) + o);
  };
  auto read_b = [&](const uint8_t *l) {
#pragma unroll
    for (int j = 0; j < CJ; ++j) {
      b[j][0] = *reinterpret_cast<const i4 *>(l + bat + 16 * QB * j);
      b[j][1] = *reinterpret_cast<const i4 *>(l + (bat ^ 64) + 16 * QB * j);
    }
  };
  // All waves, once this one has at most LEFT loads under way and no LDS access.
  auto meet = [&](auto left) {
    constexpr int LEFT = decltype(left)::value;
    static_assert(LEFT < 64, "");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((LEFT & 15) | (LEFT >> 4) << 14 | 7 << 4);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  constexpr std::integral_constant<int, 0> ALL{};

  // This workgroup's blocks: all, or the part of grid y.  Stage 0 is its last one, which
  // may be cut at column k; stage i > 0 is block kb0 + i - 1.
  const int blocks = zero ? 0 : (g.k + QB - 1) / QB;
  const int kb0 = (int)((int64_t)blocks * blockIdx.y / gridDim.y);
  const int nb = (int)((int64_t)blocks * (blockIdx.y + 1) / gridDim.y) - kb0;
  if (nb > 0) {
    const uint32_t base = lds_address(lds);
    pa.load_last(kb0 + nb - 1, base, wave, true);
    pb.load_last(kb0 + nb - 1, base + AT_B, wave, true);
    if (nb >= NS) {
#pragma unroll
      for (int s = 1; s < NS; ++s) load_all(kb0 + s - 1, base + s * STAGE);
      meet(std::integral_constant<int, (NS - 1) * LOADS>{});
    } else {
      for (int s = 1; s < nb; ++s) load_all(kb0 + s - 1, base + s * STAGE);
      meet(ALL);
    }
    if ((g.k & (QB - 1)) != 0 && kb0 + nb == blocks) {      // zeros in one operand are enough: integers have no NaN
      pb.cut(g.k & (QB - 1), lds + AT_B, tid);
      meet_lds();
    }
    read_b(lds);
    read_a(lds, 0);
    auto row_tiles = [&](const uint8_t *l) {      // all products of a stage
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        if (i + 1 < RI) read_a(l, i + 1);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < CJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[i & 1][h], b[j][h], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    int now = 0, next = STAGE;
    for (int stage = 0; stage < nb - 1; ++stage) {
      row_tiles(lds + now);
      // stages under way: up to stage + NS - 1, of which the next one is needed
      if (NS > 2 && stage + NS <= nb) meet(std::integral_constant<int, (NS - 2) * LOADS>{});
      else meet(ALL);
      if (stage + NS < nb) load_all(kb0 + stage + NS - 1, base + now);
      read_b(lds + next);
      read_a(lds + next, 0);
      now = next;
      next = next == (NS - 1) * STAGE ? 0 : next + STAGE;
    }
    row_tiles(lds + now);
  }

  // lane (r, q): rows 32 h + 8 q .. + 7 of its columns
  const int row0 = m0 + wm * (TM / WM), col0 = n0 + wn * (TN / WN);
  if (!GROUPED && gridDim.y > 1) {        // a part's sums
    int *part = static_cast<int *>(g.c) + (int64_t)blockIdx.y * g.m * g.n;
#pragma unroll
    for (int h = 0; h < RI / 2; ++h)
#pragma unroll
      for (int j = 0; j < CJ; ++j) {
        const int row = row0 + 32 * h + 8 * q, col = col0 + 16 * j + r;
        if (row < g.m && col < g.n) {
          int v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = acc[2 * h + (e >> 2)][j][e & 3];
          put_sums(part + (int64_t)col * g.m + row, g.m - row, v);
        }
      }
    return;
  }
  // C goes through LDS, a column's TM entries in a row, 16-byte pieces XOR-placed, so
  // that whole stretches of its columns are stored, past the caches: 2501 x 1111 x 1747
  // in 128 x 128 on four waves 12.8 us, through the caches 13.2, straight from the
  // registers, 64 bytes of a column at a time, 15.7.
  auto store = [&](auto element) {
    typedef decltype(element) E;
    constexpr int WIDE = sizeof(E) / 2, PIECES = WIDE * TM / 8;       // pieces of 8 entries; of a column
    constexpr int PASSES = (int)sizeof(E) * TM * TN > NS * STAGE ? 2 : 1, JS = CJ / PASSES, COLS = T / PIECES;
    static_assert((int)sizeof(E) * TM * TN <= PASSES * NS * STAGE && CJ % PASSES == 0, "");
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
      __syncthreads();
#pragma unroll
      for (int h = 0; h < RI / 2; ++h) {
        const int row = wm * (TM / WM) + 32 * h + 8 * q;
        float sa[8];
        get8(g.a.scales + m0 + row, g.m - m0 - row, sa);
#pragma unroll
        for (int jj = 0; jj < JS; ++jj) {
          const int at = 16 * (wn * JS + jj) + r, j = pass * JS + jj;      // column in LDS
          const float sb = g.b.scales[min(col0 + 16 * j + r, g.n - 1)];
          E v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = (E)(zero ? 0.0f : (float)acc[2 * h + (e >> 2)][j][e & 3] * sb * sa[e]);
          u4 w[WIDE];
          __builtin_memcpy(w, v, sizeof v);
#pragma unroll
          for (int p = 0; p < WIDE; ++p) *reinterpret_cast<u4 *>(lds + at * 16 * PIECES + 16 * ((WIDE * (row >> 3) + p) ^ (at & 15))) = w[p];
        }
      }
      __syncthreads();
      constexpr int N = 8 / WIDE;                   // entries of a piece
      const int piece = tid % PIECES, row = m0 + N * piece;
#pragma unroll 4
      for (int at = tid / PIECES; at < TN / PASSES; at += COLS) {
        const int col = n0 + at / (16 * JS) * (TN / WN) + 16 * JS * pass + at % (16 * JS);
        if (col < g.n && row < g.m) {
          const u4 w = *reinterpret_cast<const u4 *>(lds + at * 16 * PIECES + 16 * (piece ^ (at & 15)));
          E *to = static_cast<E *>(g.c) + (int64_t)col * g.ldc + row;
          if (row + N <= g.m) {
            put16<true>(to, w);
          } else {
            E v[N];
            __builtin_memcpy(v, &w, 16);
#pragma unroll
            for (int e = 0; e < N - 1; ++e)
              if (row + e < g.m) to[e] = v[e];
          }
        }
      }
    }
  };
  if (g.dt == TLR_F32) store(float{});
  else if (g.dt == TLR_F16) store((_Float16)0.0f);
  else store((__bf16)0.0f);
}

// Large products: one workgroup a CU goes through C tiles of TM x TN, its share of those
// of its XCD.  As in tile_kernel, a ring of two stages in LDS and one barrier a stage; but
// the stages of all its tiles are one sequence.  A tile's first stage and its scales are
// loaded under the last stage of the tile before, its second one before that is stored
// (64 groups, 28672 rows, 2048 x 1408 in 256 x 256 tiles 106 us, stored through a buffer of
// the ring 117, which a workgroup for each tile takes 13% longer than; 8192 x 16384 x 1024
// 138, 150).  SPREAD loads of the next stage follow each row tile's matrix instructions,
// which so long a stage likes better than all of them at its start.  Groups' pieces are
// counted once, into LDS.  PAST: stores go past the caches, which wants columns of C that
// begin with a cache line (8 groups, 16384 rows, 4096 x 4096 241 us, through the caches 273);
// the pieces of others meet in the caches (6001 x 9000 x 500 47 us, past them 100).
template <bool GROUPED, bool PAST, int TM, int TN, int WM, int WN, int SPREAD>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2))) void stream_kernel(RowGemmArgs g) {
  constexpr int T = 64 * WM * WN, RI = TM / WM / 16, CJ = TN / WN / 16, NA = TM * 8 / T, NB = TN * 8 / T;
  static_assert(RI % 2 == 0 && SPREAD * RI >= NA + NB, "");
  constexpr int AT_B = TM * QB, STAGE = (TM + TN) * QB;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * STAGE];
  __shared__ __attribute__((aligned(16))) float scales[2][TM + TN];       // of this tile's rows and columns, and the next one's
  __shared__ __attribute__((aligned(16))) uint8_t slices[WM * WN][2048];  // results on their way
  __shared__ int upto[GROUPED ? MOST_GROUPS : 1], begin[GROUPED ? MOST_GROUPS + 1 : 1];      // pieces up to and with a group; its rows
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4, wm = wave / WN, wn = wave % WN;

  int tn = (g.n + TN - 1) / TN;
  if constexpr (GROUPED) {
    if (wave == 0) {
      int before = 0;
      for (int e0 = 0; e0 < g.groups; e0 += 64) {
        const int e = e0 + lane;
        const int lo = e < g.groups ? min(max(g.offsets[e], 0), g.n) : 0;
        const int hi = e < g.groups ? max(lo, min(max(g.offsets[e + 1], 0), g.n)) : 0;
        const int sum = before + scan64((hi - lo + TN - 1) / TN, lane);
        if (e < g.groups) {
          upto[e] = sum;
          begin[e] = lo;
        }
        before = __builtin_amdgcn_readlane(sum, 63);
      }
      if (lane == 0) begin[g.groups] = min(max(g.offsets[g.groups], 0), g.n);
    }
    __syncthreads();
    tn = __builtin_amdgcn_readfirstlane(upto[g.groups - 1]);
  }
  // Workgroups go to the 8 XCDs in turn; each XCD has a contiguous part of the tiles,
  // which run down 8 row tiles at a time, and its workgroups take them in turn.
  const int tm = (g.m + TM - 1) / TM, all = tm * tn, blocks = (g.k + QB - 1) / QB;
  const int xcd = blockIdx.x & 7, peers = ((int)gridDim.x - xcd + 7) >> 3;
  int t = xcd * (all >> 3) + min(xcd, all & 7);
  const int end = t + (all >> 3) + (xcd < (all & 7) ? 1 : 0);
  t += blockIdx.x >> 3;

  struct Tile {
    int m0, n0, n, group;     // n: end of the group's rows; m0 < 0: none
  };
  auto locate = [&](int at) {
    Tile x{-1, 0, 0, 0};
    if (at >= end) return x;
    const int width = 8 * tn, band = at / width, h = min(8, tm - 8 * band), in = at - band * width, nt = in / h;
    const int m0 = (8 * band + in % h) * TM;
    if constexpr (!GROUPED) return Tile{m0, nt * TN, g.n, 0};
    for (int e0 = 0; e0 < g.groups; e0 += 64) {
      const uint64_t past = __ballot(nt < upto[min(e0 + lane, g.groups - 1)]);
      if (past) {
        const int e = e0 + __builtin_ctzll(past), lo = __builtin_amdgcn_readfirstlane(begin[e]);
        const int first = lo + (nt - (e > 0 ? __builtin_amdgcn_readfirstlane(upto[e - 1]) : 0)) * TN;
        const int last = max(lo, __builtin_amdgcn_readfirstlane(begin[e + 1]));
        // always so, unless groups that overlap have more pieces than an int counts
        if (first >= lo && first < last && m0 >= 0 && m0 < g.m) x = Tile{m0, first, last, e};
        break;
      }
    }
    return x;
  };
  // Where the loads of the next stage read: A's and B's first row and block, and bytes
  // from there to the end of the last readable chunk (0: zeros).
  const uint8_t *a_from = nullptr, *b_from = nullptr;
  int32_t a_bytes = 0, b_bytes = 0;
  auto aim = [&](const Tile &x, int kb) {
    const int readable = ((g.k + 15) & ~15) - kb * QB;
    a_from = g.a.codes + x.group * g.code_step + (int64_t)x.m0 * g.a.ld + kb * QB;
    b_from = g.b.codes + (int64_t)x.n0 * g.b.ld + kb * QB;
    a_bytes = x.m0 < 0 ? 0 : (min(TM, g.m - x.m0) - 1) * (int32_t)g.a.ld + readable;
    b_bytes = x.m0 < 0 ? 0 : (min(TN, x.n - x.n0) - 1) * (int32_t)g.b.ld + readable;
  };
  const uint32_t base = lds_address(lds);
  const int32_t a_step = (T / 8) * (int32_t)g.a.ld, b_step = (T / 8) * (int32_t)g.b.ld;
  const uint32_t a_at = (uint32_t)(tid >> 3) * (uint32_t)g.a.ld + Panel<TM, T, true>::chunk(tid);
  const uint32_t b_at = (uint32_t)(tid >> 3) * (uint32_t)g.b.ld + Panel<TN, T, false>::chunk(tid);
  auto load = [&](int p, uint32_t to) {
    if (p < NA) to_lds16(buffer(a_from + p * a_step, max(a_bytes - p * a_step, 0)), a_at, 0, to + (p * T + wave * 64) * 16);
    else to_lds16(buffer(b_from + (p - NA) * b_step, max(b_bytes - (p - NA) * b_step, 0)), b_at, 0, to + AT_B + ((p - NA) * T + wave * 64) * 16);
  };
  const int ar = wm * (TM / WM) + 8 * (r >> 2) + (r & 3), br = wn * (TN / WN) + r;
  const int aat = ar * QB + 16 * (q ^ a_key(ar)), bat = AT_B + br * QB + 16 * (q ^ b_key(br));
  i4 x[2][2], b[CJ][2];       // fragments of row tile i (mod 2) and of the stage's columns
  auto read_a = [&](const uint8_t *l, int i) {
    const int o = (i >> 1) * 32 * QB + (i & 1) * 4 * QB;
    x[i & 1][0] = *reinterpret_cast<const i4 *>(l + aat + o);
    x[i & 1][1] = *reinterpret_cast<const i4 *>(l + (aat ^ 64) + o);
  };
  auto read_b = [&](const uint8_t *l) {
#pragma unroll
    for (int j = 0; j < CJ; ++j) {
      b[j][0] = *reinterpret_cast<const i4 *>(l + bat + 16 * QB * j);
      b[j][1] = *reinterpret_cast<const i4 *>(l + (bat ^ 64) + 16 * QB * j);
    }
  };
  auto meet = [&]() {         // nothing is under way
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  auto load_scales = [&](const Tile &x, int to) {
    const bool of_a = wave < TM / 64;
    const int first = of_a ? 0 : TM, have = x.m0 < 0 ? 0 : of_a ? min(TM, g.m - x.m0) : min(TN, x.n - x.n0);
    const float *from = of_a ? g.a.scales + x.group * g.scale_step + x.m0 : g.b.scales + x.n0;
    if (wave < (TM + TN) / 64) to_lds4(buffer(reinterpret_cast<const uint8_t *>(from), 4 * have), (tid - first) * 4, lds_address(reinterpret_cast<uint8_t *>(scales[to] + wave * 64)));
  };

  // A tile's first stage is its last block, the one cut at column k; stage i > 0 is block
  // i - 1.  The second one is loaded before the stores of the tile before, so that the
  // wait for it, in order, leaves them under way.
  constexpr int LOADS = NA + NB;
  auto load_all = [&](uint32_t to) {
#pragma unroll
    for (int p = 0; p < LOADS; ++p) load(p, to);
  };
  Tile now = locate(t);
  int at = 0, turn = 0;       // LDS stage that is computed; scales of this tile
  int stores = 0;             // of the tile before, behind the second stage's loads; 0: not known
  load_scales(now, 0);
  if (blocks > 0) {
    aim(now, blocks - 1);
    load_all(base);
  }
  meet();
  if (blocks > 1) {
    aim(now, 0);
    load_all(base + STAGE);
  }
  for (; t < end; t += peers, turn ^= 1) {
    const Tile next = locate(t + peers);
    i4 acc[RI][CJ];
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
      for (int j = 0; j < CJ; ++j) acc[i][j] = i4{0, 0, 0, 0};
    if (blocks > 0 && (g.k & (QB - 1)) != 0) {      // zeros in one operand are enough: integers have no NaN
      Panel<TN, T, false>::cut(g.k & (QB - 1), lds + at + AT_B, tid);
      meet_lds();
    }
    // All products of a stage, with the loads of the next one.
    auto products = [&](auto live) {
      const uint8_t *l = lds + at;
      read_b(l);
      read_a(l, 0);
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        if (i + 1 < RI) read_a(l, i + 1);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < CJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[i & 1][h], b[j][h], acc[i][j], 0, 0, 0);
        if constexpr (decltype(live)::value)
#pragma unroll
          for (int c = 0; c < SPREAD; ++c)
            if (i * SPREAD + c < LOADS) load(i * SPREAD + c, base + (STAGE - at));
        __builtin_amdgcn_sched_barrier(0);
      }
      at = STAGE - at;
    };
    if (blocks > 1) {
      products(std::false_type{});
      asm volatile("" ::: "memory");
      if (stores == 16) __builtin_amdgcn_s_waitcnt(0 | 1 << 14 | 7 << 4);
      else if (stores == 32) __builtin_amdgcn_s_waitcnt(0 | 2 << 14 | 7 << 4);
      else __builtin_amdgcn_s_waitcnt(0);
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      for (int stage = 1; stage < blocks; ++stage) {
        if (stage + 1 < blocks) {
          a_from += QB;
          b_from += QB;
          a_bytes -= QB;
          b_bytes -= QB;
        } else {
          load_scales(next, turn ^ 1);
          aim(next, blocks - 1);
        }
        products(std::true_type{});
        if (stage + 1 < blocks) meet();
      }
      meet_lds();
      aim(next, 0);
      load_all(base + (STAGE - at));
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(LOADS | 7 << 4 | 0xf << 8);      // those before them
      asm volatile("" ::: "memory");
    } else {
      load_scales(next, turn ^ 1);
      if (blocks > 0) {
        aim(next, blocks - 1);
        products(std::true_type{});
      }
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0);
      asm volatile("" ::: "memory");
    }
    stores = 0;
    if (now.m0 >= 0) {        // always so, but for the groups that locate leaves out
      auto store = [&](auto element) {
        typedef WaveStore<decltype(element), RI, CJ, PAST> Store;
        const int row = wm * (TM / WM), col = wn * (TN / WN);
        Store::run(g, acc, slices[wave], scales[turn] + row, scales[turn] + TM + col, now.m0 + row, now.n0 + col, now.n, lane);
        static_assert(Store::STORES == 16 || Store::STORES == 32, "");
        if (now.m0 + TM <= g.m && now.n0 + TN <= now.n) stores = Store::STORES;
      };
      if (g.dt == TLR_F32) store(float{});
      else if (g.dt == TLR_F16) store((_Float16)0.0f);
      else store((__bf16)0.0f);
    }
    meet_lds();
    now = next;
  }
  __builtin_amdgcn_s_waitcnt(0);        // no load is left that writes LDS
  if constexpr (GROUPED) {
    if (!g.clear) return;
    const float zeros[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const int up = (g.m + 7) / 8;
    const int front = begin[0], behind = begin[g.groups], all = front + g.n - behind;
    for (int x = blockIdx.x; x < all; x += gridDim.x)
      for (int i = tid; i < up; i += T) store8(g, 8 * i, x < front ? x : behind + x - front, zeros);
  }
}

// C from PARTS m x n matrices of sums: a thread takes 8 consecutive rows of a column.
template <int PARTS> __global__ __launch_bounds__(256) void parts_kernel(RowGemmArgs g, const int *part) {
  const int up = (g.m + 7) / 8;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int j = (int)(at / up), i = 8 * (int)(at - (int64_t)j * up), left = g.m - i;
  if (j >= g.n) return;
  const int *p = part + (int64_t)j * g.m + i;
  const int64_t step = (int64_t)g.m * g.n;
  int x[PARTS][8];
#pragma unroll
  for (int z = 0; z < PARTS; ++z) {
    if (left >= 8) __builtin_memcpy(x[z], p + z * step, 32);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) x[z][e] = e < left ? p[z * step + e] : 0;
  }
  float sa[8], v[8];
  get8(g.a.scales + i, left, sa);
  const float sb = g.b.scales[j];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    int sum = 0;
#pragma unroll
    for (int z = 0; z < PARTS; ++z) sum += x[z][e];
    v[e] = (float)sum * sb * sa[e];
  }
  store8(g, i, j, v);
}

// ---- which kernel ------------------------------------------------------------------------------------

enum Kind { STRIP, STRIP_2, TILE_64, TILE_128, TILE_128W, STREAM };
struct Shape {
  int rows, cols, threads;  // of C and of the workgroup that computes them
};
constexpr Shape SHAPE[] = {{16, 16, 512}, {16, 32, 512}, {128, 64, 512}, {128, 128, 256}, {128, 128, 512}, {256, 256, 512}};
struct Choice {
  Kind kind;
  int parts;                // of the contraction, with a launch that adds them if more than one
};

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Pieces of B's rows at most: each group ends with a piece that may be short, and so
// do the rows before the first and behind the last.
int64_t most_pieces(Kind kind, int64_t n, int32_t groups) {
  const int64_t tn = SHAPE[kind].cols;
  return groups ? std::min(n, (n + (groups + 2) * (tn - 1)) / tn) : cdiv(n, tn);
}

// A launch has less than 2^32 threads along x; a workgroup for each tile, but one a CU
// of those that go through several.  128 x 128 tiles of four waves fit whatever the others
// do, where a result has less than 2^24 of them.
constexpr int64_t CUS = 256, THREAD_LIM = (int64_t)1 << 32, TILE_LIM = (int64_t)1 << 24;
int64_t workgroups(Kind kind, int64_t m, int64_t n, int32_t groups) {
  if (kind <= STRIP_2) return cdiv(m, 16);
  const int64_t tiles = cdiv(m, SHAPE[kind].rows) * most_pieces(kind, n, groups);
  return kind == STREAM ? std::min(tiles, CUS) : tiles;
}
bool fits(Kind kind, int parts, int64_t m, int64_t n, int32_t groups) {
  return workgroups(kind, m, n, groups) * SHAPE[kind].threads < THREAD_LIM && (kind > STRIP_2 || most_pieces(kind, n, groups) <= 65535) &&
         (parts == 1 || cdiv(m, 8) * n < THREAD_LIM - 256);
}

// The kernel with the least estimated time (us).  The estimates are fits to measured
// times (graph replays, 16-bit C) of every kernel at 44 products and 22 of groups; the
// choice costs 0.2% against the best of them, 4% at most.  Some of them, the kernel
// chosen first:
//   4608 x 37 x 2568     strip 8.5, of 32 columns 8.9, 128 x 64 tiles in four parts 9.1
//   8192 x 24 x 2048     strip of 32 columns 7.5, of 16 9.5
//   8192 x 33 x 8192     128 x 64 in four parts 16, strip of 32 columns 35
//   2501 x 1111 x 1747   128 x 128 on eight waves 12.0, on four 12.8, 128 x 64 16
//   2000 x 1000 x 8000   128 x 64 27, 128 x 128 on eight waves 34
//   2048 x 4096 x 2048   128 x 128 on four waves 19, on eight 24
//   4096 x 4096 x 4096   256 x 256 56, 128 x 128 on four waves 64
//   64 groups, 28672 rows, 2816 x 2048   256 x 256 216, 128 x 128 245
//   64 groups, 8192 rows, 2048 x 1408    128 x 128 on four waves 48, 256 x 256 61
//   32 groups, 96 rows, 2048 x 2048      128 x 128 on four waves 22, 128 x 64 24, strip 28
//   64 groups, 40 rows, 1024 x 4096      128 x 64 20, 128 x 128 on four waves 26
Choice least_estimate(int64_t m, int64_t n, int64_t k, int32_t groups) {
  const double nb = (double)std::max<int64_t>(1, cdiv(k, QB));
  // Groups that have rows, where each row falls into one of them; the weights they
  // read, MB; pieces of tn rows of B, half a piece more for each group.
  const double reached = groups ? groups * (1.0 - std::exp(-(double)n / groups)) : 1.0;
  const double weights = groups ? reached * (double)m * (double)k * 1e-6 : 0.0;
  auto pieces = [&](int tn) { return groups ? std::max(reached, (double)n / tn + 0.5 * reached) : (double)cdiv(n, tn); };
  Choice best{TILE_128, 1};
  double least = 1e300;
  // `rate`: what the kernel reads of weights, TB/s
  auto offer = [&](Kind kind, int parts, double rate, double t) {
    if (groups) t = std::max(t, 3.0 + weights / rate);
    if (t < least && fits(kind, parts, m, n, groups)) {
      least = t;
      best = Choice{kind, parts};
    }
  };
  // 2 KB of A a workgroup and block, and as many rows of B as there are up to the strip's
  auto strips = [&](Kind kind, double first, double rows, double row, double next) {
    const int tn = SHAPE[kind].cols;
    offer(kind, 1, 4.2, first + cdiv(m, 16) * pieces(tn) * nb * (rows + row * std::min((double)tn, n / reached)) + next * nb);
  };
  strips(STRIP, 2.4, 1.75e-4, 1.0e-5, 0.058);
  strips(STRIP_2, 2.55, 2.2e-4, 0.9e-5, 0.062);
  // One workgroup a CU takes `one` a block, `pair` of them together `two`.  Four waves a
  // CU keep too few loads under way for weights out of HBM.
  auto tiles = [&](Kind kind, int pair, double rate, double one, double two, double first, double next) {
    for (const int parts : {1, 2, 4, 8}) {
      if (parts > 1 && (nb < 4 * parts || groups)) break;
      const double t = (double)cdiv(m, SHAPE[kind].rows) * pieces(SHAPE[kind].cols) * parts;
      const double rounds = std::ceil(t / (256 * pair)), rest = t - 256 * pair * (rounds - 1);
      double us = first + (rounds - 1) * next + std::ceil(nb / parts) * ((rounds - 1) * two + (rest <= 256 ? one : two));
      if (parts > 1) us += 2.8 + parts * (0.1 + (double)m * (double)n * 2.1e-6);
      offer(kind, parts, kind == TILE_128 && t < 384 ? 4.4 : rate, us);
      if (kind == STREAM || (kind == TILE_128 && parts == 2)) break;
    }
  };
  tiles(TILE_64, 2, 5.0, 0.312, 0.865, 3.6, 4.4);
  tiles(TILE_128W, 1, 4.8, 0.505, 0.65, 3.85, 4.0);
  tiles(TILE_128, 2, 5.6, 0.62, 0.94, 3.8, 8.0);
  tiles(STREAM, 1, 4.6, 1.455, 1.455, 7.3, 11.6);
  return best;
}

// A call asks for its workspace and then for its launch: the last answer is kept.
Choice choose(int64_t m, int64_t n, int64_t k, int32_t groups) {
  thread_local int64_t of[4] = {-1, -1, -1, -1};
  thread_local Choice last;
  if (of[0] != m || of[1] != n || of[2] != k || of[3] != groups) {
    last = least_estimate(m, n, k, groups);
    of[0] = m;
    of[1] = n;
    of[2] = k;
    of[3] = groups;
  }
  return last;
}

size_t parts_bytes(const Choice &c, int64_t m, int64_t n) { return c.parts > 1 ? sizeof(int) * (size_t)c.parts * m * n : 0; }

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t SIZE_LIM = 0x7fffffff, PRODUCT_LIM = SIZE_LIM - 511, LD_LIM = (int64_t)1 << 22, K_LIM = 131071;

tlr_status launched(const char *what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TLR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
  return TLR_OK;
}

tlr_status check_sizes(int64_t m, int64_t n, int64_t k, int32_t groups) {
  if (m < 0 || n < 0 || k < 0 || m > PRODUCT_LIM || n > PRODUCT_LIM) return fail(TLR_ERR_INVALID_ARG, "row_gemm: size out of range");
  if (k > K_LIM) return fail(TLR_ERR_UNSUPPORTED, "row_gemm: 32-bit sums hold 131071 columns at most");
  if (groups < 0 || groups > MOST_GROUPS) return fail(TLR_ERR_INVALID_ARG, "row_gemm: groups are 1 .. 1024");
  if (cdiv(m, 128) * most_pieces(TILE_128, n, groups) >= TILE_LIM) return fail(TLR_ERR_INVALID_ARG, "row_gemm: too many tiles for a launch");
  return TLR_OK;
}

tlr_status check_operand(const char *name, const tlr_row_matrix *x, int64_t rows, int64_t k, Operand *o) {
  const std::string w = name;
  if (!x || (!x->codes && k > 0) || !x->scales) return fail(TLR_ERR_INVALID_ARG, w + ": null matrix, codes or scales");
  if (x->ld % 16 != 0 || !aligned(x->codes, 16)) return fail(TLR_ERR_INVALID_ARG, w + ": codes and their rows must be 16-byte aligned");
  if (x->ld < k || x->ld >= LD_LIM) return fail(TLR_ERR_INVALID_ARG, w + ": leading dimension out of range");
  if (!aligned(x->scales, 4)) return fail(TLR_ERR_INVALID_ARG, w + ": misaligned scales");
  *o = Operand{static_cast<const uint8_t *>(x->codes), x->scales, x->ld, (int32_t)rows};
  return TLR_OK;
}

// What products of x or of its codes check alike, and set.
tlr_status product_args(const char *name, tlr_dtype dt, int64_t m, int64_t n, int64_t k, const tlr_row_matrix *A, void *C, int64_t ldc,
                        RowGemmArgs *g) {
  const std::string w = std::string(name) + ": ";
  if (dt == TLR_F64) return fail(TLR_ERR_UNSUPPORTED, w + "TLR_F64 is not provided");
  if (dt != TLR_F32 && dt != TLR_F16 && dt != TLR_BF16) return fail(TLR_ERR_INVALID_ARG, w + "bad dtype");
  if (ldc < std::max<int64_t>(1, m) || ldc > SIZE_LIM) return fail(TLR_ERR_INVALID_ARG, w + "ldc out of range");
  if (m == 0 || n == 0) return TLR_OK;
  const tlr_status st = check_operand((w + "A").c_str(), A, m, k, &g->a);
  if (st != TLR_OK) return st;
  if (!C || !aligned(C, dt == TLR_F32 ? 4 : 2)) return fail(TLR_ERR_INVALID_ARG, w + "null or misaligned C");
  g->m = (int32_t)m;
  g->n = (int32_t)n;
  g->k = (int32_t)k;
  g->c = C;
  g->ldc = ldc;
  g->dt = dt;
  return TLR_OK;
}

// A linear layer's call: where the codes of x (rows of ld bytes), its scales and a
// product's parts stand in the workspace.  A few tokens take one launch and no
// workspace.
struct LinearParts {
  Choice choice;
  bool few;
  int64_t ld;
  size_t scales, parts, bytes;
};
// Whether a linear layer's tokens are quantized in the product's launch: what they have to
// fit into, and the work that its rounds of workgroups (512 at a time) repeat, 0.4 us for
// each vector of x a lane and as much for the rest (8192 x 8 x 4096, eight vectors: 13.2
// us, 11.3 with a launch of its own; 32768 x 1 x 4096, four rounds of one: 25.6 and 24.1).
bool few_tokens(int64_t m, int64_t n, int64_t k) {
  const int64_t vectors = cdiv(k, 512 * few_waves(n));
  return n <= FEW_TOKENS && vectors <= 4 && cdiv(m, 16 * 512) * (1 + vectors) <= 6;
}

LinearParts linear_parts(int64_t m, int64_t n, int64_t k) {
  LinearParts p{};
  if (m == 0 || n == 0) return p;
  p.choice = choose(m, n, k, 0);
  p.few = few_tokens(m, n, k);
  if (p.few) return p;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  p.ld = (k + 15) & ~(int64_t)15;
  p.scales = up((size_t)n * p.ld);
  p.parts = p.scales + up(sizeof(float) * (size_t)n);
  p.bytes = p.parts + parts_bytes(p.choice, m, n);
  return p;
}

template <Kind KIND, int WM, int WN, int NS> void tile_launch(const RowGemmArgs &g, int parts, int *ws, hipStream_t st) {
  constexpr int TM = SHAPE[KIND].rows, TN = SHAPE[KIND].cols, T = 64 * WM * WN;
  static_assert(SHAPE[KIND].threads == T, "");
  const dim3 grid((unsigned)workgroups(KIND, g.m, g.n, g.groups), (unsigned)parts);
  if (g.groups) return tile_kernel<true, TM, TN, WM, WN, NS><<<grid, T, 0, st>>>(g);
  if (parts == 1) return tile_kernel<false, TM, TN, WM, WN, NS><<<grid, T, 0, st>>>(g);
  RowGemmArgs h = g;
  h.c = ws;
  tile_kernel<false, TM, TN, WM, WN, NS><<<grid, T, 0, st>>>(h);
  const unsigned sum = (unsigned)cdiv(cdiv(g.m, 8) * g.n, 256);
  if (parts == 2) parts_kernel<2><<<sum, 256, 0, st>>>(g, ws);
  else if (parts == 4) parts_kernel<4><<<sum, 256, 0, st>>>(g, ws);
  else parts_kernel<8><<<sum, 256, 0, st>>>(g, ws);
}

template <Kind KIND, int WM, int WN, int SPREAD> void stream_launch(const RowGemmArgs &g, hipStream_t st) {
  constexpr int TM = SHAPE[KIND].rows, TN = SHAPE[KIND].cols, T = 64 * WM * WN;
  static_assert(SHAPE[KIND].threads == T, "");
  const unsigned grid = (unsigned)workgroups(KIND, g.m, g.n, g.groups);
  const bool past = ((reinterpret_cast<uintptr_t>(g.c) | (uintptr_t)(g.ldc * (g.dt == TLR_F32 ? 4 : 2))) & 127) == 0;
  if (g.groups && past) stream_kernel<true, true, TM, TN, WM, WN, SPREAD><<<grid, T, 0, st>>>(g);
  else if (g.groups) stream_kernel<true, false, TM, TN, WM, WN, SPREAD><<<grid, T, 0, st>>>(g);
  else if (past) stream_kernel<false, true, TM, TN, WM, WN, SPREAD><<<grid, T, 0, st>>>(g);
  else stream_kernel<false, false, TM, TN, WM, WN, SPREAD><<<grid, T, 0, st>>>(g);
}

template <Kind KIND> void strip_launch(const RowGemmArgs &g, hipStream_t st) {
  constexpr int NJ = SHAPE[KIND].cols / 16;
  const dim3 grid((unsigned)workgroups(KIND, g.m, g.n, g.groups), (unsigned)most_pieces(KIND, g.n, g.groups));
  if (g.groups) strip_kernel<true, NJ><<<grid, 512, 0, st>>>(g);
  else strip_kernel<false, NJ><<<grid, 512, 0, st>>>(g);
}

void gemm_launch(const RowGemmArgs &g, const Choice &c, int *ws, hipStream_t st) {
  switch (c.kind) {
    case STRIP: return strip_launch<STRIP>(g, st);
    case STRIP_2: return strip_launch<STRIP_2>(g, st);
    case TILE_64: return tile_launch<TILE_64, 4, 2, 3>(g, c.parts, ws, st);
    case TILE_128: return tile_launch<TILE_128, 2, 2, 2>(g, c.parts, ws, st);
    case TILE_128W: return tile_launch<TILE_128W, 2, 4, 3>(g, c.parts, ws, st);
    default: return stream_launch<STREAM, 2, 4, 2>(g, st);
  }
}

}  // namespace

tlr_status row_quantize(tlr_dtype dt, int64_t rows, int64_t k, const void *X, int64_t x_rows, int64_t ldx, const int32_t *index,
                        void *codes, int64_t ldq, float *scales, void *stream) {
  if (dt == TLR_F64) return fail(TLR_ERR_UNSUPPORTED, "row_quantize: TLR_F64 is not provided");
  if (dt != TLR_F32 && dt != TLR_F16 && dt != TLR_BF16) return fail(TLR_ERR_INVALID_ARG, "row_quantize: bad dtype");
  if (rows < 0 || k < 0 || x_rows < 0 || rows > SIZE_LIM || x_rows > SIZE_LIM || k > 1 << 30)
    return fail(TLR_ERR_INVALID_ARG, "row_quantize: size out of range");
  if (!index && rows != x_rows && rows > 0) return fail(TLR_ERR_INVALID_ARG, "row_quantize: without an index the result has the rows of X");
  if (ldx < std::max<int64_t>(1, k)) return fail(TLR_ERR_INVALID_ARG, "row_quantize: leading dimension of X too small");
  if (ldq % 16 != 0 || ldq < k || !aligned(codes, 16)) return fail(TLR_ERR_INVALID_ARG, "row_quantize: codes and their rows must be 16-byte aligned");
  if (rows == 0) return TLR_OK;
  if (!scales || !aligned(scales, 4) || !aligned(index, 4)) return fail(TLR_ERR_INVALID_ARG, "row_quantize: null or misaligned scales, or misaligned index");
  if (k > 0 && !codes) return fail(TLR_ERR_INVALID_ARG, "row_quantize: null codes");
  if (k > 0 && x_rows > 0 && (!X || !aligned(X, dt == TLR_F32 ? 4 : 2))) return fail(TLR_ERR_INVALID_ARG, "row_quantize: null or misaligned X");
  const RowQuantArgs a{X, rows, x_rows, ldx, ldq, index, static_cast<uint8_t *>(codes), scales, (int32_t)k};
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (dt == TLR_F32) row_quantize_launch<float>(a, st);
  else if (dt == TLR_F16) row_quantize_launch<_Float16>(a, st);
  else row_quantize_launch<__bf16>(a, st);
  return launched("row_quantize");
}

tlr_status row_gemm_plan(int64_t m, int64_t n, int64_t k, int32_t groups, tlr_block_gemm_choice *out) {
  if (!out) return fail(TLR_ERR_INVALID_ARG, "row_gemm_plan: null output");
  const tlr_status st = check_sizes(m, n, k, groups);
  if (st != TLR_OK) return st;
  *out = tlr_block_gemm_choice{};
  if (m == 0 || n == 0) return TLR_OK;
  const Choice c = choose(m, n, k, groups);
  const Shape &s = SHAPE[c.kind];
  const int64_t y = c.kind <= STRIP_2 ? most_pieces(c.kind, n, groups) : 1;
  *out = tlr_block_gemm_choice{s.rows, s.cols, s.threads, 1, c.parts, 0, workgroups(c.kind, m, n, groups), y, parts_bytes(c, m, n)};
  return TLR_OK;
}

tlr_status row_gemm(tlr_dtype dt, int64_t m, int64_t n, int64_t k, const tlr_row_matrix *A, const tlr_row_matrix *B,
                    const tlr_row_groups *groups, void *C, int64_t ldc, void *ws, size_t ws_bytes, void *stream) {
  RowGemmArgs g{};
  tlr_status st = check_sizes(m, n, k, groups ? std::max(groups->count, 1) : 0);
  if (st != TLR_OK) return st;
  if (groups) {
    if (groups->count < 1) return fail(TLR_ERR_INVALID_ARG, "row_gemm: groups are 1 .. 1024");
    if (!groups->offsets || !aligned(groups->offsets, 4)) return fail(TLR_ERR_INVALID_ARG, "row_gemm: null or misaligned offsets");
    if (groups->code_step % 16 != 0 || groups->code_step < 0 || groups->scale_step < 0 || (groups->clear & ~1))
      return fail(TLR_ERR_INVALID_ARG, "row_gemm: steps of whole 16-byte pieces, forwards, and clear 0 or 1 are needed");
    g.offsets = groups->offsets;
    g.code_step = groups->code_step;
    g.scale_step = groups->scale_step;
    g.groups = groups->count;
    g.clear = groups->clear;
  }
  if ((st = product_args("row_gemm", dt, m, n, k, A, C, ldc, &g)) != TLR_OK || m == 0 || n == 0) return st;
  if ((st = check_operand("row_gemm: B", B, n, k, &g.b)) != TLR_OK) return st;
  const Choice choice = choose(m, n, k, g.groups);
  const size_t need = parts_bytes(choice, m, n);
  if (need > 0 && (!ws || !aligned(ws, 16))) return fail(TLR_ERR_INVALID_ARG, "row_gemm: null or misaligned workspace");
  if (ws_bytes < need) return fail(TLR_ERR_WORKSPACE, "row_gemm: workspace too small");
  gemm_launch(g, choice, static_cast<int *>(ws), static_cast<hipStream_t>(stream));
  return launched("row_gemm");
}

tlr_status row_linear_workspace(int64_t m, int64_t n, int64_t k, size_t *bytes) {
  if (!bytes) return fail(TLR_ERR_INVALID_ARG, "row_linear_workspace_bytes: null output");
  const tlr_status st = check_sizes(m, n, k, 0);
  if (st == TLR_OK) *bytes = linear_parts(m, n, k).bytes;
  return st;
}

tlr_status row_linear(tlr_dtype dt, int64_t m, int64_t n, int64_t k, const tlr_row_matrix *A, const void *X, int64_t ldx, void *C,
                      int64_t ldc, void *ws, size_t ws_bytes, void *stream) {
  RowGemmArgs g{};
  tlr_status st = check_sizes(m, n, k, 0);
  if (st != TLR_OK) return st;
  if ((st = product_args("row_linear", dt, m, n, k, A, C, ldc, &g)) != TLR_OK) return st;
  if (ldx < std::max<int64_t>(1, k)) return fail(TLR_ERR_INVALID_ARG, "row_linear: leading dimension of X too small");
  if (m == 0 || n == 0) return TLR_OK;
  if (k > 0 && (!X || !aligned(X, dt == TLR_F32 ? 4 : 2))) return fail(TLR_ERR_INVALID_ARG, "row_linear: null or misaligned X");
  const LinearParts p = linear_parts(m, n, k);
  if (p.bytes > 0 && (!ws || !aligned(ws, 256))) return fail(TLR_ERR_INVALID_ARG, "row_linear: null or misaligned workspace");
  if (ws_bytes < p.bytes) return fail(TLR_ERR_WORKSPACE, "row_linear: workspace too small");
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (p.few) {
    const unsigned grid = (unsigned)cdiv(m, 16);
    if (dt == TLR_F32) few_kernel<float><<<grid, 512, 0, hs>>>(g, X, ldx);
    else if (dt == TLR_F16) few_kernel<_Float16><<<grid, 512, 0, hs>>>(g, X, ldx);
    else few_kernel<__bf16><<<grid, 512, 0, hs>>>(g, X, ldx);
    return launched("row_linear");
  }
  uint8_t *codes = static_cast<uint8_t *>(ws);
  float *scales = reinterpret_cast<float *>(codes + p.scales);
  g.b = Operand{codes, scales, p.ld, (int32_t)n};
  const RowQuantArgs a{X, n, n, ldx, p.ld, nullptr, codes, scales, (int32_t)k};
  if (dt == TLR_F32) row_quantize_launch<float>(a, hs);
  else if (dt == TLR_F16) row_quantize_launch<_Float16>(a, hs);
  else row_quantize_launch<__bf16>(a, hs);
  gemm_launch(g, p.choice, reinterpret_cast<int *>(codes + p.parts), hs);
  return launched("row_linear");
}

}  // namespace tlr
