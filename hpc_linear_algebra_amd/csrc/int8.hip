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
template <typename T, int W, int U> __global__ __launch_bounds__(256) void row_quantize_kernel(RowQuantArgs a) {
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
#pragma unroll
      for (int u = 0; u < U; ++u) get8(x + at + u * STEP, k - at - u * STEP, v[u]);
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
        if (at + u * STEP < up) *reinterpret_cast<u2 *>(out + at + u * STEP) = int8_codes8(v[u], s, q);
    } else {
      for (int c = at; c < up; c += STEP) {
        get8(x + c, k - c, v[0]);
        *reinterpret_cast<u2 *>(out + c) = int8_codes8(v[0], s, q);
      }
    }
  }
}

template <typename T> void row_quantize_launch(const RowQuantArgs &a, hipStream_t st) {
  const unsigned one = (unsigned)std::min<int64_t>((a.rows + 3) / 4, 1 << 22), all = (unsigned)std::min<int64_t>(a.rows, 1 << 22);
  if (a.k <= 512) row_quantize_kernel<T, 1, 1><<<one, 256, 0, st>>>(a);
  else if (a.k <= 2048) row_quantize_kernel<T, 1, 4><<<one, 256, 0, st>>>(a);
  else if (a.k <= 4096) row_quantize_kernel<T, 4, 2><<<all, 256, 0, st>>>(a);
  else if (a.k <= 8192) row_quantize_kernel<T, 4, 4><<<all, 256, 0, st>>>(a);
  else row_quantize_kernel<T, 4, 0><<<all, 256, 0, st>>>(a);
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
  int32_t groups, clear;                // clear: rows behind the last group become zeros
};

// The rows of B that a workgroup takes, and what belongs to them.
struct Rows {
  int first, end;           // end: of the group
  int group;                // -1: nothing to do; `groups`: zeros
};

// The `at`-th piece of TN rows, counted through the groups; `total` pieces there are.
// Offsets out of order or range give empty or shorter groups.
template <int TN> __device__ __forceinline__ int pieces(const RowGemmArgs &g, int e, int &lo, int &hi) {
  const int first = e <= g.groups ? min(max(g.offsets[e], 0), g.n) : g.n;
  const int next = e < g.groups ? min(max(g.offsets[e + 1], 0), g.n) : e == g.groups && g.clear ? g.n : 0;
  lo = first;
  hi = max(first, next);
  return (hi - lo + TN - 1) / TN;
}
__device__ __forceinline__ int scan64(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(x, d);
    if (lane >= d) x += v;
  }
  return x;
}
template <int TN> __device__ __forceinline__ int count_pieces(const RowGemmArgs &g) {
  const int lane = threadIdx.x & 63;
  int total = 0, lo, hi;
  for (int e0 = 0; e0 <= g.groups; e0 += 64) total += pieces<TN>(g, e0 + lane, lo, hi);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
  return __builtin_amdgcn_readfirstlane(total);
}
template <int TN> __device__ __forceinline__ Rows find_piece(const RowGemmArgs &g, int at) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int e0 = 0; e0 <= g.groups; e0 += 64) {
    int lo, hi;
    const int mine = pieces<TN>(g, e0 + lane, lo, hi), upto = before + scan64(mine, lane);
    const uint64_t past = __ballot(at < upto);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int start = __builtin_amdgcn_readlane(upto - mine, l);
      return Rows{__builtin_amdgcn_readlane(lo, l) + (at - start) * TN, __builtin_amdgcn_readlane(hi, l), e0 + l};
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  return Rows{0, 0, -1};
}

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

// Few columns or little work: a workgroup computes 16 rows of A against 16 rows of
// B, its eight waves taking every eighth block of 128 columns; fragments come
// straight from global memory, and the partial sums meet in LDS.
template <bool GROUPED> __global__ __launch_bounds__(512, 4) void strip_kernel(RowGemmArgs g) {
  constexpr int W = 8, UNROLL = 4;
  __shared__ int part[W][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int m0 = blockIdx.x * 16;
  int n0 = blockIdx.y * 16;
  bool zero = false;
  if constexpr (GROUPED) {
    const Rows rows = find_piece<16>(g, blockIdx.y);
    if (rows.group < 0) return;
    n0 = rows.first;
    zero = rows.group == g.groups;
    take_group(g, zero ? Rows{rows.first, rows.end, 0} : rows);
  }
  const uint8_t *arow = g.a.codes + (int64_t)min(m0 + r, g.m - 1) * g.a.ld + 16 * q;
  const uint8_t *brow = g.b.codes + (int64_t)min(n0 + r, g.n - 1) * g.b.ld + 16 * q;
  i4 acc = i4{0, 0, 0, 0};
  struct Block {
    u4 a[2], b[2];
  };
  auto load = [&](int kb, Block &x) {
    const int64_t c = (int64_t)kb * QB;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x.a[h] = *reinterpret_cast<const u4 *>(arow + c + 64 * h);
      x.b[h] = *reinterpret_cast<const u4 *>(brow + c + 64 * h);
    }
  };
  auto add = [&](const Block &x) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i4, x.a[h]), __builtin_bit_cast(i4, x.b[h]), acc, 0, 0, 0);
  };
  const int full = zero ? 0 : g.k / QB;
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
  if (!zero && kb == full && g.k > full * QB) {          // the cut block
    Block x;
    const int64_t o = (int64_t)full * QB - 16 * q;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x.a[h] = load16(arow + o, 16 * q + 64 * h, g.k - full * QB);
      x.b[h] = load16(brow + o, 16 * q + 64 * h, g.k - full * QB);
    }
    add(x);
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) part[wave][v][lane] = acc[v];
  __syncthreads();
  if (threadIdx.x < 256) {
    const int i = threadIdx.x & 15, j = threadIdx.x >> 4;      // row, column of the workgroup's block
    int v = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) v += part[w][i & 3][(i >> 2) * 16 + j];
    if (m0 + i < g.m && n0 + j < g.n) store_one(g, m0 + i, n0 + j, zero ? 0.0f : (float)v * g.b.scales[n0 + j] * g.a.scales[m0 + i]);
  }
}

// C tiles of TM x TN, WM x WN waves, each RI x CJ tiles of 16 x 16; the codes of two
// blocks of 128 columns in LDS, one read while the other is loaded.
template <bool GROUPED, int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2))) void tile_kernel(RowGemmArgs g) {
  constexpr int T = 64 * WM * WN, RI = TM / WM / 16, CJ = TN / WN / 16;
  static_assert(RI % 2 == 0, "");
  constexpr int AT_B = TM * QB, STAGE = (TM + TN) * QB;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4, wm = wave / WN, wn = wave % WN;

  // tile of this workgroup: workgroups go to the 8 XCDs in turn; each XCD takes
  // a contiguous part of the tiles, which run down 8 row tiles at a time
  int mt, nt;
  {
    const int tm = (g.m + TM - 1) / TM, tn = GROUPED ? count_pieces<TN>(g) : (g.n + TN - 1) / TN, all = tm * tn;
    const int id = blockIdx.x, x = id & 7, part = all >> 3, more = all & 7;
    if ((id >> 3) >= part + (x < more)) return;
    const int t = x * part + min(x, more) + (id >> 3);
    const int width = 8 * tn, band = t / width, h = min(8, tm - 8 * band), in = t - band * width;
    mt = 8 * band + in % h;
    nt = in / h;
  }
  const int m0 = mt * TM;
  int n0 = nt * TN;
  bool zero = false;
  if constexpr (GROUPED) {
    const Rows rows = find_piece<TN>(g, nt);
    if (rows.group < 0) return;
    n0 = rows.first;
    zero = rows.group == g.groups;
    take_group(g, zero ? Rows{rows.first, rows.end, 0} : rows);
  }
  i4 acc[RI][CJ];
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int j = 0; j < CJ; ++j) acc[i][j] = i4{0, 0, 0, 0};

  Panel<TM, T, true> pa;
  Panel<TN, T, false> pb;
  pa.init(g.a, m0, g.k, tid);
  pb.init(g.b, n0, g.k, tid);
  const int ar = wm * (TM / WM) + 8 * (r >> 2) + (r & 3), br = wn * (TN / WN) + r;
  const int aat = ar * QB + 16 * (q ^ a_key(ar)), bat = AT_B + br * QB + 16 * (q ^ b_key(br));
  auto meet = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  const int blocks = zero ? 0 : (g.k + QB - 1) / QB;
  const uint32_t base = lds_address(lds);
  if (blocks > 0) {
    pa.load_last(blocks - 1, base, wave, true);
    pb.load_last(blocks - 1, base + AT_B, wave, true);
    meet();
    if (g.k & (QB - 1)) {
      pa.cut(g.k & (QB - 1), lds, tid);
      pb.cut(g.k & (QB - 1), lds + AT_B, tid);
      meet();
    }
  }
  int now = 0;
  for (int kb = 0; kb < blocks; ++kb) {
    if (kb + 1 < blocks) {
#pragma unroll
      for (int i = 0; i < pa.N; ++i) pa.load(i, kb, base + (STAGE - now), wave);
#pragma unroll
      for (int i = 0; i < pb.N; ++i) pb.load(i, kb, base + (STAGE - now) + AT_B, wave);
    }
    const uint8_t *l = lds + now;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i4 b[CJ];
#pragma unroll
      for (int j = 0; j < CJ; ++j) b[j] = *reinterpret_cast<const i4 *>(l + (bat ^ 64 * h) + 16 * QB * j);
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        const i4 a = *reinterpret_cast<const i4 *>(l + (aat ^ 64 * h) + (i >> 1) * 32 * QB + (i & 1) * 4 * QB);
#pragma unroll
        for (int j = 0; j < CJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b[j], acc[i][j], 0, 0, 0);
      }
    }
    meet();
    now = STAGE - now;
  }

  // lane (r, q): rows 32 h + 8 q .. + 7 of its columns
  const int row0 = m0 + wm * (TM / WM), col0 = n0 + wn * (TN / WN);
#pragma unroll
  for (int h = 0; h < RI / 2; ++h) {
    const int row = row0 + 32 * h + 8 * q;
    if (row < g.m) {
      float sa[8];
      get8(g.a.scales + row, g.m - row, sa);
#pragma unroll
      for (int j = 0; j < CJ; ++j) {
        const int col = col0 + 16 * j + r;
        if (col < g.n) {
          const float sb = g.b.scales[col];
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = zero ? 0.0f : (float)acc[2 * h + (e >> 2)][j][e & 3] * sb * sa[e];
          store8(g, row, col, v);
        }
      }
    }
  }
}

// ---- which kernel ------------------------------------------------------------------------------------

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

enum Kind { STRIP, TILE_128 };
struct Shape {
  int rows, cols, threads;
};
constexpr Shape SHAPE[] = {{16, 16, 512}, {128, 128, 256}};

constexpr int64_t THREAD_LIM = (int64_t)1 << 32;

// Pieces of B's rows at most: each group ends with a piece that may be short, and so do the rows behind the last.
int64_t most_pieces(Kind kind, int64_t n, int32_t groups) {
  const int64_t tn = SHAPE[kind].cols;
  return groups ? std::min(n, (n + (groups + 1) * (tn - 1)) / tn) : cdiv(n, tn);
}
bool fits(Kind kind, int64_t m, int64_t n, int32_t groups) {
  const int64_t p = most_pieces(kind, n, groups);
  return kind == STRIP ? cdiv(m, 16) * 512 < THREAD_LIM && p <= 65535 : cdiv(m, SHAPE[kind].rows) * p * SHAPE[kind].threads < THREAD_LIM;
}

Kind choose(int64_t m, int64_t n, int64_t, int32_t groups) {
  const int64_t each = groups ? cdiv(n, groups) : n;
  return each <= 32 && fits(STRIP, m, n, groups) ? STRIP : TILE_128;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t SIZE_LIM = 0x7fffffff, PRODUCT_LIM = SIZE_LIM - 511, LD_LIM = (int64_t)1 << 22, K_LIM = 131071;
constexpr int MOST_GROUPS = 1024;

tlr_status launched(const char *what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TLR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
  return TLR_OK;
}

tlr_status check_sizes(int64_t m, int64_t n, int64_t k, int32_t groups) {
  if (m < 0 || n < 0 || k < 0 || m > PRODUCT_LIM || n > PRODUCT_LIM) return fail(TLR_ERR_INVALID_ARG, "row_gemm: size out of range");
  if (k > K_LIM) return fail(TLR_ERR_UNSUPPORTED, "row_gemm: 32-bit sums hold 131071 columns at most");
  if (groups < 0 || groups > MOST_GROUPS) return fail(TLR_ERR_INVALID_ARG, "row_gemm: groups are 1 .. 1024");
  if (!fits(TILE_128, m, n, groups)) return fail(TLR_ERR_INVALID_ARG, "row_gemm: too many tiles for a launch");
  return TLR_OK;
}

tlr_status check_operand(const char *name, const tlr_row_matrix *x, int64_t rows, int64_t k, Operand *o) {
  const std::string w = std::string("row_gemm: ") + name;
  if (!x || (!x->codes && k > 0) || !x->scales) return fail(TLR_ERR_INVALID_ARG, w + ": null matrix, codes or scales");
  if (x->ld % 16 != 0 || !aligned(x->codes, 16)) return fail(TLR_ERR_INVALID_ARG, w + ": codes and their rows must be 16-byte aligned");
  if (x->ld < k || x->ld >= LD_LIM) return fail(TLR_ERR_INVALID_ARG, w + ": leading dimension out of range");
  if (!aligned(x->scales, 4)) return fail(TLR_ERR_INVALID_ARG, w + ": misaligned scales");
  *o = Operand{static_cast<const uint8_t *>(x->codes), x->scales, x->ld, (int32_t)rows};
  return TLR_OK;
}

template <Kind KIND, int WM, int WN> void tile_launch(const RowGemmArgs &g, hipStream_t st) {
  constexpr int TM = SHAPE[KIND].rows, TN = SHAPE[KIND].cols;
  static_assert(SHAPE[KIND].threads == 64 * WM * WN, "");
  const unsigned grid = (unsigned)(cdiv(g.m, TM) * most_pieces(KIND, g.n, g.offsets ? g.groups : 0));
  if (g.offsets) tile_kernel<true, TM, TN, WM, WN><<<grid, 64 * WM * WN, 0, st>>>(g);
  else tile_kernel<false, TM, TN, WM, WN><<<grid, 64 * WM * WN, 0, st>>>(g);
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
  const Kind c = choose(m, n, k, groups);
  const Shape &s = SHAPE[c];
  const int64_t p = most_pieces(c, n, groups);
  *out = tlr_block_gemm_choice{s.rows, s.cols, s.threads, 1, 1, 0, c == STRIP ? cdiv(m, 16) : cdiv(m, s.rows) * p, c == STRIP ? p : 1, 0};
  return TLR_OK;
}

tlr_status row_gemm(tlr_dtype dt, int64_t m, int64_t n, int64_t k, const tlr_row_matrix *A, const tlr_row_matrix *B,
                    const tlr_row_groups *groups, void *C, int64_t ldc, void *ws, size_t ws_bytes, void *stream) {
  if (dt == TLR_F64) return fail(TLR_ERR_UNSUPPORTED, "row_gemm: C of type TLR_F64 is not provided");
  if (dt != TLR_F32 && dt != TLR_F16 && dt != TLR_BF16) return fail(TLR_ERR_INVALID_ARG, "row_gemm: bad dtype of C");
  tlr_status st = check_sizes(m, n, k, groups ? std::max(groups->count, 1) : 0);
  if (st != TLR_OK) return st;
  if (ldc < std::max<int64_t>(1, m) || ldc > SIZE_LIM) return fail(TLR_ERR_INVALID_ARG, "row_gemm: ldc out of range");
  RowGemmArgs g{};
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
  if (m == 0 || n == 0) return TLR_OK;
  if ((st = check_operand("A", A, m, k, &g.a)) != TLR_OK) return st;
  if ((st = check_operand("B", B, n, k, &g.b)) != TLR_OK) return st;
  if (!C || !aligned(C, dt == TLR_F32 ? 4 : 2)) return fail(TLR_ERR_INVALID_ARG, "row_gemm: null or misaligned C");
  g.m = (int32_t)m;
  g.n = (int32_t)n;
  g.k = (int32_t)k;
  g.c = C;
  g.ldc = ldc;
  g.dt = dt;
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (choose(m, n, k, g.groups) == STRIP) {
    const dim3 grid((unsigned)cdiv(m, 16), (unsigned)most_pieces(STRIP, n, g.groups));
    if (groups) strip_kernel<true><<<grid, 512, 0, hs>>>(g);
    else strip_kernel<false><<<grid, 512, 0, hs>>>(g);
  } else {
    tile_launch<TILE_128, 2, 2>(g, hs);
  }
  return launched("row_gemm");
}

}  // namespace tlr
