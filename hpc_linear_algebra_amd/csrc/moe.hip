// A mixture-of-experts layer for a few tokens, gfx950.
//
//   l = Wr x;  prob = softmax(l);  the topk experts e of largest l;
//   y = sum_e prob_e D_e (silu(G_e x) * (U_e x)).
//
// With few tokens every chosen expert's weights are read once and used for a
// handful of columns: the layer is bound by the weights' bytes.  The products
// run on the 16-bit matrix cores with the weight rows as the 16-row operand
// (fragments straight from global memory, no LDS: nothing is shared but the
// tokens, which stay in L2) and the tokens of one expert as the columns.
// 8-bit weights are widened to the 16-bit type in registers, exactly, and
// their scale is applied to each block's float sum.  64 tokens of 128 experts
// (2048, 1024, top 8, bf16): gate/up 179 - 185 us for 1.06 GB (5.7 - 5.9 TB/s), down
// 90 - 94 us for 0.53 GB; 13 tokens of 96 experts (2064, 1168, top 6, e4m3): 52 and
// 32 us for 263 and 131 MB.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "tlr_ops.h"

namespace tlr {

namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int MAX_TOKENS = 256, MAX_EXPERTS = 512, MAX_TOPK = 16;
constexpr int RT = 16;                    // tokens of a router workgroup
constexpr int FEW = 256;                  // assignments that an expert's workgroup looks through itself
constexpr int MAX_SPLITS = 4;             // workgroups that share a router tile's columns
constexpr int ROUTED = 32, BLOCKS = 64;   // counters: 0.. router groups, ROUTED all groups, BLOCKS.. row blocks of y

// The 16-bit type of x, y and the products.  LOW: what the lower of the two
// numbers that stand for silu(g) u is multiplied with.  Half precision ends at
// 2^-24 and would cut the sum of the two there; with 2^11 it is cut at 2^-35, and
// the largest remainder, 16 beside 65504, still fits.
template <typename H> struct Num;
template <> struct Num<_Float16> {
  static constexpr float LOW = 0x1p11f;
  typedef _Float16 v8 __attribute__((ext_vector_type(8)));
  typedef _Float16 v2 __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ f4 mma(u4 a, u4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  template <bool HI> static __device__ __forceinline__ uint32_t widen(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
  }
};
template <> struct Num<__bf16> {
  static constexpr float LOW = 1.0f;
  typedef __bf16 v8 __attribute__((ext_vector_type(8)));
  typedef __bf16 v2 __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ f4 mma(u4 a, u4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  template <bool HI> static __device__ __forceinline__ uint32_t widen(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  }
};

struct MoeArgs {
  int32_t tokens, hidden, inter, experts, topk, normalize;
  const uint16_t *x;
  int64_t ldx;
  uint16_t *y;
  int64_t ldy;
  const uint16_t *router;
  const uint8_t *gate_up, *down;
  const float *gate_up_scales, *down_scales;
  int32_t *ids;
  float *weights;
  int32_t *arrived;         // counters of workgroups that are done; 0 between calls
  int32_t *units;           // how many experts were chosen
  int4 *unit;               // each of them: expert, first place in order, assignments, 0
  int32_t *order;           // assignments (token * topk + choice) by expert
  double *logits;           // splits x tokens x experts: parts of the router product
  int32_t splits;
  int32_t sorted;           // the experts' workgroups take their assignments from the router's tables
  uint16_t *hi, *lo;        // tokens*topk x inter: silu(g) u as hi + lo / LOW
  float *part;              // tokens*topk x hidden: the experts' outputs
};

// Values that workgroups of one launch pass on go past the chiplets' caches, both
// ways, by relaxed agent-scope accesses.  arrive() counts this workgroup as
// done once all of its stores have been acknowledged there, and says whether it
// was the last of n; the counter is 0 again then.  A release fence would write
// back the whole L2 besides (a router of 64 tokens: 32 us with, 20 without).
template <typename T> __device__ __forceinline__ void put(T *p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T> __device__ __forceinline__ T get(const T *p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool arrive(int32_t *counter, int n, int *shared) {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0);      // every wave: its own stores
  __syncthreads();
  if (threadIdx.x == 0) {
    const int before = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *shared = before == n - 1;
    if (before == n - 1) put(counter, 0);
  }
  __syncthreads();
  asm volatile("" ::: "memory");
  return *shared != 0;
}

// Eight 16-bit entries as floats.
template <typename H> __device__ __forceinline__ void unpack8(u4 w, float (&v)[8]) {
  typedef typename Num<H>::v8 v8;
  const v8 h = __builtin_bit_cast(v8, w);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)h[e];
}

// A double as a number whose order is the logits' order, NaN on top.
__device__ __forceinline__ uint64_t sort_key(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  if (x != x) return ~0ull;
  const uint64_t z = x == 0.0 ? 0ull : b;      // -0 and 0 tie
  return (z >> 63) ? ~z : z | 0x8000000000000000ull;
}

// Largest of all lanes' x, in all of them.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x128, 0xf, 0xf, true));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x124, 0xf, 0xf, true));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x122, 0xf, 0xf, true));
  x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x121, 0xf, 0xf, true));
  const uint32_t a = max((uint32_t)__builtin_amdgcn_readlane((int)x, 0), (uint32_t)__builtin_amdgcn_readlane((int)x, 16));
  const uint32_t b = max((uint32_t)__builtin_amdgcn_readlane((int)x, 32), (uint32_t)__builtin_amdgcn_readlane((int)x, 48));
  return max(a, b);
}

// One wave chooses the experts of token t: topk times the largest key, its high
// word first, then its low word, then the lowest index.  PER experts a lane.
template <int PER> __device__ __forceinline__ void select(const MoeArgs &a, int t, int lane) {
  const double *l = a.logits + (int64_t)t * a.experts;
  double x[PER];
  uint64_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    double part[MAX_SPLITS];          // clamped, not branched on: all loads in flight at once
#pragma unroll
    for (int z = 0; z < MAX_SPLITS; ++z)
      part[z] = get(l + (int64_t)min(z, a.splits - 1) * a.tokens * a.experts + min(e, a.experts - 1));
    x[i] = part[0];
#pragma unroll
    for (int z = 1; z < MAX_SPLITS; ++z) x[i] += z < a.splits ? part[z] : 0.0;
    key[i] = e < a.experts ? sort_key(x[i]) : 0;      // no number's key is 0
  }
  double best = 0.0, mine = 0.0;      // lane j: the logit of choice j
  int id = 0;
  for (int j = 0; j < a.topk; ++j) {
    uint64_t top = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) top = max(top, key[i]);
    const uint32_t hi = wave_max((uint32_t)(top >> 32));
    const uint64_t tied = __ballot((uint32_t)(top >> 32) == hi);
    // one lane has that high word, most often: its low word then
    const uint32_t lo = (tied & (tied - 1)) == 0 ? (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)top, __builtin_ctzll(tied))
                                                 : wave_max((uint32_t)(top >> 32) == hi ? (uint32_t)top : 0u);
    const uint64_t k = (uint64_t)hi << 32 | lo;
    int e = -1;
    double v = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint64_t b = __ballot(key[i] == k);
      if (e < 0 && b != 0) {
        const int at = __builtin_ctzll(b);
        e = at + 64 * i;
        const uint64_t w = __builtin_bit_cast(uint64_t, x[i]);
        v = __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(w >> 32), at) << 32 |
                                           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)w, at));
        if (lane == at) key[i] = 0;
      }
    }
    if (j == 0) best = v;
    if (lane == j) {
      mine = v;
      id = e;
    }
  }
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) z += lane + 64 * i < a.experts ? expf((float)(x[i] - best)) : 0.0f;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) z += __shfl_xor(z, o);
  const float p = lane < a.topk ? expf((float)(mine - best)) : 0.0f;
  if (a.normalize) {
    z = p;                            // 0 past the choices: the sum over 16 lanes
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) z += __shfl_xor(z, o);
  }
  if (lane < a.topk) {
    put(a.ids + t * a.topk + lane, id);
    a.weights[t * a.topk + lane] = p / z;
  }
}

// One workgroup: the assignments by expert and the chosen experts.  Places within
// an expert go in the order of the atomics, which no result depends on: an
// assignment is a column of a product, whichever one.
template <int THREADS> __device__ __forceinline__ void sort(const MoeArgs &a) {
  __shared__ int count[MAX_EXPERTS], place[MAX_EXPERTS];
  constexpr int MAX = MAX_TOKENS * MAX_TOPK / THREADS;
  const int tid = threadIdx.x, n = a.tokens * a.topk;
  for (int e = tid; e < MAX_EXPERTS; e += THREADS) count[e] = 0;
  __syncthreads();
  int id[MAX];
#pragma unroll
  for (int i = 0; i < MAX; ++i) {
    id[i] = tid + i * THREADS < n ? get(a.ids + tid + i * THREADS) : -1;
    if (id[i] >= 0) atomicAdd(&count[id[i]], 1);
  }
  __syncthreads();
  if (tid < 64) {
    constexpr int PER = MAX_EXPERTS / 64;
    int c[PER], sum = 0, some = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      c[i] = count[tid * PER + i];
      sum += c[i];
      some += c[i] > 0 ? 1 : 0;
    }
    int at = sum, u = some;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int x = __shfl_up(at, o), y = __shfl_up(u, o);
      at += tid >= o ? x : 0;
      u += tid >= o ? y : 0;
    }
    if (tid == 63) *a.units = u;
    at -= sum;
    u -= some;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      place[tid * PER + i] = at;
      if (c[i] > 0) a.unit[u++] = int4{tid * PER + i, at, c[i], 0};
      at += c[i];
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MAX; ++i)
    if (id[i] >= 0) a.order[atomicAdd(&place[id[i]], 1)] = tid + i * THREADS;
}

// The experts of token t chosen by one wave.
__device__ __forceinline__ void choose(const MoeArgs &a, int t, int lane) {
  if (a.experts <= 64) select<1>(a, t, lane);
  else if (a.experts <= 128) select<2>(a, t, lane);
  else if (a.experts <= 256) select<4>(a, t, lane);
  else select<8>(a, t, lane);
}

// Few tokens, one by one: a wave per expert, sums in double.  A product of two half
// precision numbers is an exact float; one of two bfloat16 numbers may lie outside
// float's range and is taken in double.  The workgroup that is done last with a
// token chooses: a launch of its own would cost 4 us.  Against the matrix kernel
// below the layer takes 1.8 us less at 16 tokens and 8 experts, 1.0 less at 8 and
// 32, 0.8 less at 16 and 32; 0.8 more at 12 and 64, 0.6 more at 8 and 96.
bool singly(int64_t tokens, int experts) { return tokens == 1 || (tokens <= 16 && tokens * experts <= 512); }
template <typename H> __global__ __launch_bounds__(256) void router_one_kernel(MoeArgs a) {
  __shared__ int last;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = blockIdx.x * 4 + wave, t = blockIdx.y;
  if (e < a.experts) {
    const uint16_t *w = a.router + (int64_t)e * a.hidden, *x = a.x + t * a.ldx;
    double s = 0.0;
#pragma unroll 4
    for (int c = 8 * lane; c < a.hidden; c += 512) {
      float wf[8], xf[8];
      unpack8<H>(*reinterpret_cast<const u4 *>(w + c), wf);
      unpack8<H>(*reinterpret_cast<const u4 *>(x + c), xf);
#pragma unroll
      for (int v = 0; v < 8; ++v)
        if constexpr (std::is_same_v<H, _Float16>) s += (double)(wf[v] * xf[v]);
        else s = __builtin_fma((double)wf[v], (double)xf[v], s);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if (lane == 0) put(a.logits + (int64_t)t * a.experts + e, s);
  }
  if (!arrive(a.arrived + t, gridDim.x, &last)) return;
  if (wave == 0) choose(a, t, lane);
  if (!a.sorted) return;
  if (arrive(a.arrived + ROUTED, gridDim.y, &last)) sort<256>(a);
}

constexpr int RW = 16;      // waves of a router workgroup
static_assert(RW == RT, "a wave chooses for each token");

// More of them: 16 experts x 16 tokens on the 64-bit matrix cores, the waves and
// the workgroups of grid z taking groups of 32 columns in turn.  Lane (r, q)
// supplies columns 8 q .. + 7 of expert row r and of token r and holds the sums
// of experts q + 4 v and token r.  The vector units took 20 us for 64 tokens of
// 128 experts (2048 columns), much of it converting every product; here every
// entry is converted once a tile: 13 us, 3.5 of them the product, the rest loads
// and counts from one workgroup to the next.  The workgroup that is done last
// with its tokens chooses their experts, a wave per token, and the last of all
// sorts the assignments.
template <typename H> __global__ __launch_bounds__(64 * RW) void router_kernel(MoeArgs a) {
  typedef double d4 __attribute__((ext_vector_type(4)));
  __shared__ double part[RW][4][64];
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4, e0 = blockIdx.x * 16, t0 = blockIdx.y * RT;
  const uint16_t *w = a.router + (int64_t)min(e0 + r, a.experts - 1) * a.hidden;
  const uint16_t *x = a.x + min(t0 + r, a.tokens - 1) * a.ldx;
  d4 acc = d4{0, 0, 0, 0};
  for (int k0 = 32 * (wave + RW * (int)blockIdx.z); k0 < a.hidden; k0 += 32 * RW * (int)gridDim.z) {
    const int k = k0 + 8 * q;
    const bool in = k < a.hidden;
    float wf[8], xf[8];
    unpack8<H>(*reinterpret_cast<const u4 *>(w + (in ? k : 0)), wf);
    unpack8<H>(*reinterpret_cast<const u4 *>(x + (in ? k : 0)), xf);
#pragma unroll
    for (int v = 0; v < 8; ++v)
      acc = __builtin_amdgcn_mfma_f64_16x16x4f64(in ? (double)wf[v] : 0.0, in ? (double)xf[v] : 0.0, acc, 0, 0, 0);
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) part[wave][v][lane] = acc[v];
  __syncthreads();
  if (tid < 256) {
    const int i = q + 4 * wave, t = r;
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < RW; ++k) s += part[k][wave][lane];
    if (e0 + i < a.experts && t0 + t < a.tokens) put(a.logits + ((int64_t)blockIdx.z * a.tokens + t0 + t) * a.experts + e0 + i, s);
  }
  if (!arrive(a.arrived + blockIdx.y, gridDim.x * gridDim.z, &last)) return;
  if (t0 + wave < a.tokens) choose(a, t0 + wave, lane);
  if (!a.sorted) return;
  if (arrive(a.arrived + ROUTED, gridDim.y, &last)) sort<64 * RW>(a);
}

// A column group of an expert's rows and of NJ tiles of 16 token columns, as
// loaded: lane (r, q) = (lane % 16, lane / 16) holds columns k0 + 64 s + 16 q ..
// + 15 of weight row r and of token column r.  16-bit weights: 64 columns (a
// row's piece is a 128-byte line), 8-bit ones: 128, which share a scale.
template <typename H, bool W8, int RTILE, int NJ, bool TWO> struct Group {
  static constexpr int SUB = W8 ? 2 : 1, COLS = 64 * SUB;
  u4 w[RTILE][2], x[NJ][SUB][2], x2[TWO ? NJ : 1][SUB][2];
  float s[RTILE];

  // CUT: the group may reach past column K (a multiple of 16): zeros there.
  template <bool CUT>
  __device__ __forceinline__ void load(int g, int K, int q, const uint8_t *const (&wp)[RTILE], const float *const (&ws)[RTILE],
                                       int64_t wlds, const uint16_t *const (&xp)[NJ], const uint16_t *const (&xp2)[NJ]) {
    const u4 zero = u4{0, 0, 0, 0};
#pragma unroll
    for (int b = 0; b < SUB; ++b) {
      int k = g * COLS + 64 * b + 16 * q;
      const bool in = !CUT || k < K;
      if (CUT) k = in ? k : 0;
#pragma unroll
      for (int i = 0; i < RTILE; ++i) {
        if constexpr (W8) {
          w[i][b] = *reinterpret_cast<const u4 *>(wp[i] + k);
          if (CUT) w[i][b] = in ? w[i][b] : zero;
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            w[i][h] = reinterpret_cast<const u4 *>(wp[i] + 2 * k)[h];
            if (CUT) w[i][h] = in ? w[i][h] : zero;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[j][b][h] = reinterpret_cast<const u4 *>(xp[j] + k)[h];
          if (CUT) x[j][b][h] = in ? x[j][b][h] : zero;
          if constexpr (TWO) {
            x2[j][b][h] = reinterpret_cast<const u4 *>(xp2[j] + k)[h];
            if (CUT) x2[j][b][h] = in ? x2[j][b][h] : zero;
          }
        }
    }
    if constexpr (W8)
#pragma unroll
      for (int i = 0; i < RTILE; ++i) s[i] = ws[i][g * wlds];
  }

  __device__ __forceinline__ void add(f4 (&acc)[RTILE][NJ]) const {
#pragma unroll
    for (int i = 0; i < RTILE; ++i) {
      f4 d[NJ], low[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        d[j] = W8 ? f4{0, 0, 0, 0} : acc[i][j];
        low[j] = f4{0, 0, 0, 0};
      }
#pragma unroll
      for (int b = 0; b < SUB; ++b) {
        u4 f[2];
        if constexpr (W8) {
          const u4 c = w[i][b];
#pragma unroll
          for (int p = 0; p < 2; ++p)
            f[p] = u4{Num<H>::template widen<false>(c[2 * p]), Num<H>::template widen<true>(c[2 * p]),
                      Num<H>::template widen<false>(c[2 * p + 1]), Num<H>::template widen<true>(c[2 * p + 1])};
        } else {
          f[0] = w[i][0];
          f[1] = w[i][1];
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          d[j] = Num<H>::mma(f[0], x[j][b][0], d[j]);
          d[j] = Num<H>::mma(f[1], x[j][b][1], d[j]);
          if constexpr (TWO) {
            f4 &l = Num<H>::LOW == 1.0f ? d[j] : low[j];
            l = Num<H>::mma(f[0], x2[j][b][0], l);
            l = Num<H>::mma(f[1], x2[j][b][1], l);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        if constexpr (TWO && Num<H>::LOW != 1.0f)
#pragma unroll
          for (int v = 0; v < 4; ++v) d[j][v] = __builtin_fmaf(low[j][v], 1.0f / Num<H>::LOW, d[j][v]);
        if constexpr (W8)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(s[i], d[j][v], acc[i][j][v]);
        else acc[i][j] = d[j];
      }
    }
  }
};

// RTILE row tiles of an expert's matrix against NJ tiles of token columns, this
// wave taking every waves-th column group, UNROLL of them in flight.
template <typename H, bool W8, int RTILE, int NJ, bool TWO, int UNROLL>
__device__ __forceinline__ void multiply(f4 (&acc)[RTILE][NJ], const uint8_t *const (&w)[RTILE], const float *const (&ws)[RTILE],
                                         int64_t wlds, const uint16_t *const (&x)[NJ], const uint16_t *const (&x2)[NJ], int K,
                                         int wave, int waves, int q) {
  typedef Group<H, W8, RTILE, NJ, TWO> G;
  const int full = K / G::COLS;
  int g = wave;
  for (; g + (UNROLL - 1) * waves < full; g += UNROLL * waves) {
    G v[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) v[u].template load<false>(g + u * waves, K, q, w, ws, wlds, x, x2);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) v[u].add(acc);
  }
  for (; g * G::COLS < K; g += waves) {
    G v;
    v.template load<true>(g, K, q, w, ws, wlds, x, x2);
    v.add(acc);
  }
}

// silu(g) u as a sum hi + lo / LOW of two numbers of the type: one would round the
// sum that the down product takes to 8 or 11 bits, two keep 16 or 22.
template <typename H> __device__ __forceinline__ void put_act(const MoeArgs &a, int64_t at, float g, float u) {
  const float v = g / (1.0f + expf(-g)) * u;
  const H hi = (H)v;
  const float rest = v - (float)hi;
  const H lo = (H)(__builtin_isfinite(rest) ? rest * Num<H>::LOW : 0.0f);     // beyond the type's range hi is infinite
  a.hi[at] = __builtin_bit_cast(uint16_t, hi);
  a.lo[at] = __builtin_bit_cast(uint16_t, lo);
}

constexpr int WV = 4;       // waves of an expert workgroup

// The expert of this workgroup's grid row and its assignments, order[0 .. count).
// SORTED: from the router's tables.  Otherwise every workgroup looks through the
// choices (at most FEW, one a thread): with fewer of them than experts a grid row
// is an assignment, which stands for its expert when no earlier one has the same,
// else a grid row is an expert.  False if there is nothing to do.
template <bool SORTED>
__device__ __forceinline__ bool work(const MoeArgs &a, int *list, int *places, int &e, int &count, const int *&order) {
  if constexpr (SORTED) {
    if ((int)blockIdx.y >= *a.units) return false;
    const int4 unit = a.unit[blockIdx.y];
    e = unit.x;
    count = unit.z;
    order = a.order + unit.y;
    return true;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = a.tokens * a.topk;
  const bool by_row = n < a.experts;
  e = by_row ? a.ids[blockIdx.y] : (int)blockIdx.y;
  const bool hit = tid < n && a.ids[min(tid, n - 1)] == e;
  const uint64_t b = __ballot(hit);
  if (lane == 0) places[wave] = __popcll(b);
  __syncthreads();
  int before = 0;
  count = 0;
#pragma unroll
  for (int w = 0; w < WV; ++w) {
    before += w < wave ? places[w] : 0;
    count += places[w];
  }
  if (hit) list[before + __popcll(b & ((1ull << lane) - 1))] = tid;
  __syncthreads();
  order = list;
  return count > 0 && (!by_row || list[0] == (int)blockIdx.y);
}

// silu(G x) * (U x) for 16 of an expert's inter rows and 16 NJ of its tokens.
template <typename H, bool W8, int NJ, int UNROLL>
__device__ __forceinline__ void gate_up(const MoeArgs &a, int e, int count, const int *order, int n0, float (*part)[2][4][64]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4, i0 = blockIdx.x * 16;
  const int64_t es = W8 ? 1 : 2;
  const uint8_t *w[2];
  const float *ws[2] = {nullptr, nullptr};
  const int64_t wlds = (2 * a.inter + 127) / 128;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t row = (int64_t)i * a.inter + i0;
    w[i] = a.gate_up + ((int64_t)e * 2 * a.inter + row + r) * a.hidden * es;
    if constexpr (W8) ws[i] = a.gate_up_scales + (int64_t)e * ((a.hidden + 127) / 128) * wlds + (row >> 7);
  }
  const uint16_t *x[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) x[j] = a.x + (order[min(n0 + 16 * j + r, count - 1)] / a.topk) * a.ldx;
  f4 acc[2][NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[0][j] = acc[1][j] = f4{0, 0, 0, 0};
  multiply<H, W8, 2, NJ, false, UNROLL>(acc, w, ws, wlds, x, x, a.hidden, wave, WV, q);
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[wave][i][v][lane] = acc[i][j][v];
    __syncthreads();
    // thread (row i, column c) of the 16 x 16 block
    const int i = tid & 15, c = tid >> 4, at = (i >> 2) * 16 + c;
    if (n0 + 16 * j + c < count) {
      float g = 0.0f, u = 0.0f;
#pragma unroll
      for (int k = 0; k < WV; ++k) {
        g += part[k][0][i & 3][at];
        u += part[k][1][i & 3][at];
      }
      put_act<H>(a, (int64_t)order[n0 + 16 * j + c] * a.inter + i0 + i, g, u);
    }
  }
}

template <typename H, bool W8, bool SORTED> __global__ __launch_bounds__(64 * WV) void gate_up_kernel(MoeArgs a) {
  __shared__ float part[WV][2][4][64];
  __shared__ int list[SORTED ? 1 : FEW], places[WV];
  int e, count;
  const int *order;
  if (!work<SORTED>(a, list, places, e, count, order)) return;
  int n0 = 0;
  for (; n0 + 16 < count; n0 += 32) gate_up<H, W8, 2, 1>(a, e, count, order, n0, part);
  if (n0 < count) gate_up<H, W8, 1, 2>(a, e, count, order, n0, part);
}

// 16 RTILE rows of an expert's down product for 16 NJ of its tokens.
template <typename H, bool W8, int RTILE, int NJ, int UNROLL>
__device__ __forceinline__ void down(const MoeArgs &a, int e, int count, const int *order, int n0, float (*part)[RTILE][4][64]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4, h0 = blockIdx.x * 16 * RTILE;
  const int64_t es = W8 ? 1 : 2;
  const int64_t wlds = (a.hidden + 127) / 128;
  const uint8_t *w[RTILE];
  const float *ws[RTILE];
#pragma unroll
  for (int i = 0; i < RTILE; ++i) {
    const int h = min(h0 + 16 * i, a.hidden - 16);      // a tile past the end: the last one again, not stored
    w[i] = a.down + ((int64_t)e * a.hidden + h + r) * a.inter * es;
    ws[i] = W8 ? a.down_scales + (int64_t)e * ((a.inter + 127) / 128) * wlds + (h >> 7) : nullptr;
  }
  const uint16_t *x[NJ], *x2[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int64_t at = (int64_t)order[min(n0 + 16 * j + r, count - 1)] * a.inter;
    x[j] = a.hi + at;
    x2[j] = a.lo + at;
  }
  f4 acc[RTILE][NJ];
#pragma unroll
  for (int i = 0; i < RTILE; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f4{0, 0, 0, 0};
  multiply<H, W8, RTILE, NJ, true, UNROLL>(acc, w, ws, wlds, x, x2, a.inter, wave, WV, q);
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RTILE; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[wave][i][v][lane] = acc[i][j][v];
    __syncthreads();
    const int i = tid & 15, c = tid >> 4, o = (i >> 2) * 16 + c;
    if (n0 + 16 * j + c < count) {
      float *to = a.part + (int64_t)order[n0 + 16 * j + c] * a.hidden + h0 + i;
#pragma unroll
      for (int t = 0; t < RTILE; ++t) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < WV; ++k) s += part[k][t][i & 3][o];
        if (h0 + 16 * t >= a.hidden) continue;
        if constexpr (RTILE == 1) put(to + 16 * t, s);
        else to[16 * t] = s;
      }
    }
  }
}

// y of a token at row h from the parts of its experts, in the order of its choices.
template <typename H, bool SAME_LAUNCH> __device__ __forceinline__ void add_parts(const MoeArgs &a, int t, int h) {
  const float *from = a.part + (int64_t)t * a.topk * a.hidden + h, *weight = a.weights + t * a.topk;
  float s = 0.0f;
#pragma unroll 8
  for (int j = 0; j < a.topk; ++j) {
    const float *p = from + (int64_t)j * a.hidden;
    s += weight[j] * (SAME_LAUNCH ? get(p) : *p);
  }
  a.y[t * a.ldy + h] = __builtin_bit_cast(uint16_t, (H)s);
}

// Down products of one expert and 16 RTILE rows of y.  RTILE 1 (few workgroups):
// the workgroup that is last with its rows adds the parts.  RTILE 2: left to a
// launch of its own, since a workgroup would hold its place for another 2 us until
// it knows whether it is the last (2 tokens, 1 of 8 experts of 512 x 256: 12.7 us
// with, 14.2 without; 16 tokens, 2 of 8 of 512 x 1024: 17.5 and 18.3; 4 tokens, 8
// of 64 of 512 x 256: 20.6 and 17.5); 4 waves a SIMD for 8-bit weights, whose two groups
// in flight would take 148 registers.
template <typename H, bool W8, int RTILE, bool SORTED>
__global__ __launch_bounds__(64 * WV, W8 && RTILE == 2 ? 4 : 1) void down_kernel(MoeArgs a) {
  __shared__ float part[WV][RTILE][4][64];
  __shared__ int list[SORTED ? 1 : FEW], places[WV];
  int e, count;
  const int *order;
  const bool some = work<SORTED>(a, list, places, e, count, order);
  if (SORTED && !some) return;
  if (some) {
    int n0 = 0;
    for (; n0 + 16 < count; n0 += 32) down<H, W8, RTILE, 2, 1>(a, e, count, order, n0, part);
    if (n0 < count) down<H, W8, RTILE, 1, W8 && RTILE == 2 ? 1 : 2>(a, e, count, order, n0, part);
  }
  if constexpr (RTILE == 1) {
    __shared__ int last;
    // rows without an expert count too where their number is not known
    if (!arrive(a.arrived + BLOCKS + blockIdx.x, SORTED ? *a.units : gridDim.y, &last)) return;
    for (int x = threadIdx.x; x < 16 * a.tokens; x += 64 * WV) add_parts<H, true>(a, x >> 4, blockIdx.x * 16 + (x & 15));
  }
}

// 16 weights of a row as floats.
template <typename H, bool W8> __device__ __forceinline__ void floats16(const u4 (&w)[W8 ? 1 : 2], float (&y)[16]) {
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    float z[8];
    if constexpr (W8) {
      typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = (int)w[0][2 * b + i];
        const f2 l = __builtin_amdgcn_cvt_pk_f32_fp8(c, false), h = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
        z[4 * i] = l[0];
        z[4 * i + 1] = l[1];
        z[4 * i + 2] = h[0];
        z[4 * i + 3] = h[1];
      }
    } else {
      unpack8<H>(w[b], z);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[8 * b + i] = z[i];
  }
}

// One token.  Its products are the weights' bytes and nothing else, and one
// column of sixteen is all that the matrix cores would have, so they run in
// float on the vector units, threads side by side along a row.

// silu(G x) * (U x) of one choice: a wave takes ONE_PAIRS gate rows and their up
// rows (2048 x 1024, 8 of 64 experts in bf16, the whole layer: 26.1 us with one
// pair, 26.4 with two, 28.6 with four, 27.8 with the matrix kernel).
constexpr int ONE_PAIRS = 1;
template <typename H, bool W8> __global__ __launch_bounds__(256) void gate_up_one_kernel(MoeArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i0 = (blockIdx.x * 4 + wave) * ONE_PAIRS, j = blockIdx.y, e = a.ids[j];
  const int64_t slds = (2 * a.inter + 127) / 128, sblocks = (a.hidden + 127) / 128;
  constexpr int N = W8 ? 1 : 2, ES = W8 ? 1 : 2;
  float acc[ONE_PAIRS][2];
#pragma unroll
  for (int p = 0; p < ONE_PAIRS; ++p) acc[p][0] = acc[p][1] = 0.0f;
#pragma unroll 1
  for (int c = 16 * lane; c < a.hidden; c += 1024) {
    u4 w[ONE_PAIRS][2][N];
    float s[ONE_PAIRS][2];
#pragma unroll
    for (int p = 0; p < ONE_PAIRS; ++p)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int64_t row = (int64_t)g * a.inter + i0 + p;
        const u4 *from = reinterpret_cast<const u4 *>(a.gate_up + (((int64_t)e * 2 * a.inter + row) * a.hidden + c) * ES);
#pragma unroll
        for (int b = 0; b < N; ++b) w[p][g][b] = from[b];
        if constexpr (W8) s[p][g] = a.gate_up_scales[(e * sblocks + (c >> 7)) * slds + (row >> 7)];
      }
    const u4 x2[2] = {reinterpret_cast<const u4 *>(a.x + c)[0], reinterpret_cast<const u4 *>(a.x + c)[1]};
    float x[16];
    floats16<H, false>(x2, x);
#pragma unroll
    for (int p = 0; p < ONE_PAIRS; ++p)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float y[16], d = W8 ? 0.0f : acc[p][g];
        floats16<H, W8>(w[p][g], y);
#pragma unroll
        for (int i = 0; i < 16; ++i) d = __builtin_fmaf(y[i], x[i], d);
        acc[p][g] = W8 ? __builtin_fmaf(s[p][g], d, acc[p][g]) : d;
      }
  }
#pragma unroll
  for (int p = 0; p < ONE_PAIRS; ++p) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      acc[p][0] += __shfl_xor(acc[p][0], o);
      acc[p][1] += __shfl_xor(acc[p][1], o);
    }
    if (lane == 0) put_act<H>(a, (int64_t)j * a.inter + i0 + p, acc[p][0], acc[p][1]);
  }
}

// ONE_ROWS rows of y whole: the threads share the (choice, 16 columns) pairs of
// the topk down products and weight every sum where it arises, so that nothing is
// left to add and no workgroup waits for another (2048 rows of 8 x 1024 in bf16:
// 9.8 us on the matrix cores with the last workgroups adding, this way 7).
constexpr int ONE_ROWS = 2;
template <typename H, bool W8> __global__ __launch_bounds__(256) void down_one_kernel(MoeArgs a) {
  __shared__ float part[4][ONE_ROWS];
  const int tid = threadIdx.x, h0 = blockIdx.x * ONE_ROWS;
  const int chunks = a.inter / 16, all = a.topk * chunks;
  const int64_t slds = (a.hidden + 127) / 128, sblocks = (a.inter + 127) / 128;
  constexpr int N = W8 ? 1 : 2, ES = W8 ? 1 : 2;
  float acc[ONE_ROWS];
#pragma unroll
  for (int r = 0; r < ONE_ROWS; ++r) acc[r] = 0.0f;
#pragma unroll 1
  for (int f = tid; f < all; f += 256) {
    const int j = f / chunks, c = 16 * (f - j * chunks), e = a.ids[j];
    float p = a.weights[j];
    const int64_t at = (int64_t)j * a.inter + c;
    const u4 hi[2] = {reinterpret_cast<const u4 *>(a.hi + at)[0], reinterpret_cast<const u4 *>(a.hi + at)[1]};
    const u4 lo[2] = {reinterpret_cast<const u4 *>(a.lo + at)[0], reinterpret_cast<const u4 *>(a.lo + at)[1]};
    const uint8_t *from = a.down + (((int64_t)e * a.hidden + h0) * a.inter + c) * ES;
    u4 w[ONE_ROWS][N];
#pragma unroll
    for (int r = 0; r < ONE_ROWS; ++r)
#pragma unroll
      for (int b = 0; b < N; ++b) w[r][b] = reinterpret_cast<const u4 *>(from + (int64_t)r * a.inter * ES)[b];
    if constexpr (W8) p *= a.down_scales[(e * sblocks + (c >> 7)) * slds + (h0 >> 7)];
    float x[16], l[16];
    floats16<H, false>(hi, x);
    floats16<H, false>(lo, l);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __builtin_fmaf(l[i], 1.0f / Num<H>::LOW, x[i]);      // exact: lo ends where the float that both were cut from did
#pragma unroll
    for (int r = 0; r < ONE_ROWS; ++r) {
      float y[16], d = 0.0f;
      floats16<H, W8>(w[r], y);
#pragma unroll
      for (int i = 0; i < 16; ++i) d = __builtin_fmaf(y[i], x[i], d);
      acc[r] = __builtin_fmaf(p, d, acc[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < ONE_ROWS; ++r) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) acc[r] += __shfl_xor(acc[r], o);
    if ((tid & 63) == 0) part[tid >> 6][r] = acc[r];
  }
  __syncthreads();
  if (tid < ONE_ROWS)
    a.y[h0 + tid] = __builtin_bit_cast(uint16_t, (H)(part[0][tid] + part[1][tid] + part[2][tid] + part[3][tid]));
}

template <typename H> __global__ __launch_bounds__(256) void combine_kernel(MoeArgs a) {
  const int h = blockIdx.x * 256 + threadIdx.x;
  if (h < a.hidden) add_parts<H, false>(a, blockIdx.y, h);
}

template <typename H, bool W8> void launch(MoeArgs &a, hipStream_t st) {
  // Sorting takes the router 2 - 3 us; without it every workgroup of an expert
  // spends a little.  4 tokens, 4 of 32 experts of 1024 x 512: 21.2 us without,
  // 23.8 sorted; 16 tokens 29.6 and 32.0; 8 tokens in e4m3 21.4 and 23.1; 10 tokens,
  // 8 of 96, 53.1 and 50.0; 13 tokens, 6 of 96 of 2064 x 1168, 102.3 and 99.3.
  const int slots = std::min(a.tokens * a.topk, a.experts);
  a.sorted = a.tokens > 1 && (a.tokens * a.topk > FEW || slots * (a.inter / 16) >= 2048);
  if (singly(a.tokens, a.experts)) router_one_kernel<H><<<dim3((a.experts + 3) / 4, a.tokens), 256, 0, st>>>(a);
  else router_kernel<H><<<dim3((a.experts + 15) / 16, (a.tokens + RT - 1) / RT, a.splits), 64 * RW, 0, st>>>(a);
  if (a.tokens == 1) {
    gate_up_one_kernel<H, W8><<<dim3(a.inter / (4 * ONE_PAIRS), a.topk), 256, 0, st>>>(a);
    down_one_kernel<H, W8><<<dim3(a.hidden / ONE_ROWS), 256, 0, st>>>(a);
    return;
  }
  const bool sorted = a.sorted != 0;
  const dim3 gate(a.inter / 16, slots);
  if (sorted) gate_up_kernel<H, W8, true><<<gate, 64 * WV, 0, st>>>(a);
  else gate_up_kernel<H, W8, false><<<gate, 64 * WV, 0, st>>>(a);
  if (slots * (a.hidden / 32) < 200) {
    const dim3 rows(a.hidden / 16, slots);
    if (sorted) down_kernel<H, W8, 1, true><<<rows, 64 * WV, 0, st>>>(a);
    else down_kernel<H, W8, 1, false><<<rows, 64 * WV, 0, st>>>(a);
    return;
  }
  const dim3 rows((a.hidden + 31) / 32, slots);
  if (sorted) down_kernel<H, W8, 2, true><<<rows, 64 * WV, 0, st>>>(a);
  else down_kernel<H, W8, 2, false><<<rows, 64 * WV, 0, st>>>(a);
  combine_kernel<H><<<dim3((a.hidden + 255) / 256, a.tokens), 256, 0, st>>>(a);
}

__global__ __launch_bounds__(256) void clear_kernel(int32_t *p, int n) {
  for (int i = threadIdx.x; i < n; i += 256) p[i] = 0;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

tlr_status check_layer(const tlr_moe_layer *l) {
  if (!l) return fail(TLR_ERR_INVALID_ARG, "moe: null layer");
  if (l->dt == TLR_F32 || l->dt == TLR_F64) return fail(TLR_ERR_UNSUPPORTED, "moe: x and y are TLR_F16 or TLR_BF16");
  if (l->dt != TLR_F16 && l->dt != TLR_BF16) return fail(TLR_ERR_INVALID_ARG, "moe: bad dtype");
  if (l->wdt != l->dt && l->wdt != TLR_E4M3) return fail(TLR_ERR_UNSUPPORTED, "moe: weights are of x's type or TLR_E4M3");
  if (l->hidden < 16 || l->inter < 16 || l->hidden % 16 || l->inter % 16 || l->hidden > 65536 || l->inter > 65536)
    return fail(TLR_ERR_INVALID_ARG, "moe: hidden and inter are multiples of 16, at most 65536");
  if (l->experts < 1 || l->experts > MAX_EXPERTS || l->topk < 1 || l->topk > MAX_TOPK || l->topk > l->experts)
    return fail(TLR_ERR_INVALID_ARG, "moe: experts or topk out of range");
  if ((l->normalize != 0 && l->normalize != 1) || l->reserved != 0) return fail(TLR_ERR_INVALID_ARG, "moe: normalize is 0 or 1, reserved 0");
  return TLR_OK;
}

// Workspace of `tokens` tokens; offsets of its parts.
struct Parts {
  size_t arrived, units, unit, order, logits, hi, lo, part, total;
};
size_t counters(const tlr_moe_layer *l) { return BLOCKS + (size_t)l->hidden / 16; }
// Workgroups that share a router tile's columns: one group of 32 a wave.
int splits_of(const tlr_moe_layer *l, int64_t tokens) {
  return singly(tokens, l->experts) ? 1 : std::min(MAX_SPLITS, (l->hidden + 32 * RW - 1) / (32 * RW));
}
Parts parts_of(const tlr_moe_layer *l, int64_t tokens) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Parts p;
  const size_t n = (size_t)tokens * l->topk;
  p.arrived = 0;
  p.units = p.arrived + counters(l) * 4;
  p.unit = up(p.units + 4);
  p.order = p.unit + sizeof(int4) * MAX_EXPERTS;
  p.logits = p.order + up(n * 4);
  p.hi = p.logits + up((size_t)splits_of(l, tokens) * tokens * l->experts * 8);
  p.lo = p.hi + up(n * l->inter * 2);
  p.part = p.lo + up(n * l->inter * 2);
  p.total = p.part + up(n * l->hidden * 4);
  return p;
}

}  // namespace

tlr_status moe_workspace(const tlr_moe_layer *layer, int32_t max_tokens, size_t *bytes) {
  if (!bytes) return fail(TLR_ERR_INVALID_ARG, "moe_workspace_bytes: null output");
  const tlr_status st = check_layer(layer);
  if (st != TLR_OK) return st;
  if (max_tokens < 0 || max_tokens > MAX_TOKENS) return fail(TLR_ERR_INVALID_ARG, "moe_workspace_bytes: 0 to 256 tokens");
  *bytes = parts_of(layer, max_tokens).total;
  return TLR_OK;
}

tlr_status moe_init(const tlr_moe_layer *layer, void *ws, size_t ws_bytes, void *stream) {
  const tlr_status st = check_layer(layer);
  if (st != TLR_OK) return st;
  if (!ws || !aligned(ws, 256)) return fail(TLR_ERR_INVALID_ARG, "moe_init: null or misaligned workspace");
  if (ws_bytes < parts_of(layer, 0).total) return fail(TLR_ERR_WORKSPACE, "moe_init: workspace too small");
  clear_kernel<<<1, 256, 0, static_cast<hipStream_t>(stream)>>>(static_cast<int32_t *>(ws), (int)counters(layer));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TLR_ERR_HIP, std::string("moe_init: ") + hipGetErrorString(e));
  return TLR_OK;
}

tlr_status moe(const tlr_moe_layer *l, int32_t tokens, const void *X, int64_t ldx, void *Y, int64_t ldy,
               int32_t *ids, float *weights, void *ws, size_t ws_bytes, void *stream) {
  const tlr_status st = check_layer(l);
  if (st != TLR_OK) return st;
  if (tokens < 0 || tokens > MAX_TOKENS) return fail(TLR_ERR_INVALID_ARG, "moe: 0 to 256 tokens");
  if (tokens == 0) return TLR_OK;
  if (!l->router || !l->gate_up || !l->down || !X || !Y || !ids || !weights || !ws)
    return fail(TLR_ERR_INVALID_ARG, "moe: null buffer");
  if (!aligned(l->router, 16) || !aligned(l->gate_up, 16) || !aligned(l->down, 16) || !aligned(X, 16) || ldx % 8 ||
      !aligned(Y, 2) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(ws, 256))
    return fail(TLR_ERR_INVALID_ARG, "moe: misaligned buffer");
  if (ldx < l->hidden || ldy < l->hidden) return fail(TLR_ERR_INVALID_ARG, "moe: leading dimension too small");
  const bool w8 = l->wdt == TLR_E4M3;
  if (w8 && (!l->gate_up_scales || !l->down_scales || !aligned(l->gate_up_scales, 4) || !aligned(l->down_scales, 4)))
    return fail(TLR_ERR_INVALID_ARG, "moe: null or misaligned scales");
  const Parts p = parts_of(l, tokens);
  if (ws_bytes < p.total) return fail(TLR_ERR_WORKSPACE, "moe: workspace too small");
  uint8_t *b = static_cast<uint8_t *>(ws);
  MoeArgs a{tokens, l->hidden, l->inter, l->experts, l->topk, l->normalize,
            static_cast<const uint16_t *>(X), ldx, static_cast<uint16_t *>(Y), ldy,
            static_cast<const uint16_t *>(l->router), static_cast<const uint8_t *>(l->gate_up),
            static_cast<const uint8_t *>(l->down), l->gate_up_scales, l->down_scales, ids, weights,
            reinterpret_cast<int32_t *>(b + p.arrived), reinterpret_cast<int32_t *>(b + p.units),
            reinterpret_cast<int4 *>(b + p.unit), reinterpret_cast<int32_t *>(b + p.order),
            reinterpret_cast<double *>(b + p.logits), splits_of(l, tokens), 0, reinterpret_cast<uint16_t *>(b + p.hi),
            reinterpret_cast<uint16_t *>(b + p.lo), reinterpret_cast<float *>(b + p.part)};
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (l->dt == TLR_F16) w8 ? launch<_Float16, true>(a, hs) : launch<_Float16, false>(a, hs);
  else w8 ? launch<__bf16, true>(a, hs) : launch<__bf16, false>(a, hs);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TLR_ERR_HIP, std::string("moe: ") + hipGetErrorString(e));
  return TLR_OK;
}

}  // namespace tlr
