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
// their scale is applied to each block's float sum.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <string>

#include "tlr_ops.h"

namespace tlr {

namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int MAX_TOKENS = 256, MAX_EXPERTS = 512, MAX_TOPK = 16;
constexpr int MAX_LIST = MAX_TOKENS;      // assignments of one expert: at most one per token

// The 16-bit type of x, y and the products.
template <typename H> struct Num;
template <> struct Num<_Float16> {
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
  double *logits;           // tokens x experts
  uint16_t *hi, *lo;        // tokens*topk x inter: silu(g) u as hi + lo
  float *part;              // tokens*topk x hidden: the experts' outputs
  int32_t slots;            // grid rows of the expert launches
};

// Eight 16-bit entries as floats.
template <typename H> __device__ __forceinline__ void unpack8(u4 w, float (&v)[8]) {
  typedef typename Num<H>::v8 v8;
  const v8 h = __builtin_bit_cast(v8, w);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)h[e];
}

constexpr int RT = 8;       // tokens of a router workgroup

// Logits: one wave per expert and RT tokens.  A product of two 16-bit numbers
// is an exact float; the sums run in double.
template <typename H> __global__ __launch_bounds__(256) void router_kernel(MoeArgs a) {
  const int lane = threadIdx.x & 63, e = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int t0 = blockIdx.y * RT;
  if (e >= a.experts) return;
  const uint16_t *w = a.router + (int64_t)e * a.hidden;
  double acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = 0.0;
  for (int c = 8 * lane; c < a.hidden; c += 512) {
    float wf[8];
    unpack8<H>(*reinterpret_cast<const u4 *>(w + c), wf);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      if (t0 + i >= a.tokens) break;
      float xf[8];
      unpack8<H>(*reinterpret_cast<const u4 *>(a.x + (t0 + i) * a.ldx + c), xf);
#pragma unroll
      for (int v = 0; v < 8; ++v) acc[i] += (double)(wf[v] * xf[v]);
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    if (t0 + i >= a.tokens) break;
    double s = acc[i];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if (lane == 0) a.logits[(int64_t)(t0 + i) * a.experts + e] = s;
  }
}

// A double as a number whose order is the logits' order, NaN on top.
__device__ __forceinline__ uint64_t sort_key(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  if (x != x) return ~0ull;
  const uint64_t z = x == 0.0 ? 0ull : b;      // -0 and 0 tie
  return (z >> 63) ? ~z : z | 0x8000000000000000ull;
}

// One workgroup per token: an expert's place is the number of experts before
// it (larger logit, or the same and a lower index); the first topk are chosen.
__global__ __launch_bounds__(256) void select_kernel(MoeArgs a) {
  __shared__ uint64_t key[MAX_EXPERTS];
  __shared__ float zs[4], chosen[MAX_TOPK];
  __shared__ double best;
  const int tid = threadIdx.x, t = blockIdx.x;
  const double *l = a.logits + (int64_t)t * a.experts;
  for (int e = tid; e < a.experts; e += 256) key[e] = sort_key(l[e]);
  __syncthreads();
  int place[MAX_EXPERTS / 256];
#pragma unroll
  for (int i = 0; i < MAX_EXPERTS / 256; ++i) {
    const int e = tid + 256 * i;
    place[i] = a.experts;
    if (e >= a.experts) continue;
    const uint64_t mine = key[e];
    int n = 0;
    for (int f = 0; f < a.experts; ++f) n += (key[f] > mine || (key[f] == mine && f < e)) ? 1 : 0;
    place[i] = n;
    if (n == 0) best = l[e];
  }
  __syncthreads();
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < MAX_EXPERTS / 256; ++i) {
    const int e = tid + 256 * i;
    if (e >= a.experts) continue;
    const float p = expf((float)(l[e] - best));
    z += p;
    if (place[i] < a.topk) {
      chosen[place[i]] = p;
      a.ids[t * a.topk + place[i]] = e;
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) z += __shfl_xor(z, o);
  if ((tid & 63) == 0) zs[tid >> 6] = z;
  __syncthreads();
  if (tid < a.topk) {
    float sum = zs[0] + zs[1] + zs[2] + zs[3];
    if (a.normalize) {
      sum = 0.0f;
      for (int j = 0; j < a.topk; ++j) sum += chosen[j];
    }
    a.weights[t * a.topk + tid] = chosen[tid] / sum;
  }
}

// The expert of this workgroup (grid row) and the list of its assignments
// (token * topk + choice) in increasing order; false when it has none.  With
// fewer assignments than experts a grid row is an assignment, which stands for
// its expert when no earlier one has the same; else a grid row is an expert.
__device__ __forceinline__ bool my_expert(const MoeArgs &a, int row, int *list, int *scratch, int &e, int &count) {
  const int n = a.tokens * a.topk, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  e = a.slots == a.experts ? row : a.ids[row];
  const bool by_row = a.slots != a.experts;
  count = 0;
  bool first = true;
  for (int i0 = 0; i0 < n; i0 += 256) {
    const int i = i0 + tid;
    const bool hit = i < n && a.ids[i] == e;
    const uint64_t b = __ballot(hit);
    if (lane == 0) scratch[wave] = __popcll(b);
    __syncthreads();
    int before = count;
    for (int w = 0; w < wave; ++w) before += scratch[w];
    if (hit) list[before + __popcll(b & ((1ull << lane) - 1))] = i;
    count += scratch[0] + scratch[1] + scratch[2] + scratch[3];
    __syncthreads();
  }
  if (by_row) first = count > 0 && list[0] == row;
  return first && count > 0;
}

// RTILE row tiles (16 rows each) of an expert's matrix against NJ tiles of 16
// token columns over this wave's part of the contraction: lane (r, q) =
// (lane % 16, lane / 16) supplies columns k0 + 16 q .. + 15 of weight row r and
// of token column r for each group of 64 (two matrix instructions).  TWO: the
// tokens come as a sum of two matrices.
template <typename H, bool W8, int NJ, int RTILE, bool TWO>
__device__ __forceinline__ void multiply(f4 (&acc)[RTILE][NJ], const uint8_t *const (&w)[RTILE],
                                         const float *const (&ws)[RTILE], int64_t wlds, const uint16_t *const (&x)[NJ],
                                         const uint16_t *const (&x2)[NJ], int K, int wave, int waves, int q) {
  for (int g = wave; g * 64 < K; g += waves) {
    const int k = g * 64 + 16 * q;
    const bool in = k < K;
    const u4 zero = u4{0, 0, 0, 0};
    u4 wf[RTILE][2];
#pragma unroll
    for (int i = 0; i < RTILE; ++i) {
      if constexpr (W8) {
        const u4 c = in ? *reinterpret_cast<const u4 *>(w[i] + k) : zero;
#pragma unroll
        for (int p = 0; p < 2; ++p)
          wf[i][p] = u4{Num<H>::template widen<false>(c[2 * p]), Num<H>::template widen<true>(c[2 * p]),
                        Num<H>::template widen<false>(c[2 * p + 1]), Num<H>::template widen<true>(c[2 * p + 1])};
      } else {
        const u4 *p = reinterpret_cast<const u4 *>(w[i] + 2 * k);
        wf[i][0] = in ? p[0] : zero;
        wf[i][1] = in ? p[1] : zero;
      }
    }
    float s[RTILE];
    if constexpr (W8)
#pragma unroll
      for (int i = 0; i < RTILE; ++i) s[i] = ws[i][(g >> 1) * wlds];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const u4 *p = reinterpret_cast<const u4 *>(x[j] + k);
      const u4 b0 = in ? p[0] : zero, b1 = in ? p[1] : zero;
      u4 c0 = zero, c1 = zero;
      if constexpr (TWO) {
        const u4 *p2 = reinterpret_cast<const u4 *>(x2[j] + k);
        c0 = in ? p2[0] : zero;
        c1 = in ? p2[1] : zero;
      }
#pragma unroll
      for (int i = 0; i < RTILE; ++i) {
        f4 d = W8 ? f4{0, 0, 0, 0} : acc[i][j];
        d = Num<H>::mma(wf[i][0], b0, d);
        d = Num<H>::mma(wf[i][1], b1, d);
        if constexpr (TWO) {
          d = Num<H>::mma(wf[i][0], c0, d);
          d = Num<H>::mma(wf[i][1], c1, d);
        }
        if constexpr (W8) {
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(s[i], d[v], acc[i][j][v]);
        } else {
          acc[i][j] = d;
        }
      }
    }
  }
}

constexpr int WV = 4;       // waves of an expert workgroup

// silu(G x) * (U x) for 16 of an expert's inter rows and all of its tokens.
template <typename H, bool W8> __global__ __launch_bounds__(64 * WV) void gate_up_kernel(MoeArgs a) {
  __shared__ int list[MAX_LIST], scratch[WV];
  __shared__ float part[WV][2][4][64];
  int e, count;
  if (!my_expert(a, blockIdx.y, list, scratch, e, count)) return;
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
  for (int n0 = 0; n0 < count; n0 += 16) {
    f4 acc[2][1] = {{f4{0, 0, 0, 0}}, {f4{0, 0, 0, 0}}};
    const uint16_t *x[1] = {a.x + (list[min(n0 + r, count - 1)] / a.topk) * a.ldx};
    multiply<H, W8, 1, 2, false>(acc, w, ws, wlds, x, x, a.hidden, wave, WV, q);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[wave][i][v][lane] = acc[i][0][v];
    __syncthreads();
    // thread (row i, column c) of the 16 x 16 block
    const int i = tid & 15, c = tid >> 4, at = (i >> 2) * 16 + c;
    if (n0 + c < count) {
      float g = 0.0f, u = 0.0f;
#pragma unroll
      for (int k = 0; k < WV; ++k) {
        g += part[k][0][i & 3][at];
        u += part[k][1][i & 3][at];
      }
      const float v = g / (1.0f + expf(-g)) * u;
      const H hi = (H)v;
      const float rest = v - (float)hi;
      const H lo = (H)(__builtin_isfinite(rest) ? rest : 0.0f);     // beyond the type's range hi is infinite
      const int64_t o = (int64_t)list[n0 + c] * a.inter + i0 + i;
      a.hi[o] = __builtin_bit_cast(uint16_t, hi);
      a.lo[o] = __builtin_bit_cast(uint16_t, lo);
    }
  }
}

// 16 rows of an expert's down product for all of its tokens.
template <typename H, bool W8> __global__ __launch_bounds__(64 * WV) void down_kernel(MoeArgs a) {
  __shared__ int list[MAX_LIST], scratch[WV];
  __shared__ float part[WV][4][64];
  int e, count;
  if (!my_expert(a, blockIdx.y, list, scratch, e, count)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4, h0 = blockIdx.x * 16;
  const int64_t es = W8 ? 1 : 2;
  const int64_t wlds = (a.hidden + 127) / 128;
  const uint8_t *w[1] = {a.down + ((int64_t)e * a.hidden + h0 + r) * a.inter * es};
  const float *ws[1] = {nullptr};
  if constexpr (W8) ws[0] = a.down_scales + (int64_t)e * ((a.inter + 127) / 128) * wlds + (h0 >> 7);
  for (int n0 = 0; n0 < count; n0 += 16) {
    f4 acc[1][1] = {{f4{0, 0, 0, 0}}};
    const int64_t at = (int64_t)list[min(n0 + r, count - 1)] * a.inter;
    const uint16_t *x[1] = {a.hi + at}, *x2[1] = {a.lo + at};
    multiply<H, W8, 1, 1, true>(acc, w, ws, wlds, x, x2, a.inter, wave, WV, q);
    __syncthreads();
#pragma unroll
    for (int v = 0; v < 4; ++v) part[wave][v][lane] = acc[0][0][v];
    __syncthreads();
    const int i = tid & 15, c = tid >> 4, o = (i >> 2) * 16 + c;
    if (n0 + c < count) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < WV; ++k) s += part[k][i & 3][o];
      a.part[(int64_t)list[n0 + c] * a.hidden + h0 + i] = s;
    }
  }
}

template <typename H> __global__ __launch_bounds__(256) void combine_kernel(MoeArgs a) {
  const int h = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (h >= a.hidden) return;
  float s = 0.0f;
  for (int j = 0; j < a.topk; ++j) s += a.weights[t * a.topk + j] * a.part[(int64_t)(t * a.topk + j) * a.hidden + h];
  a.y[t * a.ldy + h] = __builtin_bit_cast(uint16_t, (H)s);
}

template <typename H, bool W8> void launch(const MoeArgs &a, hipStream_t st) {
  router_kernel<H><<<dim3((a.experts + 3) / 4, (a.tokens + RT - 1) / RT), 256, 0, st>>>(a);
  select_kernel<<<dim3(a.tokens), 256, 0, st>>>(a);
  gate_up_kernel<H, W8><<<dim3(a.inter / 16, a.slots), 64 * WV, 0, st>>>(a);
  down_kernel<H, W8><<<dim3(a.hidden / 16, a.slots), 64 * WV, 0, st>>>(a);
  combine_kernel<H><<<dim3((a.hidden + 255) / 256, a.tokens), 256, 0, st>>>(a);
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
  size_t logits, hi, lo, part, total;
};
Parts parts_of(const tlr_moe_layer *l, int64_t tokens) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  Parts p;
  const size_t n = (size_t)tokens * l->topk;
  p.logits = 0;
  p.hi = p.logits + up((size_t)tokens * l->experts * 8);
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
  (void)ws, (void)ws_bytes, (void)stream;
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
            reinterpret_cast<double *>(b + p.logits), reinterpret_cast<uint16_t *>(b + p.hi),
            reinterpret_cast<uint16_t *>(b + p.lo), reinterpret_cast<float *>(b + p.part),
            std::min(tokens * l->topk, l->experts)};
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (l->dt == TLR_F16) w8 ? launch<_Float16, true>(a, hs) : launch<_Float16, false>(a, hs);
  else w8 ? launch<__bf16, true>(a, hs) : launch<__bf16, false>(a, hs);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TLR_ERR_HIP, std::string("moe: ") + hipGetErrorString(e));
  return TLR_OK;
}

}  // namespace tlr
