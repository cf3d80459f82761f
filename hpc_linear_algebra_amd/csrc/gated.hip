// The gated activation y = silu(g) u with an 8-bit checkpoint for its backward
// pass, for gfx950.
//
// A row of X holds `inter` entries of g and as many of u.  For the backward pass
// the row is kept as 8-bit integers with a float scale for every 128 entries of
// each half; the gradient is taken at the values that these stand for:
//   dg = dy u s (1 + g (1 - s)),  du = dy g s,  s = 1 / (1 + exp(-g)).
// Every entry is read and written once, so that both directions are bound by HBM
// (16384 x 4096 bf16: forward 99 us, backward 93, 0.54 GB each).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "int8.h"
#include "tlr_ops.h"

namespace tlr {

namespace {

// 1 / (1 + exp(-g)) and 1 minus it, both to float precision where they are normal
// floats: the exponential of a negative number never overflows, and neither result
// comes from a difference.  The hardware's exponential has no results below 2^-126
// but 0, so the smaller of the two is 0 from |g| = 87.34 on.  Beside the larger one
// that is nothing; the sigmoid of a far negative gate is replaced (below).
struct Sigmoid {
  float s, rest;
};
__device__ __forceinline__ Sigmoid sigmoid(float g) {
  // exp(-|g|) = 2^t; t's rounding is carried along, which keeps full precision
  // where t is large.  Past -150 it is 0 anyway (and an infinity gives no difference of two)
  const float a = fmaxf(-__builtin_fabsf(g), -150.0f), log2e = 0x1.715476p0f, low = 0x1.4ae0cp-26f;
  const float t = a * log2e, c = __builtin_fmaf(a, low, __builtin_fmaf(a, log2e, -t));
  const float p = __builtin_amdgcn_exp2f(t), e = __builtin_fmaf(p * 0x1.62e43p-1f, c, p);
  const float r = __builtin_amdgcn_rcpf(1.0f + e), n = e * r;
  return g < 0.0f ? Sigmoid{n, r} : Sigmoid{r, n};
}

// Gates whose sigmoid is exp(g) to more than a double's precision and near or below the
// smallest normal float.  Times large factors it may be an ordinary number (-88 and
// 1e38: -53), so that products with it are in doubles.  An infinite one stays: -inf times 0.
// Halves are 65504 at most: three of them times exp(-86) are nothing.
constexpr float FAR = 86.0f;
template <typename T> constexpr bool WIDE_RANGE = !std::is_same<T, _Float16>::value;
__device__ __forceinline__ bool is_far(float g) { return g < -FAR && g >= -0x1.fffffep127f; }
__device__ __forceinline__ double far_sigmoid(float g) {
  const float a = fmaxf(g, -700.0f), log2e = 0x1.715476p0f, low = 0x1.4ae0cp-26f;       // 2^-1010: nothing times any floats
  const float n = __builtin_rintf(a * log2e);
  return ldexp((double)__builtin_amdgcn_exp2f(__builtin_fmaf(a, low, __builtin_fmaf(a, log2e, -n))), (int)n);
}

struct GatedArgs {
  const void *x, *dy;
  void *y, *dx;
  int64_t ldx, lddy, ldy, lddx, ldq, lds;
  uint8_t *codes;
  float *scales;
  uint32_t tasks, nq;       // 128 entries of both halves each; those of a row
  int32_t inter;
};

// 16 lanes take 128 entries of g and those of u, 8 each a lane.
template <typename T, bool KEEP> __global__ __launch_bounds__(256) void gated_kernel(GatedArgs a) {
  const int c = threadIdx.x & 15;
  for (uint32_t task = blockIdx.x * 16 + (threadIdx.x >> 4); task < a.tasks; task += gridDim.x * 16) {
    const int64_t row = task / a.nq;
    const int q = (int)(task % a.nq), col = q * QB + 8 * c, left = a.inter - col;
    const T *x = static_cast<const T *>(a.x) + row * a.ldx + col;
    Eight<T> xg, xu;
    if (left >= 8) {
      xg.template load<true>(x, left);
      xu.template load<true>(x + a.inter, left);
    } else {
      xg.template load<false>(x, left);
      xu.template load<false>(x + a.inter, left);
    }
    float g[8], u[8], y[8];
    xg.get(g);
    xu.get(u);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = g[e] * sigmoid(g[e]).s * u[e];
    uint32_t top[2] = {0, 0};           // largest magnitudes of the lane's g and u
#pragma unroll
    for (int e = 0; e < 8; ++e) top[0] = max(top[0], mag(g[e]));
    if (WIDE_RANGE<T> && top[0] > mag(FAR))
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (is_far(g[e])) y[e] = (float)(g[e] * far_sigmoid(g[e]) * u[e]);
    put8(static_cast<T *>(a.y) + row * a.ldy + col, left, y);
    if constexpr (KEEP) {
      const int64_t at = 2 * row;
#pragma unroll
      for (int e = 0; e < 8; ++e) top[1] = max(top[1], mag(u[e]));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float(&v)[8] = h ? u : g;
        const float s = int8_scale(max16(top[h]));
        if (c == 0) a.scales[(at + h) * a.lds + q] = s;
        if (col < ((a.inter + 15) & ~15)) *reinterpret_cast<u2 *>(a.codes + (at + h) * a.ldq + col) = int8_codes8(v, s, 1.0f / s);
      }
    }
  }
}

__device__ __forceinline__ float code(u2 w, int e) { return (float)(int8_t)(w[e >> 2] >> (8 * (e & 3))); }

template <typename T> __global__ __launch_bounds__(256) void gated_grad_kernel(GatedArgs a) {
  const int c = threadIdx.x & 15;
  for (uint32_t task = blockIdx.x * 16 + (threadIdx.x >> 4); task < a.tasks; task += gridDim.x * 16) {
    const int64_t row = task / a.nq;
    const int q = (int)(task % a.nq), col = q * QB + 8 * c, left = a.inter - col;
    if (left <= 0) continue;
    const int64_t at = 2 * row;
    const u2 cg = *reinterpret_cast<const u2 *>(a.codes + at * a.ldq + col), cu = *reinterpret_cast<const u2 *>(a.codes + (at + 1) * a.ldq + col);
    const float sg = a.scales[at * a.lds + q], su = a.scales[(at + 1) * a.lds + q];
    float dy[8], dg[8], du[8];
    get8(static_cast<const T *>(a.dy) + row * a.lddy + col, left, dy);
    uint32_t least = 0xffffffffu;       // of the dy, without their signs; zeros are above all others
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float g = sg * code(cg, e), u = su * code(cu, e);
      const Sigmoid s = sigmoid(g);
      const float d = dy[e] * s.s;
      dg[e] = d * u * __builtin_fmaf(g, s.rest, 1.0f);
      du[e] = d * g;
      least = min(least, 2 * __builtin_bit_cast(uint32_t, dy[e]) - 1);
    }
    // Where dy s falls below the normal floats, u or g may bring the product back: such ones again, in doubles.  There are none
    // in a block whose gates are 32 at most (the sigmoid 2^-47 at least) where dy is 0 or 2^-79 at least.
    if (WIDE_RANGE<T> && (sg > 32.0f / 128 || least < 2 * __builtin_bit_cast(uint32_t, 0x1p-79f) - 1))
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = sg * code(cg, e), u = su * code(cu, e);
        const Sigmoid s = sigmoid(g);
        const bool far = is_far(g);
        if (dy[e] != 0.0f && (far || __builtin_fabsf(dy[e] * s.s) < 0x1p-126f)) {
          const double d = dy[e] * (far ? far_sigmoid(g) : s.s);
          dg[e] = (float)(d * u * (far ? 1.0f + g : __builtin_fmaf(g, s.rest, 1.0f)));
          du[e] = (float)(d * g);
        }
      }
    T *dx = static_cast<T *>(a.dx) + row * a.lddx + col;
    put8(dx, left, dg);
    put8(dx + a.inter, left, du);
  }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t SIZE_LIM = 0x7fffffff;

// What both directions check; sets the sizes.
tlr_status check(const char *name, tlr_dtype dt, int64_t rows, int64_t inter, const void *codes, int64_t ldq, const float *scales,
                 int64_t lds, GatedArgs *a) {
  const std::string w = std::string(name) + ": ";
  if (dt == TLR_F64) return fail(TLR_ERR_UNSUPPORTED, w + "TLR_F64 is not provided");
  if (dt != TLR_F32 && dt != TLR_F16 && dt != TLR_BF16) return fail(TLR_ERR_INVALID_ARG, w + "bad dtype");
  if (rows < 0 || inter < 0 || rows > SIZE_LIM || inter > SIZE_LIM / 2) return fail(TLR_ERR_INVALID_ARG, w + "size out of range");
  const int64_t nq = (inter + QB - 1) / QB;
  if (rows * nq > SIZE_LIM) return fail(TLR_ERR_INVALID_ARG, w + "too many entries");
  if (codes) {
    if (!aligned(codes, 16) || ldq % 16 != 0 || ldq < inter) return fail(TLR_ERR_INVALID_ARG, w + "codes: rows of at least inter bytes, 16-byte aligned, are needed");
    if (!scales || !aligned(scales, 4) || lds < nq) return fail(TLR_ERR_INVALID_ARG, w + "scales: null, misaligned, or rows too short");
  }
  a->codes = static_cast<uint8_t *>(const_cast<void *>(codes));
  a->scales = const_cast<float *>(scales);
  a->ldq = ldq;
  a->lds = lds;
  a->inter = (int32_t)inter;
  a->nq = (uint32_t)nq;
  a->tasks = (uint32_t)(rows * nq);
  return TLR_OK;
}

unsigned grid_of(uint32_t tasks) { return std::min<uint32_t>(tasks / 16 + (tasks % 16 != 0), 1 << 20); }

tlr_status launched(const char *what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TLR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
  return TLR_OK;
}

template <typename T> void forward(const GatedArgs &a, hipStream_t st) {
  if (a.codes) gated_kernel<T, true><<<grid_of(a.tasks), 256, 0, st>>>(a);
  else gated_kernel<T, false><<<grid_of(a.tasks), 256, 0, st>>>(a);
}

}  // namespace

tlr_status gated(tlr_dtype dt, int64_t rows, int64_t inter, const void *X, int64_t ldx, void *Y, int64_t ldy, void *codes,
                 int64_t ldq, float *scales, int64_t lds, void *stream) {
  GatedArgs a{};
  const tlr_status bad = check("gated", dt, rows, inter, codes, ldq, scales, lds, &a);
  if (bad != TLR_OK) return bad;
  if (ldx < 2 * inter || ldy < inter) return fail(TLR_ERR_INVALID_ARG, "gated: leading dimension too small");
  if (rows == 0 || inter == 0) return TLR_OK;
  const int es = dt == TLR_F32 ? 4 : 2;
  if (!X || !Y || !aligned(X, es) || !aligned(Y, es)) return fail(TLR_ERR_INVALID_ARG, "gated: null or misaligned X or Y");
  a.x = X;
  a.ldx = ldx;
  a.y = Y;
  a.ldy = ldy;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (dt == TLR_F32) forward<float>(a, st);
  else if (dt == TLR_F16) forward<_Float16>(a, st);
  else forward<__bf16>(a, st);
  return launched("gated");
}

tlr_status gated_grad(tlr_dtype dt, int64_t rows, int64_t inter, const void *dY, int64_t lddy, const void *codes, int64_t ldq,
                      const float *scales, int64_t lds, void *dX, int64_t lddx, void *stream) {
  GatedArgs a{};
  const tlr_status bad = check("gated_grad", dt, rows, inter, codes, ldq, scales, lds, &a);
  if (bad != TLR_OK) return bad;
  if (lddy < inter || lddx < 2 * inter) return fail(TLR_ERR_INVALID_ARG, "gated_grad: leading dimension too small");
  if (rows == 0 || inter == 0) return TLR_OK;
  const int es = dt == TLR_F32 ? 4 : 2;
  if (!codes) return fail(TLR_ERR_INVALID_ARG, "gated_grad: null codes");
  if (!dY || !dX || !aligned(dY, es) || !aligned(dX, es)) return fail(TLR_ERR_INVALID_ARG, "gated_grad: null or misaligned dY or dX");
  a.dy = dY;
  a.lddy = lddy;
  a.dx = dX;
  a.lddx = lddx;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const unsigned grid = grid_of(a.tasks);
  if (dt == TLR_F32) gated_grad_kernel<float><<<grid, 256, 0, st>>>(a);
  else if (dt == TLR_F16) gated_grad_kernel<_Float16><<<grid, 256, 0, st>>>(a);
  else gated_grad_kernel<__bf16><<<grid, 256, 0, st>>>(a);
  return launched("gated_grad");
}

}  // namespace tlr
