// Tokens sorted by expert and back, with weights, and the gradients, for gfx950.
//
// A router gives each token `topk` assignments to experts.  The sort gives each
// assignment a row, so that every expert's rows are consecutive and in the order
// of their tokens (a counting sort; no atomics on results, so the same inputs give
// the same rows).  gather copies a token to its rows, combine adds its rows with
// the router's weights; the gradient of one is the other:
//   gather   xs[p(t,s)] = x[t]                  dx[t] = sum_s dxs[p(t,s)]
//   combine  out[t] = sum_s w[t,s] y[p(t,s)]    dy[p(t,s)] = w[t,s] dout[t],
//                                               dw[t,s] = <dout[t], y[p(t,s)]>
// Assignments to no expert have the rows behind the last expert's: they are filled
// with zeros and never read.  All of it moves each row once, bound by HBM; sums
// are in float, in the order of s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "int8.h"
#include "tlr_ops.h"

namespace tlr {

namespace {

// ---- sort --------------------------------------------------------------------------------------------

constexpr int MOST_EXPERTS = 1024, MOST_TOPK = 64;

struct SortArgs {
  const void *ids;
  int32_t *offsets, *place, *rows;
  int32_t *counts;          // (parts, experts + 1), and a row of totals behind them
  int32_t n, topk, experts, parts;
  int32_t scanned;          // counts: of the parts before, and the totals
};

// The expert of an assignment; `experts` for none.
template <typename ID> __device__ __forceinline__ int expert_of(const SortArgs &a, int i) {
  const ID e = static_cast<const ID *>(a.ids)[i];
  return e >= 0 && e < (ID)a.experts ? (int)e : a.experts;
}

// The lanes whose e (-1: none) is this lane's, by one ballot for each bit.
__device__ __forceinline__ uint64_t same_lanes(int e, int bits) {
  uint64_t same = __ballot(e >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool on = (e >> b) & 1;
    const uint64_t m = __ballot(on);
    same &= on ? m : ~m;
  }
  return same;
}

// How many assignments of its part each expert has: the first lane of an expert adds
// for the others.
template <typename ID, int EACH> __global__ __launch_bounds__(1024) void count_kernel(SortArgs a) {
  __shared__ int32_t hist[MOST_EXPERTS + 1];
  const int lane = threadIdx.x & 63, bits = 32 - __builtin_clz(a.experts);
  int e[EACH];
#pragma unroll
  for (int c = 0; c < EACH; ++c) {
    const int64_t i = ((int64_t)blockIdx.x * EACH + c) * 1024 + threadIdx.x;
    e[c] = i < a.n ? expert_of<ID>(a, (int)i) : -1;
  }
  for (int x = threadIdx.x; x <= a.experts; x += 1024) hist[x] = 0;
  __syncthreads();
#pragma unroll
  for (int c = 0; c < EACH; ++c) {
    const uint64_t same = same_lanes(e[c], bits);
    if (e[c] >= 0 && (same & ((1ull << lane) - 1)) == 0) atomicAdd(&hist[e[c]], __builtin_popcountll(same));
  }
  __syncthreads();
  for (int x = threadIdx.x; x <= a.experts; x += 1024) a.counts[(int64_t)blockIdx.x * (a.experts + 1) + x] = hist[x];
}

// Counts of many parts to those of the parts before each, and the totals: a workgroup
// takes 64 experts, a wave every sixteenth of the parts.
__global__ __launch_bounds__(1024) void scan_kernel(SortArgs a) {
  __shared__ int32_t sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, x = blockIdx.x * 64 + lane, row = a.experts + 1;
  const int each = (a.parts + 15) / 16, from = min(wave * each, a.parts), to = min(from + each, a.parts);
  int sum = 0;
  if (x < row)
#pragma unroll 8
    for (int p = from; p < to; ++p) sum += a.counts[(int64_t)p * row + x];
  sums[wave][lane] = sum;
  __syncthreads();
  if (x >= row) return;
  int before = 0;
  for (int w = 0; w < wave; ++w) before += sums[w][lane];
  for (int p = from; p < to; ++p) {
    const int v = a.counts[(int64_t)p * row + x];
    a.counts[(int64_t)p * row + x] = before;
    before += v;
  }
  if (wave == 15) a.counts[(int64_t)a.parts * row + x] = before;
}

// Rows of a part's assignments, EACH for each of W waves' threads.  A wave takes 64
// consecutive ones at a time: a lane's rank is the number of lanes before it with its
// expert, added to the wave's count so far.  Ranks, counts of the waves before, counts
// of the parts before and the experts' first rows add up to the row.
template <typename ID, int W, int EACH> __global__ __launch_bounds__(64 * W) void sort_kernel(SortArgs a) {
  constexpr int MOST = W == 16 ? MOST_EXPERTS : 64 * W;
  __shared__ int32_t hist[W][MOST + 1];
  __shared__ int32_t sums[W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t first = (int64_t)blockIdx.x * (64 * W * EACH) + wave * 64 * EACH + lane;
  int e[EACH], rank[EACH];
#pragma unroll
  for (int c = 0; c < EACH; ++c) e[c] = first + 64 * c < a.n ? expert_of<ID>(a, (int)(first + 64 * c)) : -1;
  for (int x = lane; x <= a.experts; x += 64) hist[wave][x] = 0;
  const int bits = 32 - __builtin_clz(a.experts);
#pragma unroll
  for (int c = 0; c < EACH; ++c) {
    const uint64_t same = same_lanes(e[c], bits);
    const int before = __builtin_popcountll(same & ((1ull << lane) - 1));
    asm volatile("" ::: "memory");        // the wave's LDS accesses stay in this order
    if (e[c] >= 0) {
      const int so_far = hist[wave][e[c]];
      asm volatile("" ::: "memory");
      rank[c] = so_far + before;
      if (before == 0) hist[wave][e[c]] = so_far + __builtin_popcountll(same);
    }
    asm volatile("" ::: "memory");
  }
  __syncthreads();
  // thread x: expert x (the last column, of no expert, is thread 0's as well)
  auto column = [&](int x, int &before, int &all) {
    before = all = 0;
    int part = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int v = hist[w][x];
      hist[w][x] = part;
      part += v;
    }
    const int32_t *counts = a.counts + x;
    const int64_t row = a.experts + 1;
    if (a.parts == 1) {
      all = part;
    } else if (a.scanned) {
      before = counts[blockIdx.x * row];
      all = counts[a.parts * row];
    } else {
      for (int p0 = 0; p0 < a.parts; p0 += 16) {        // 16 loads in flight
        int v[16];
#pragma unroll
        for (int p = 0; p < 16; ++p) v[p] = counts[min(p0 + p, a.parts - 1) * row];
#pragma unroll
        for (int p = 0; p < 16; ++p) {
          before += p0 + p < (int)blockIdx.x ? v[p] : 0;
          all += p0 + p < a.parts ? v[p] : 0;
        }
      }
    }
  };
  int before = 0, all = 0;
  if (tid < a.experts) column(tid, before, all);
  int scan = all;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(scan, d);
    if (lane >= d) scan += v;
  }
  if (lane == 63) sums[wave] = scan;
  __syncthreads();
  int total = 0, start = scan - all;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < wave) start += sums[w];
    total += sums[w];
  }
  if (tid < a.experts) {
#pragma unroll
    for (int w = 0; w < W; ++w) hist[w][tid] += start + before;
    if (blockIdx.x == 0) a.offsets[tid] = start;
  }
  if (tid == 0) {
    int none_before, none;
    column(a.experts, none_before, none);
#pragma unroll
    for (int w = 0; w < W; ++w) hist[w][a.experts] += total + none_before;
    if (blockIdx.x == 0) a.offsets[a.experts] = total;
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < EACH; ++c)
    if (e[c] >= 0) {
      const int i = (int)(first + 64 * c), p = hist[wave][e[c]] + rank[c];
      a.place[i] = p;
      // always in range, unless ids were written between the launches
      if ((uint32_t)p < (uint32_t)a.n) a.rows[p] = e[c] < a.experts ? i / a.topk : -1;
    }
}

// One workgroup sorts up to ONE assignments; more go in parts of 1024 or, from FINE on, of
// 4096, and beyond SUMMED parts their counts are summed by a launch of its own.
constexpr int64_t ONE = 4096, FINE = 65536, SUMMED = 64;
int64_t part_of(int64_t n) { return n <= FINE ? 1024 : 4096; }
int64_t parts_of(int64_t n) { return n <= ONE ? 1 : (n + part_of(n) - 1) / part_of(n); }

template <typename ID> void sort_launch(const SortArgs &a, hipStream_t st) {
  if (a.parts > 1) {
    const bool fine = a.n <= FINE;
    if (fine) count_kernel<ID, 1><<<a.parts, 1024, 0, st>>>(a);
    else count_kernel<ID, 4><<<a.parts, 1024, 0, st>>>(a);
    if (a.scanned) scan_kernel<<<a.experts / 64 + 1, 1024, 0, st>>>(a);
    if (fine) sort_kernel<ID, 16, 1><<<a.parts, 1024, 0, st>>>(a);
    else sort_kernel<ID, 16, 4><<<a.parts, 1024, 0, st>>>(a);
  } else if (a.n <= 256 && a.experts <= 256) sort_kernel<ID, 4, 1><<<1, 256, 0, st>>>(a);
  else if (a.n <= 1024 && a.experts <= 256) sort_kernel<ID, 4, 4><<<1, 256, 0, st>>>(a);
  else sort_kernel<ID, 16, 4><<<1, 1024, 0, st>>>(a);
}

// ---- rows --------------------------------------------------------------------------------------------

struct RowArgs {
  const void *x;            // gather: tokens; combine: rows; gradient: tokens (dout)
  void *y;                  // gather: rows; combine: tokens; gradient: rows (dy)
  const void *rows;         // gradient: the rows that were combined
  int64_t ldx, ldy, ldr;
  const int32_t *place, *end;
  const float *weights;
  float *dweights;
  int32_t tokens, topk, hidden, chunks;
};

// An assignment's row; -1 if none is its own.  Nothing but 0 .. tokens * topk - 1
// is used as one, whatever stands in `place`.
__device__ __forceinline__ int row_of(const RowArgs &a, int64_t i, int end) {
  const int p = a.place[i];
  return p >= 0 && p < end ? p : -1;
}
__device__ __forceinline__ int end_of(const RowArgs &a) { return min(*a.end, a.tokens * a.topk); }

// A wave takes 1024 bytes of a token's row and writes them topk times (sizes in
// bytes).  PAST: past the caches, for results that do not fit there (8192 tokens to 8
// rows of 8 KB: 103 us, through them 118).
template <bool PAST> __global__ __launch_bounds__(256) void gather_kernel(RowArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t tasks = (int64_t)a.tokens * a.chunks, all = (int64_t)a.tokens * a.topk;
  const int end = end_of(a);
  for (int64_t task = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); task < tasks; task += (int64_t)gridDim.x * 4) {
    const int64_t t = task / a.chunks;
    const int at = (int)(task - t * a.chunks) * 1024 + lane * 16, left = a.hidden - at;
    if (left <= 0) continue;
    const char *p = static_cast<const char *>(a.x) + t * a.ldx + at;
    u4 v = u4{0, 0, 0, 0};
    if (left >= 16) v = get16<false>(p);
    else
#pragma unroll
      for (int h = 0; h < 8; ++h)
        if (2 * h < left) v[h >> 1] |= (uint32_t) reinterpret_cast<const uint16_t *>(p)[h] << (16 * (h & 1));
    for (int s = 0; s < a.topk; ++s) {
      const int row = a.place[t * a.topk + s];
      if (row < 0 || row >= all) continue;
      char *y = static_cast<char *>(a.y) + row * a.ldy + at;
      const u4 o = row < end ? v : u4{0, 0, 0, 0};
      if (left >= 16) put16<PAST>(y, o);
      else
#pragma unroll
        for (int h = 0; h < 8; ++h)
          if (2 * h < left) reinterpret_cast<uint16_t *>(y)[h] = (uint16_t)(o[h >> 1] >> (16 * (h & 1)));
    }
  }
}

// Calls f with N = MOST or, for the last ones, 4, 2, 1 (as a type) and the first of as many assignments, until topk are
// covered.
template <int MOST, typename F> __device__ __forceinline__ void in_groups(int topk, F f) {
  int s = 0;
  for (; s + MOST <= topk; s += MOST) f(std::integral_constant<int, MOST>{}, s);
  if (MOST > 4 && s + 4 <= topk) {
    f(std::integral_constant<int, 4>{}, s);
    s += 4;
  }
  if (s + 2 <= topk) {
    f(std::integral_constant<int, 2>{}, s);
    s += 2;
  }
  if (s < topk) f(std::integral_constant<int, 1>{}, s);
}

// A wave adds 512 entries of a token's rows, the loads of up to eight rows in flight.
// Rows are read past the caches (8192 tokens of 8 x 4096: 139 us, through them 168;
// 1000 of 6 x 2048: 8.0 and 10.4).  Rows of no expert are replaced by row 0 for the
// load and left out of the sum.
template <typename T> __global__ __launch_bounds__(256) void combine_kernel(RowArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t tasks = (int64_t)a.tokens * a.chunks;
  const int end = end_of(a);
  for (int64_t task = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); task < tasks; task += (int64_t)gridDim.x * 4) {
    const int64_t t = task / a.chunks;
    const int at = (int)(task - t * a.chunks) * 512 + lane * 8, left = a.hidden - at;
    if (left <= 0) continue;
    const T *x = static_cast<const T *>(a.x) + at;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    auto add = [&](auto whole, auto n, int s0) {
      constexpr int N = decltype(n)::value;
      int row[N];
      float w[N];
      Eight<T> v[N];
#pragma unroll
      for (int s = 0; s < N; ++s) {
        row[s] = row_of(a, t * a.topk + s0 + s, end);
        w[s] = a.weights ? a.weights[t * a.topk + s0 + s] : 1.0f;
      }
#pragma unroll
      for (int s = 0; s < N; ++s) v[s].template load<decltype(whole)::value, true>(x + max(row[s], 0) * a.ldx, left);
#pragma unroll
      for (int s = 0; s < N; ++s)
        if (row[s] >= 0) {
          float y[8];
          v[s].get(y);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] = __builtin_fmaf(w[s], y[e], sum[e]);
        }
    };
    if (left >= 8) in_groups<8>(a.topk, [&](auto n, int s0) { add(std::true_type{}, n, s0); });
    else in_groups<8>(a.topk, [&](auto n, int s0) { add(std::false_type{}, n, s0); });
    put8(static_cast<T *>(a.y) + t * a.ldy + at, left, sum);
  }
}

// A workgroup takes a token: four of its rows at a time take w dout and give their dot
// products with it; dout comes from the caches again for the next four.  8192 tokens of
// 8 x 4096: 232 us with reads and writes of rows past the caches, 252 with eight rows at
// a time, 313 with those through the caches.
template <typename T, bool PAST> __global__ __launch_bounds__(256) void combine_grad_kernel(RowArgs a) {
  __shared__ float part[4][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int end = end_of(a);
  const int64_t all = (int64_t)a.tokens * a.topk;
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const T *d = static_cast<const T *>(a.x) + t * a.ldx;
    in_groups<4>(a.topk, [&](auto n, int s0) {
      constexpr int N = decltype(n)::value;
      int row[N];               // -1: nothing to write
      bool real[N];
      float w[N], dot[N];
#pragma unroll
      for (int s = 0; s < N; ++s) {
        row[s] = a.place[t * a.topk + s0 + s];
        if (row[s] < 0 || row[s] >= all) row[s] = -1;
        real[s] = row[s] >= 0 && row[s] < end;
        w[s] = a.weights[t * a.topk + s0 + s];
        dot[s] = 0.0f;
      }
      for (int at = tid * 8; at < a.hidden; at += 2048) {
        const int left = a.hidden - at;
        Eight<T> x, y[N];
        auto load = [&](auto whole) {
          constexpr bool WHOLE = decltype(whole)::value;
          x.template load<WHOLE>(d + at, left);
          if (a.rows)
#pragma unroll
            for (int s = 0; s < N; ++s) y[s].template load<WHOLE, true>(static_cast<const T *>(a.rows) + (real[s] ? row[s] : 0) * a.ldr + at, left);
        };
        if (left >= 8) load(std::true_type{});
        else load(std::false_type{});
        float v[8];
        x.get(v);
        if (a.rows)
#pragma unroll
          for (int s = 0; s < N; ++s)
            if (real[s]) {
              float r[8];
              y[s].get(r);
#pragma unroll
              for (int e = 0; e < 8; ++e) dot[s] = __builtin_fmaf(v[e], r[e], dot[s]);
            }
        if (a.y)
#pragma unroll
          for (int s = 0; s < N; ++s)
            if (row[s] >= 0) {
              float o[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = real[s] ? w[s] * v[e] : 0.0f;
              put8<PAST>(static_cast<T *>(a.y) + row[s] * a.ldy + at, left, o);
            }
      }
      if (!a.dweights) return;
#pragma unroll
      for (int s = 0; s < N; ++s) {
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) dot[s] += __shfl_xor(dot[s], x);
        if (lane == 0) part[wave][s] = dot[s];
      }
      __syncthreads();
      if (tid < N) a.dweights[t * a.topk + s0 + tid] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
      __syncthreads();
    });
  }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t SIZE_LIM = 0x7fffffff, MOST = 1 << 24;      // assignments

tlr_status launched(const char *what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(TLR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
  return TLR_OK;
}

tlr_status check_counts(const std::string &w, int64_t tokens, int32_t topk) {
  if (topk < 1 || topk > MOST_TOPK) return fail(TLR_ERR_INVALID_ARG, w + "topk is 1 .. 64");
  if (tokens < 0 || tokens > SIZE_LIM || tokens * topk > MOST) return fail(TLR_ERR_INVALID_ARG, w + "too many tokens");
  return TLR_OK;
}

// What the operators on rows check; sets the sizes.
tlr_status check_rows(const char *name, tlr_dtype dt, int64_t tokens, int32_t topk, int64_t hidden, const int32_t *place,
                      const int32_t *end, RowArgs *a) {
  const std::string w = std::string(name) + ": ";
  if (dt == TLR_F64) return fail(TLR_ERR_UNSUPPORTED, w + "TLR_F64 is not provided");
  if (dt != TLR_F32 && dt != TLR_F16 && dt != TLR_BF16) return fail(TLR_ERR_INVALID_ARG, w + "bad dtype");
  const tlr_status st = check_counts(w, tokens, topk);
  if (st != TLR_OK) return st;
  if (hidden < 0 || hidden > 1 << 24) return fail(TLR_ERR_INVALID_ARG, w + "hidden out of range");
  if (tokens > 0 && hidden > 0 && (!place || !end || !aligned(place, 4) || !aligned(end, 4)))
    return fail(TLR_ERR_INVALID_ARG, w + "null or misaligned place or end");
  a->place = place;
  a->end = end;
  a->tokens = (int32_t)tokens;
  a->topk = topk;
  a->hidden = (int32_t)hidden;
  return TLR_OK;
}

tlr_status check_matrix(const char *what, tlr_dtype dt, const void *p, int64_t ld, int64_t hidden) {
  if (ld < hidden || ld > SIZE_LIM) return fail(TLR_ERR_INVALID_ARG, std::string(what) + ": leading dimension out of range");
  if (!p || !aligned(p, dt == TLR_F32 ? 4 : 2)) return fail(TLR_ERR_INVALID_ARG, std::string(what) + ": null or misaligned");
  return TLR_OK;
}

// Results that fit into the caches are left there for their reader.
bool past_caches(int64_t bytes) { return bytes >= (int64_t)1 << 26; }

template <typename T> void combine_grad_launch(const RowArgs &a, unsigned grid, hipStream_t st) {
  if (past_caches((int64_t)sizeof(T) * a.tokens * a.topk * a.hidden)) combine_grad_kernel<T, true><<<grid, 256, 0, st>>>(a);
  else combine_grad_kernel<T, false><<<grid, 256, 0, st>>>(a);
}

unsigned wave_grid(int64_t tasks) { return (unsigned)std::min<int64_t>((tasks + 3) / 4, 1 << 22); }

}  // namespace

tlr_status expert_sort_workspace(int64_t tokens, int32_t topk, int32_t experts, size_t *bytes) {
  if (!bytes) return fail(TLR_ERR_INVALID_ARG, "expert_sort_workspace_bytes: null output");
  const tlr_status st = check_counts("expert_sort_workspace_bytes: ", tokens, topk);
  if (st != TLR_OK) return st;
  if (experts < 1 || experts > MOST_EXPERTS) return fail(TLR_ERR_INVALID_ARG, "expert_sort_workspace_bytes: experts are 1 .. 1024");
  const int64_t parts = parts_of(tokens * topk);
  *bytes = parts > 1 ? sizeof(int32_t) * (size_t)(parts + 1) * (experts + 1) : 0;
  return TLR_OK;
}

tlr_status expert_sort(int32_t id_bytes, int64_t tokens, int32_t topk, int32_t experts, const void *ids, int32_t *offsets,
                       int32_t *place, int32_t *rows, void *ws, size_t ws_bytes, void *stream) {
  if (id_bytes != 4 && id_bytes != 8) return fail(TLR_ERR_INVALID_ARG, "expert_sort: ids have 4 or 8 bytes");
  size_t need = 0;
  const tlr_status st = expert_sort_workspace(tokens, topk, experts, &need);
  if (st != TLR_OK) return st;
  const int64_t n = tokens * topk;
  if (!offsets || !aligned(offsets, 4)) return fail(TLR_ERR_INVALID_ARG, "expert_sort: null or misaligned offsets");
  if (n > 0 && (!ids || !aligned(ids, id_bytes) || !place || !aligned(place, 4) || !rows || !aligned(rows, 4)))
    return fail(TLR_ERR_INVALID_ARG, "expert_sort: null or misaligned ids, place or rows");
  if (need > 0 && (!ws || !aligned(ws, 4))) return fail(TLR_ERR_INVALID_ARG, "expert_sort: null or misaligned workspace");
  if (ws_bytes < need) return fail(TLR_ERR_WORKSPACE, "expert_sort: workspace too small");
  const SortArgs a{ids, offsets, place, rows, static_cast<int32_t *>(ws), (int32_t)n, topk, experts, (int32_t)parts_of(n), parts_of(n) > SUMMED};
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (id_bytes == 4) sort_launch<int32_t>(a, hs);
  else sort_launch<int64_t>(a, hs);
  return launched("expert_sort");
}

tlr_status expert_gather(tlr_dtype dt, int64_t tokens, int32_t topk, int64_t hidden, const void *X, int64_t ldx,
                         const int32_t *place, const int32_t *end, void *Y, int64_t ldy, void *stream) {
  RowArgs a{};
  tlr_status st = check_rows("expert_gather", dt, tokens, topk, hidden, place, end, &a);
  if (st != TLR_OK || tokens == 0 || hidden == 0) return st;
  if ((st = check_matrix("expert_gather: X", dt, X, ldx, hidden)) != TLR_OK) return st;
  if ((st = check_matrix("expert_gather: Y", dt, Y, ldy, hidden)) != TLR_OK) return st;
  const int es = dt == TLR_F32 ? 4 : 2;
  a.x = X;
  a.ldx = ldx * es;
  a.y = Y;
  a.ldy = ldy * es;
  a.hidden *= es;
  a.chunks = (a.hidden + 1023) / 1024;
  const unsigned grid = wave_grid(tokens * a.chunks);
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (past_caches(tokens * topk * a.hidden)) gather_kernel<true><<<grid, 256, 0, hs>>>(a);
  else gather_kernel<false><<<grid, 256, 0, hs>>>(a);
  return launched("expert_gather");
}

tlr_status expert_combine(tlr_dtype dt, int64_t tokens, int32_t topk, int64_t hidden, const void *Y, int64_t ldy,
                          const int32_t *place, const int32_t *end, const float *weights, void *out, int64_t ldo, void *stream) {
  RowArgs a{};
  tlr_status st = check_rows("expert_combine", dt, tokens, topk, hidden, place, end, &a);
  if (st != TLR_OK || tokens == 0 || hidden == 0) return st;
  if ((st = check_matrix("expert_combine: Y", dt, Y, ldy, hidden)) != TLR_OK) return st;
  if ((st = check_matrix("expert_combine: out", dt, out, ldo, hidden)) != TLR_OK) return st;
  if (!aligned(weights, 4)) return fail(TLR_ERR_INVALID_ARG, "expert_combine: misaligned weights");
  a.x = Y;
  a.ldx = ldy;
  a.y = out;
  a.ldy = ldo;
  a.weights = weights;
  a.chunks = (a.hidden + 511) / 512;
  const unsigned grid = wave_grid(tokens * a.chunks);
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (dt == TLR_F32) combine_kernel<float><<<grid, 256, 0, hs>>>(a);
  else if (dt == TLR_F16) combine_kernel<_Float16><<<grid, 256, 0, hs>>>(a);
  else combine_kernel<__bf16><<<grid, 256, 0, hs>>>(a);
  return launched("expert_combine");
}

tlr_status expert_combine_grad(tlr_dtype dt, int64_t tokens, int32_t topk, int64_t hidden, const void *dout, int64_t ldd,
                               const void *Y, int64_t ldy, const int32_t *place, const int32_t *end, const float *weights,
                               void *dY, int64_t lddy, float *dweights, void *stream) {
  RowArgs a{};
  tlr_status st = check_rows("expert_combine_grad", dt, tokens, topk, hidden, place, end, &a);
  if (st != TLR_OK || tokens == 0) return st;
  if (!dY && !dweights) return TLR_OK;
  if (hidden > 0 && (st = check_matrix("expert_combine_grad: dout", dt, dout, ldd, hidden)) != TLR_OK) return st;
  if (hidden > 0 && dY && (st = check_matrix("expert_combine_grad: dY", dt, dY, lddy, hidden)) != TLR_OK) return st;
  if (hidden > 0 && dweights && (st = check_matrix("expert_combine_grad: Y", dt, Y, ldy, hidden)) != TLR_OK) return st;
  if (!weights || !aligned(weights, 4)) return fail(TLR_ERR_INVALID_ARG, "expert_combine_grad: null or misaligned weights");
  if (!aligned(dweights, 4)) return fail(TLR_ERR_INVALID_ARG, "expert_combine_grad: misaligned dweights");
  if (!place || !end || !aligned(place, 4) || !aligned(end, 4))
    return fail(TLR_ERR_INVALID_ARG, "expert_combine_grad: null or misaligned place or end");
  a.x = dout;
  a.ldx = ldd;
  a.y = dY;
  a.ldy = lddy;
  a.rows = dweights ? Y : nullptr;
  a.ldr = ldy;
  a.weights = weights;
  a.dweights = dweights;
  const unsigned grid = (unsigned)std::min<int64_t>(tokens, 1 << 20);
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (dt == TLR_F32) combine_grad_launch<float>(a, grid, hs);
  else if (dt == TLR_F16) combine_grad_launch<_Float16>(a, grid, hs);
  else combine_grad_launch<__bf16>(a, grid, hs);
  return launched("expert_combine_grad");
}

}  // namespace tlr
