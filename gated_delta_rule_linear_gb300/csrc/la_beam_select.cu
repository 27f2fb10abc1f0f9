// Beam search's selection: of W beams with V continuations each, the K best by
// c(w, v) = scores[w] + x[w][v] - log sum_u exp x[w][u].
//
// Bound by reading the logits once. Two kernels. The first takes a segment of a
// row: the K best of it, by logits (inside a row the order of c is that of x),
// and the segment's part of the sum. The second takes a request: the log of each
// beam's sum, the segments' candidates' scores in 64 bits, and their K best.
//
// K best of a segment. A thread holds 16 elements; each warp sorts its lanes'
// largest, and no element below a warp's K-th largest lane can be among the K
// best: the highest of these bounds leaves little more than K elements, which
// are collected and sorted. Keys are value and index together, so that equal
// logits (bfloat16 has many) neither break the order nor the bound on how many
// are collected.
//
// The sum. exp(x - max) with 24 bits (a polynomial: the special-function unit's
// 22 bits would blur the comparison of two beams), summed in pairs inside a
// thread and in 64-bit fixed point across threads: the sum does not depend on
// the order, two beams with the same logits get the same one.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "la_serve_internal.h"

namespace la {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPer = 16;                       // elements of a thread
constexpr int kSegment = kThreads * kPer;
constexpr double kFixed = 17592186044416.0;    // 2^44: a segment's sum of at most 4096 stays below 2^57

// What the first kernel leaves of a segment; its K keys are in an array of their own.
struct Segment {
  u64 sum;      // of exp(x - max), fixed point
  float max;
  int bad;      // it has a NaN or +infinity
};

// The order of floats (no NaN) as that of unsigned integers.
__device__ __forceinline__ unsigned ordered(float x) {
  const int b = __float_as_int(x);
  return static_cast<unsigned>(b ^ (b >> 31 & 0x7fffffff)) ^ 0x80000000u;
}
__device__ __forceinline__ float unordered(unsigned u) {
  const int b = static_cast<int>(u ^ 0x80000000u);
  return __int_as_float(b ^ (b >> 31 & 0x7fffffff));
}

constexpr unsigned kPlusInf = 0xff800000u;  // ordered(+infinity); NaNs are above (x + 0 has made them positive)

// exp(x), x <= 0, to about 2^-24: x = (n + f) ln 2 with the product's rounding carried along, then the
// series of 2^f = exp(f ln 2) for |f| <= 1/2 to its seventh power (2^-27 off).
__device__ __forceinline__ float exp_of(float x) {
  x = fmaxf(x, -87.f);  // below: 1e-38 each
  const float t = x * 1.44269504f;
  const float lo = fmaf(x, 1.44269504f, -t) + x * 1.925963033e-8f;
  const float n = rintf(t);
  const float f = ((t - n) + lo) * 0.693147181f;
  float y = 1.f / 5040;
  y = fmaf(y, f, 1.f / 720);
  y = fmaf(y, f, 1.f / 120);
  y = fmaf(y, f, 1.f / 24);
  y = fmaf(y, f, 1.f / 6);
  y = fmaf(y, f, 0.5f);
  y = fmaf(y, f, 1.f);
  y = fmaf(y, f, 1.f);
  return y * __int_as_float((static_cast<int>(n) + 127) << 23);
}

// Bitonic exchange with the lane j away; `top` keeps the larger key.
__device__ __forceinline__ u64 exchange(u64 k, int j, bool top) {
  const u64 o = __shfl_xor_sync(~0u, k, j);
  return (o > k) == top ? o : k;
}
struct Key128 {  // a candidate: score (ordered), then the order of w * V + v; 0, 0: none
  u64 score;
  unsigned rank;  // ~(w * V + v)
};
__device__ __forceinline__ bool above(u64 a, u64 b) { return a > b; }
__device__ __forceinline__ bool above(const Key128 &a, const Key128 &b) {
  return a.score > b.score || (a.score == b.score && a.rank > b.rank);
}
__device__ __forceinline__ Key128 exchange(const Key128 &k, int j, bool top) {
  const Key128 o = {__shfl_xor_sync(~0u, k.score, j), __shfl_xor_sync(~0u, k.rank, j)};
  return above(o, k) == top ? o : k;
}
__device__ __forceinline__ u64 reversed(u64 k) { return __shfl_xor_sync(~0u, k, 31); }
__device__ __forceinline__ Key128 reversed(const Key128 &k) {
  return {__shfl_xor_sync(~0u, k.score, 31), __shfl_xor_sync(~0u, k.rank, 31)};
}

// A warp's keys in descending order over its lanes.
template <typename Key>
__device__ __forceinline__ Key sorted(Key k, int lane) {
#pragma unroll
  for (int n = 2; n <= 32; n *= 2)
#pragma unroll
    for (int j = n / 2; j > 0; j /= 2) k = exchange(k, j, ((lane & n) == 0) == ((lane & j) == 0));
  return k;
}
// The 32 largest of two such lists, as one.
template <typename Key>
__device__ __forceinline__ Key merged(Key a, const Key &b, int lane) {
  const Key r = reversed(b);
  if (above(r, a)) a = r;
#pragma unroll
  for (int j = 16; j > 0; j /= 2) a = exchange(a, j, (lane & j) == 0);
  return a;
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads) segment_kernel(const BeamSelect p, int segments, Segment *seg, u64 *keys) {
  __shared__ u64 list[kSegment];
  __shared__ u64 bound[kWarps], sums[kWarps];
  __shared__ unsigned most[kWarps];
  __shared__ int count;
  const int row = blockIdx.x / segments, j = blockIdx.x % segments, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (p.done && p.done[row]) return;
  const T *x = static_cast<const T *>(p.logits) + row * p.ld;
  const int v0 = j * kSegment;
  constexpr int E = WIDE ? 16 / sizeof(T) : 1;
  // element e of the thread's i-th vector is v0 + (i * kThreads + tid) * E + e
  float f[kPer];
#pragma unroll
  for (int i = 0; i < kPer / E; ++i) {
    const int v = v0 + (i * kThreads + tid) * E;
    if constexpr (E == 1) {
      f[i] = v < p.V ? static_cast<float>(x[v]) : -INFINITY;
    } else {
      if (v + E <= p.V) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(x + v));
        const unsigned a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if constexpr (sizeof(T) == 4) f[i * E + e] = __uint_as_float(a[e]);
          else f[i * E + e] = __uint_as_float(e & 1 ? a[e / 2] & 0xffff0000u : a[e / 2] << 16);
        }
      } else {  // the row ends inside, or before
#pragma unroll
        for (int e = 0; e < E; ++e) f[i * E + e] = v + e < p.V ? static_cast<float>(x[v + e]) : -INFINITY;
      }
    }
  }
  if (tid == 0) count = 0;
  // the largest of the thread, with the lowest index: key 0 for places behind the row's end
  u64 top = 0;
  auto key = [&](int i) {
    const int v = v0 + (i / E * kThreads + tid) * E + i % E;
    return v < p.V ? (u64)ordered(f[i]) << 32 | ~static_cast<unsigned>(v) : 0ull;
  };
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    f[i] += 0.f;  // one zero, and one NaN
    const u64 k = key(i);
    if (k > top) top = k;
  }
  const u64 order = sorted(top, lane);
  const u64 kth = __shfl_sync(~0u, order, p.K - 1);
  if (lane == 0) {
    bound[warp] = kth;
    most[warp] = static_cast<unsigned>(order >> 32);
  }
  __syncthreads();
  u64 low = 0;
  unsigned high = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    low = bound[i] > low ? bound[i] : low;
    high = max(high, most[i]);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const u64 k = key(i);
    if (k && k >= low) list[atomicAdd(&count, 1)] = k;
  }
  const bool bad = high >= kPlusInf;
  const float m = unordered(high);
  // the sum, where there is one
  u64 sum = 0;
  if (!bad && m > -INFINITY) {
    float e[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) e[i] = key(i) ? exp_of(f[i] - m) : 0.f;
#pragma unroll
    for (int n = kPer / 2; n > 0; n /= 2)
#pragma unroll
      for (int i = 0; i < n; ++i) e[i] += e[i + n];
    sum = static_cast<u64>(static_cast<double>(e[0]) * kFixed);
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(~0u, sum, d);
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  // the list's K best: every warp sorts what it takes of it, the first one joins them
  const int n = count;
  u64 best = 0;
  for (int i = warp * 32; i < n; i += kThreads) {
    const u64 k = sorted(i + lane < n ? list[i + lane] : 0, lane);
    best = merged(best, k, lane);
  }
  if (n > 32) {
    __syncthreads();
    list[tid] = best;
    __syncthreads();
    if (warp == 0)
      for (int i = 1; i < min(kWarps, (n + 31) / 32); ++i) best = merged(best, list[i * 32 + lane], lane);
  }
  if (warp == 0) {
    if (lane < p.K) keys[(size_t)blockIdx.x * p.K + lane] = best;
    if (lane == 0) {
      u64 s = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) s += sums[i];
      seg[blockIdx.x] = {s, m, bad};
    }
  }
}

__device__ __forceinline__ u64 ordered(double x) {
  const long long b = __double_as_longlong(x);
  return static_cast<u64>(b ^ (b >> 63 & 0x7fffffffffffffffll)) ^ 0x8000000000000000ull;
}
__device__ __forceinline__ double unordered(u64 u) {
  const long long b = static_cast<long long>(u ^ 0x8000000000000000ull);
  return __longlong_as_double(b ^ (b >> 63 & 0x7fffffffffffffffll));
}

__global__ void __launch_bounds__(kThreads) select_kernel(const BeamSelect p, int segments, const Segment *seg, const u64 *keys) {
  __shared__ double lse[kMaxBeams];   // of each beam; NaN: its candidates have no value
  __shared__ Key128 lists[kThreads];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int w = warp; w < p.W; w += kWarps) {
    const int row = b * p.W + w;
    double value = CUDART_NAN;
    const float score = p.scores[row];
    const bool ends = p.done && p.done[row];
    if (!ends && isfinite(score)) {
      const Segment *s = seg + (size_t)row * segments;
      float m = -INFINITY;
      int bad = 0;
      for (int i = lane; i < segments; i += 32) {
        m = fmaxf(m, s[i].max);
        bad |= s[i].bad;
      }
#pragma unroll
      for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
      if (!__any_sync(~0u, bad) && m > -INFINITY) {
        double sum = 0;
        for (int i = lane; i < segments; i += 32)
          if (s[i].sum) sum += static_cast<double>(s[i].sum) * (1.0 / kFixed) * exp(static_cast<double>(s[i].max) - m);
#pragma unroll
        for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(~0u, sum, d);
        value = m + log(sum);
      }
    }
    if (lane == 0) lse[w] = value;
  }
  __syncthreads();
  const u64 none = ordered(-(double)INFINITY);
  Key128 best = {0, 0};
  const int each = segments * p.K;
  for (int i0 = warp * 32; i0 < p.W * each; i0 += kThreads) {
    const int i = i0 + lane;
    Key128 k = {0, 0};
    if (i < p.W * each) {
      const int w = i / each, at = i % each, row = b * p.W + w;
      const float score = p.scores[row];
      if (p.done && p.done[row]) {
        // eos, and the first tokens besides it without a value
        if (at == 0) {
          k = {isfinite(score) ? ordered((double)score) : none, ~static_cast<unsigned>(w * p.V + p.eos)};
        } else if (at < p.K && at < p.V) {
          k = {none, ~static_cast<unsigned>(w * p.V + at - (at <= p.eos))};
        }
      } else if (isnan(lse[w])) {
        if (at < p.K && at < p.V) k = {none, ~static_cast<unsigned>(w * p.V + at)};
      } else {
        const u64 c = keys[(size_t)row * each + at];
        if (c) {
          const double x = (double)score + ((double)unordered(static_cast<unsigned>(c >> 32)) - lse[w]);
          k = {ordered(x), ~(static_cast<unsigned>(w * p.V) + ~static_cast<unsigned>(c))};
        }
      }
    }
    best = merged(best, sorted(k, lane), lane);
  }
  lists[tid] = best;
  for (int half = kWarps / 2; half > 0; half /= 2) {
    __syncthreads();
    if (warp < half) {
      best = merged(best, lists[tid + half * 32], lane);
      lists[tid] = best;
    }
  }
  if (tid < p.K) {
    const unsigned at = ~best.rank;
    const size_t out = (size_t)b * p.K + tid;
    p.scores_out[out] = static_cast<float>(unordered(best.score));
    p.parent[out] = at / p.V;
    p.token[out] = at % p.V;
  }
}

template <typename T>
void launch(const BeamSelect &p, int segments, Segment *seg, u64 *keys, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.B) * p.W * segments;
  const bool wide = (reinterpret_cast<uintptr_t>(p.logits) & 15) == 0 && p.ld * sizeof(T) % 16 == 0;
  if (wide) segment_kernel<T, true><<<grid, kThreads, 0, stream>>>(p, segments, seg, keys);
  else segment_kernel<T, false><<<grid, kThreads, 0, stream>>>(p, segments, seg, keys);
}

int fail(const char *what, cudaError_t e) {
  set_error("la_beam_select: %s: %s", what, cudaGetErrorString(e));
  return LA_ERR_CUDA;
}

}  // namespace

int launch_beam_select(const BeamSelect &p, cudaStream_t stream) {
  const int segments = (p.V - 1) / kSegment + 1;
  const size_t parts = (size_t)p.B * p.W * segments;
  uint8_t *ws = nullptr;
  cudaMemPool_t pool = library_pool();
  if (!pool) return fail("could not create the workspace pool", cudaGetLastError());
  cudaError_t e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), parts * (sizeof(Segment) + sizeof(u64) * p.K),
                                          pool, stream);
  if (e != cudaSuccess) return fail("workspace allocation failed", e);
  Segment *seg = reinterpret_cast<Segment *>(ws);
  u64 *keys = reinterpret_cast<u64 *>(seg + parts);
  if (p.f32) launch<float>(p, segments, seg, keys, stream);
  else launch<__nv_bfloat16>(p, segments, seg, keys, stream);
  e = cudaGetLastError();
  if (e == cudaSuccess) {
    select_kernel<<<p.B, kThreads, 0, stream>>>(p, segments, seg, keys);
    e = cudaGetLastError();
  }
  const cudaError_t f = cudaFreeAsync(ws, stream);
  if (e == cudaSuccess) e = f;
  return e == cudaSuccess ? LA_OK : fail("launch failed", e);
}

}  // namespace la
