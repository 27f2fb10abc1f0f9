// Beam search's selection: of W beams with V continuations each, the K best by
// c(w, v) = scores[w] + x[w][v] - log sum_u exp x[w][u].
//
// Bound by reading the logits once. Two kernels. The first takes a segment of a
// row: the K best of it, by logits (inside a row the order of c is that of x),
// and the segment's part of the sum. The second takes a request: the log of each
// beam's sum, the segments' candidates' scores in 64 bits, and their K best.
//
// K best of a segment. A thread holds 8, 16 or 32 elements; each warp sorts its
// lanes' largest, and no element below a warp's K-th largest lane can be among
// the K best: the highest of these bounds leaves little more than K elements, of
// a few threads, which are collected and sorted as (value, index). Rows with so
// many equal logits that the list runs over go round by round instead.
//
// The sum. exp2((x - max) log2 e), in pairs inside a thread, in 64-bit fixed point
// across threads and segments: what is added does not depend on where a row lies
// or which threads had it, so that two beams with the same logits get the same
// sum. Rows that do not start at 16 bytes are therefore shifted into place.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>

#include "la_serve_internal.h"
#include "la_sm100.cuh"

namespace la {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kList = 512;                    // elements that a segment's bound may leave
constexpr float kLog2e = 1.44269504f;
constexpr float kFixed = 17592186044416.f;    // 2^44: a segment's sum of at most 8192 stays below 2^58

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

// Bitonic exchange with the lane j away; `top` keeps the larger key.
template <typename Word>
__device__ __forceinline__ Word exchange(Word k, int j, bool top) {
  const Word o = __shfl_xor_sync(~0u, k, j);
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

// max(a, b), NaN if one of them is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 16 bytes of a row of logits at element v of it: E elements, -infinity behind the row's end. SHIFT: the row may start
// anywhere, `off` bytes behind a multiple of 16; the granules of 16 bytes are read whole, but never outside [lo, hi).
template <typename T, bool SHIFT, int E>
__device__ __forceinline__ void load_row(const T *x, int v, int V, int off, const char *lo, const char *hi, float (&f)[E]) {
  static_assert(E * sizeof(T) == 16, "");
  unsigned w[4];
  const char *at = reinterpret_cast<const char *>(x + v) - off;
  const bool whole = v + E <= V;
  if (whole && (!SHIFT || (at >= lo && at + (off ? 32 : 16) <= hi))) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(at));
    if constexpr (SHIFT) {
      uint4 b = a;
      if (off) b = __ldcs(reinterpret_cast<const uint4 *>(at) + 1);  // the next thread's, from L1
      const unsigned in[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      const unsigned bits = off % 4 * 8;
      switch (off / 4) {
#define LA_SHIFTED(Q)                                                                                \
  case Q:                                                                                            \
    _Pragma("unroll") for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(in[Q + i], in[Q + i + (Q + i < 7)], bits); \
    break;
        LA_SHIFTED(0) LA_SHIFTED(1) LA_SHIFTED(2) LA_SHIFTED(3)
#undef LA_SHIFTED
      }
    } else {
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if constexpr (sizeof(T) == 4) f[e] = __uint_as_float(w[e]);
      else f[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = v + e < V ? static_cast<float>(x[v + e]) : -INFINITY;
  }
}

// A segment: kThreads * PER elements of a row.
template <typename T, int PER, bool SHIFT>
__global__ void __launch_bounds__(kThreads) segment_kernel(const BeamSelect p, int segments, Segment *seg, u64 *keys) {
  constexpr int E = 16 / sizeof(T), N = PER / E, kSegment = kThreads * PER;
  __shared__ u64 list[kList];
  __shared__ u64 sums[kWarps];
  __shared__ float bounds[kWarps], tops[kWarps];
  __shared__ int count;
  const int row = blockIdx.x / segments, j = blockIdx.x % segments, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (p.done && p.done[row]) return;
  const T *x = static_cast<const T *>(p.logits) + row * p.ld;
  const int v0 = j * kSegment + tid * E;  // element e of the thread's i-th vector is v0 + i * kThreads * E + e
  const char *lo = static_cast<const char *>(p.logits);
  const char *hi = reinterpret_cast<const char *>(static_cast<const T *>(p.logits) + ((size_t)p.B * p.W - 1) * p.ld + p.V);
  const int off = SHIFT ? static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15) : 0;
  float f[N][E];
#pragma unroll
  for (int i = 0; i < N; ++i) load_row<T, SHIFT, E>(x, v0 + i * kThreads * E, p.V, off, lo, hi, f[i]);
  if (tid == 0) count = 0;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) top = max_nan(top, f[i][e]);
  const bool nan = isnan(top);
  if (nan) top = INFINITY;
  // the warp's K-th largest lane, as ordered integers (+0 and -0 alike)
  const unsigned order = sorted(ordered(top + 0.f), lane);
  if (lane == 0) tops[warp] = unordered(order);
  if (lane == p.K - 1) bounds[warp] = unordered(order);
  __syncthreads();
  float low = bounds[0], m = tops[0];
#pragma unroll
  for (int i = 1; i < kWarps; ++i) {
    low = fmaxf(low, bounds[i]);
    m = fmaxf(m, tops[i]);
  }
  const bool bad = m == INFINITY;
  // the sum, where there is one
  u64 sum = 0;
  if (!bad && m > -INFINITY) {
    float t[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float g[E];
#pragma unroll
      for (int e = 0; e < E; ++e) g[e] = sm100::ex2((f[i][e] - m) * kLog2e);
#pragma unroll
      for (int n = E / 2; n > 0; n /= 2)
#pragma unroll
        for (int e = 0; e < n; ++e) g[e] += g[e + n];
      t[i] = g[0];
    }
#pragma unroll
    for (int n = N / 2; n > 0; n /= 2)
#pragma unroll
      for (int i = 0; i < n; ++i) t[i] += t[i + n];
    sum = static_cast<u64>(t[0] * kFixed);
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(~0u, sum, d);
  if (lane == 0) sums[warp] = sum;
  auto key = [&](int i, int e) {
    const int v = v0 + i * kThreads * E + e;
    return v < p.V ? (u64)ordered(f[i][e] + 0.f) << 32 | ~static_cast<unsigned>(v) : 0ull;
  };
  // (a bad row's candidates are not looked at)
  if (!bad && top >= low)
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (f[i][e] >= low && v0 + i * kThreads * E + e < p.V) {
          const int at = atomicAdd(&count, 1);
          if (at < kList) list[at] = key(i, e);
        }
  __syncthreads();
  const int n = count;
  u64 best = 0;
  if (n > kList) {
    // the next one below the last, K times
    u64 last = ~0ull;
    for (int k = 0; k < p.K; ++k) {
      u64 mine = 0;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const u64 c = key(i, e);
          if (c < last && c > mine) mine = c;
        }
#pragma unroll
      for (int d = 16; d > 0; d /= 2) mine = max(mine, __shfl_xor_sync(~0u, mine, d));
      if (lane == 0) list[(k & 1) * kWarps + warp] = mine;
      __syncthreads();
      last = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) last = max(last, list[(k & 1) * kWarps + i]);
      if (lane == k) best = last;
    }
  } else {
    // every warp sorts what it takes of the list, the first one joins them
    for (int i = warp * 32; i < n; i += kThreads) best = merged(best, sorted(i + lane < n ? list[i + lane] : 0, lane), lane);
    if (n > 32) {
      __syncthreads();
      list[tid] = best;
      __syncthreads();
      if (warp == 0)
        for (int i = 1; i < min(kWarps, (n + 31) / 32); ++i) best = merged(best, list[i * 32 + lane], lane);
    }
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

// exp(x) for x <= 0, to about 2^-24, as a factor of 2^32.
__device__ __forceinline__ unsigned weight(float x) {
  return x == 0.f ? ~0u : __float2uint_rz(expf(x) * 4294967296.f);
}

constexpr int kSelectThreads = 512, kSelectWarps = kSelectThreads / 32;

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const BeamSelect p, int segments, const Segment *seg,
                                                                const u64 *keys) {
  __shared__ double lse[kMaxBeams];   // of each beam; NaN: its candidates have no value
  __shared__ u64 total[kMaxBeams];
  __shared__ float tops[kMaxBeams];
  __shared__ u64 bounds[kSelectWarps];
  __shared__ Key128 list[kList];
  __shared__ int count;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float *scores = p.scores + b * p.W;
  const unsigned char *done = p.done ? p.done + b * p.W : nullptr;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid == 0) count = 0;
  for (int w = warp; w < p.W; w += kSelectWarps) {
    if (done && done[w]) continue;
    const Segment *s = seg + (size_t)(b * p.W + w) * segments;
    float m = -INFINITY;
    bool bad = false;
    for (int i = lane; i < segments; i += 32) {
      m = fmaxf(m, s[i].max);
      bad |= s[i].bad != 0;
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
    if (__any_sync(~0u, bad) || m == -INFINITY) {
      if (lane == 0) total[w] = 0;
      continue;
    }
    u64 sum = 0;
    for (int i = lane; i < segments; i += 32) {
      const unsigned f = s[i].sum ? weight(s[i].max - m) : 0;
      sum += f == ~0u ? s[i].sum : __umul64hi(s[i].sum, (u64)f << 32);
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(~0u, sum, d);
    if (lane == 0) {
      total[w] = sum;
      tops[w] = m;
    }
  }
  __syncthreads();
  if (tid < p.W) {  // all logs of a request in one warp: 64-bit instructions are few on this chip
    double value = CUDART_NAN;
    if (!(done && done[tid]) && total[tid] && isfinite(scores[tid])) value = tops[tid] + log((double)total[tid] * (1.0 / kFixed));
    lse[tid] = value;
  }
  __syncthreads();
  const u64 none = ordered(-(double)INFINITY);
  const int each = segments * p.K, lists = p.W * segments;
  // the r-th candidate of segment j of beam w; each segment's come in descending order
  auto candidate = [&](int w, int j, int r) -> Key128 {
    const int at = j * p.K + r;
    if (done && done[w]) {
      // eos, and the first tokens besides it without a value
      if (at == 0) return {isfinite(scores[w]) ? ordered((double)scores[w]) : none, ~static_cast<unsigned>(w * p.V + p.eos)};
      if (at < p.K && at < p.V) return {none, ~static_cast<unsigned>(w * p.V + at - (at <= p.eos))};
      return {0, 0};
    }
    if (isnan(lse[w])) return at < p.K && at < p.V ? Key128{none, ~static_cast<unsigned>(w * p.V + at)} : Key128{0, 0};
    const u64 c = keys[(size_t)(b * p.W + w) * each + at];
    if (!c) return {0, 0};
    const double x = (double)scores[w] + ((double)unordered(static_cast<unsigned>(c >> 32)) - lse[w]);
    return {ordered(x), ~(static_cast<unsigned>(w * p.V) + ~static_cast<unsigned>(c))};
  };
  // as in a segment: the K-th of the lists' first candidates bounds what can be among the K best
  u64 head = 0;
  for (int i = tid; i < lists; i += kSelectThreads) head = max(head, candidate(i / segments, i % segments, 0).score);
  const u64 order = sorted(head, lane);
  if (lane == p.K - 1) bounds[warp] = order;
  __syncthreads();
  u64 low = 1;
#pragma unroll
  for (int i = 0; i < kSelectWarps; ++i) low = max(low, bounds[i]);
  for (int i = tid; i < lists; i += kSelectThreads)
    for (int r = 0; r < p.K; ++r) {
      const Key128 k = candidate(i / segments, i % segments, r);
      if (k.score < low) break;
      const int at = atomicAdd(&count, 1);
      if (at < kList) list[at] = k;
    }
  __syncthreads();
  const int n = count;
  Key128 best = {0, 0};
  if (n > kList) {  // all of them
    for (int i0 = warp * 32; i0 < p.W * each; i0 += kSelectThreads) {
      const int i = i0 + lane;
      Key128 k = {0, 0};
      if (i < p.W * each) k = candidate(i / each, i % each / p.K, i % p.K);
      best = merged(best, sorted(k, lane), lane);
    }
  } else {
    const int i = warp * 32 + lane;
    if (warp * 32 < n) best = sorted(i < n ? list[i] : Key128{0, 0}, lane);
  }
  for (int half = kSelectWarps / 2; half > 0; half /= 2) {
    if (n <= half * 32) continue;  // (nothing in those warps)
    __syncthreads();
    if (warp >= half && warp < 2 * half) list[tid - half * 32] = best;
    __syncthreads();
    if (warp < half) best = merged(best, list[tid], lane);
  }
  if (tid < p.K) {
    const unsigned at = ~best.rank;
    const size_t out = (size_t)b * p.K + tid;
    p.scores_out[out] = static_cast<float>(unordered(best.score));
    p.parent[out] = at / p.V;
    p.token[out] = at % p.V;
  }
}

// Elements of a thread: few where the grid would leave SMs idle (four beams of 32000 float32 logits, both kernels:
// 8 a thread TODO us, 32 TODO us), many where the sorting of the lanes counts (32 x 8 rows of 50257: TODO).
int per_thread(const BeamSelect &p) {
  const long long all = (long long)p.B * p.W * p.V, room = 2ll * kThreads * std::max(sm_count(), 1);
  return all <= 8 * room ? 8 : all <= 16 * room ? 16 : 32;
}

template <typename T, int PER>
void launch_per(const BeamSelect &p, int segments, Segment *seg, u64 *keys, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.B) * p.W * segments;
  const bool wide = (reinterpret_cast<uintptr_t>(p.logits) & 15) == 0 && p.ld * sizeof(T) % 16 == 0;
  if (wide) segment_kernel<T, PER, false><<<grid, kThreads, 0, stream>>>(p, segments, seg, keys);
  else segment_kernel<T, PER, true><<<grid, kThreads, 0, stream>>>(p, segments, seg, keys);
}

template <typename T>
void launch(const BeamSelect &p, int per, int segments, Segment *seg, u64 *keys, cudaStream_t stream) {
  if (per == 8) launch_per<T, 8>(p, segments, seg, keys, stream);
  else if (per == 16) launch_per<T, 16>(p, segments, seg, keys, stream);
  else launch_per<T, 32>(p, segments, seg, keys, stream);
}

int fail(const char *what, cudaError_t e) {
  set_error("la_beam_select: %s: %s", what, cudaGetErrorString(e));
  return LA_ERR_CUDA;
}

}  // namespace

int launch_beam_select(const BeamSelect &p, cudaStream_t stream) {
  const int per = per_thread(p), segments = (p.V - 1) / (kThreads * per) + 1;
  const size_t parts = (size_t)p.B * p.W * segments;
  uint8_t *ws = nullptr;
  cudaMemPool_t pool = library_pool();
  if (!pool) return fail("could not create the workspace pool", cudaGetLastError());
  cudaError_t e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), parts * (sizeof(Segment) + sizeof(u64) * p.K),
                                          pool, stream);
  if (e != cudaSuccess) return fail("workspace allocation failed", e);
  Segment *seg = reinterpret_cast<Segment *>(ws);
  u64 *keys = reinterpret_cast<u64 *>(seg + parts);
  if (p.f32) launch<float>(p, per, segments, seg, keys, stream);
  else launch<__nv_bfloat16>(p, per, segments, seg, keys, stream);
  e = cudaGetLastError();
  if (e == cudaSuccess) {  // launched while the first one runs, and waits for its end
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.B);
    cfg.blockDim = dim3(kSelectThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, select_kernel, p, segments, static_cast<const Segment *>(seg), static_cast<const u64 *>(keys));
  }
  const cudaError_t f = cudaFreeAsync(ws, stream);
  if (e == cudaSuccess) e = f;
  return e == cudaSuccess ? LA_OK : fail("launch failed", e);
}

}  // namespace la
