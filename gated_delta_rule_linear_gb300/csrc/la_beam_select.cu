// Beam search's selection: of W beams with V continuations each, the K best by
// c(w, v) = scores[w] + x[w][v] - log sum_u exp x[w][u].
//
// Bound by reading the logits once. Two kernels. In the first a warp takes a part
// of a row: the K best of it, by logits (inside a row the order of c is that of
// x), and the part's share of the sum. The second takes a request: the log of
// each beam's sum, the parts' candidates' scores in 64 bits, and their K best.
//
// K best of a part. A warp goes through it tile by tile with a cut below which
// nothing can be among its K best: first the K-th largest of its lanes' largest,
// later the K-th of what it has. What passes is collected, and sorted into the
// list of the best when there is a warpful, which is rare: K log(tiles) elements
// of a part pass. Keys are value and index together, so that the order is right
// for equal logits (bfloat16 has many). Warps do not wait for one another.
//
// The sum. exp(x - r) with one reference r for a part, its first largest value:
// a floating-point sum may grow above one. In pairs inside a tile, in 64 bits
// across lanes. Which elements meet in which order depends on their index alone,
// not on where a row lies, so that two beams with the same logits get the same
// sum; rows that do not start at 16 bytes are shifted into place for this.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>

#include "la_serve_internal.h"
#include "la_sm100.cuh"

namespace la {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 128, kWarps = kThreads / 32;  // of the first kernel
constexpr float kLog2e = 1.44269504f;

// What the first kernel leaves of a part; its K keys are in an array of their own.
struct Part {
  double sum;   // of exp(x - ref)
  float ref;
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

// A warp's keys in descending order over its lanes. (Rolled, as all that runs a few times only: fetching straight-line
// code costs more than running it.)
template <typename Key>
__device__ __forceinline__ Key sorted(Key k, int lane) {
#pragma unroll 1
  for (int n = 2; n <= 32; n *= 2)
#pragma unroll 1
    for (int j = n / 2; j > 0; j /= 2) k = exchange(k, j, ((lane & n) == 0) == ((lane & j) == 0));
  return k;
}
// The 32 largest of two such lists, as one.
template <typename Key>
__device__ __forceinline__ Key merged(Key a, const Key &b, int lane) {
  const Key r = reversed(b);
  if (above(r, a)) a = r;
#pragma unroll 1
  for (int j = 16; j > 0; j /= 2) a = exchange(a, j, (lane & j) == 0);
  return a;
}

// max(a, b), NaN if one of them is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ unsigned max_nan2(unsigned a, unsigned b) {  // two bfloat16
  unsigned r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 16 bytes of logits.
template <typename T> struct Granule {
  static constexpr int E = 16 / sizeof(T);
  unsigned w[4];
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  }
  __device__ __forceinline__ float max() const {
    if constexpr (sizeof(T) == 4) {
      return max_nan(max_nan((*this)[0], (*this)[1]), max_nan((*this)[2], (*this)[3]));
    } else {
      const unsigned m = max_nan2(max_nan2(w[0], w[1]), max_nan2(w[2], w[3]));
      return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
  }
  // Elements v .. v + E - 1 of a row of V, -infinity behind its end. SHIFT: the row may start anywhere, `off` bytes
  // behind a multiple of 16; granules of memory are read whole, but never outside [lo, hi).
  template <bool SHIFT>
  __device__ __forceinline__ void load(const T *x, int v, int V, int off, const char *lo, const char *hi) {
    const char *at = reinterpret_cast<const char *>(x + v) - off;
    uint4 a = make_uint4(kNone, kNone, kNone, kNone);
    if (v < V && at >= lo && at + (SHIFT && off ? 32 : 16) <= hi) {
      a = __ldcs(reinterpret_cast<const uint4 *>(at));
      if constexpr (SHIFT) {
        uint4 b = a;
        if (off) b = __ldcs(reinterpret_cast<const uint4 *>(at) + 1);  // the next lane's, from L1
        if (off & 8) a = make_uint4(a.z, a.w, b.x, b.y), b = make_uint4(b.z, b.w, b.z, b.w);
        if (off & 4) a = make_uint4(a.y, a.z, a.w, b.x), b.x = b.y;
        if (off & 2)
          a = make_uint4(__funnelshift_r(a.x, a.y, 16), __funnelshift_r(a.y, a.z, 16), __funnelshift_r(a.z, a.w, 16),
                         __funnelshift_r(a.w, b.x, 16));
      }
    } else if (v < V) {
      a = one_by_one(x, v, V);
    }
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    if (v + E > V) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int behind = V - v - i * E / 4;  // elements of this word inside the row
        if (behind <= 0) w[i] = kNone;
        else if (sizeof(T) == 2 && behind == 1) w[i] = w[i] & 0xffffu | kNone & 0xffff0000u;
      }
    }
  }

 private:
  static constexpr unsigned kNone = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -infinity
  static __device__ __noinline__ uint4 one_by_one(const T *x, int v, int V) {
    u64 half[2] = {0, 0};
#pragma unroll 1
    for (int e = 0; e < E; ++e) {
      if (v + e >= V) break;
      u64 bits;
      if constexpr (sizeof(T) == 4) bits = __float_as_uint(static_cast<float>(x[v + e]));
      else bits = *reinterpret_cast<const unsigned short *>(x + v + e);
      bits <<= e % (E / 2) * 8 * static_cast<int>(sizeof(T));
      if (e < E / 2) half[0] |= bits;
      else half[1] |= bits;
    }
    return make_uint4(static_cast<unsigned>(half[0]), static_cast<unsigned>(half[0] >> 32), static_cast<unsigned>(half[1]),
                      static_cast<unsigned>(half[1] >> 32));
  }
};

// A warp's collection: granules with an element above the cut, and such elements' keys.
template <int N> struct Collected {
  uint4 granule[32 * N];
  int index[32 * N];   // of a granule's first element
  u64 key[64];
};

// A warp, one part: `tiles` tiles of 32 * N granules, the next one's logits on their way meanwhile.
template <typename T, int N, bool SHIFT>
__global__ void __launch_bounds__(kThreads) part_kernel(const BeamSelect p, int total, int parts, int tiles, Part *part,
                                                        u64 *keys) {
  constexpr int E = Granule<T>::E, kTile = 32 * N * E;
  __shared__ Collected<N> collected[kWarps];
  wait_for_stream();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int id = blockIdx.x * kWarps + warp;
  if (id >= total) return;
  const int row = id / parts;
  if (p.done && p.done[row]) return;
  Collected<N> &c = collected[warp];
  const char *lo = static_cast<const char *>(p.logits);
  const char *hi = reinterpret_cast<const char *>(static_cast<const T *>(p.logits) + ((size_t)p.B * p.W - 1) * p.ld + p.V);
  const T *x = static_cast<const T *>(p.logits) + row * p.ld;
  const int off = SHIFT ? static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15) : 0;
  const int first = id % parts * tiles * kTile, left = (p.V - first + kTile - 1) / kTile, n_tiles = min(tiles, left);
  Granule<T> next[N];
  u64 best = 0;                      // lane i: the i-th of the list
  int count = 0;                     // keys collected
  float cut = -INFINITY, top = -INFINITY, ref = -INFINITY, sum = 0.f;
#pragma unroll 1
  for (int t = -1; t < n_tiles; ++t) {
    Granule<T> f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = next[i];
    const int v0 = first + t * kTile + lane * E;  // element e of the lane's i-th granule is v0 + i * 32 * E + e
    if (t + 1 < n_tiles) {
#pragma unroll
      for (int i = 0; i < N; ++i) next[i].template load<SHIFT>(x, v0 + kTile + i * 32 * E, p.V, off, lo, hi);
    }
    if (t < 0) continue;
    float most[N], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      most[i] = f[i].max();
      m = max_nan(m, most[i]);
    }
    top = max_nan(top, m);
    const unsigned mine = ordered(isnan(m) ? INFINITY : m + 0.f);
    const float high = unordered(__reduce_max_sync(~0u, mine));
    if (t == 0) cut = unordered(__shfl_sync(~0u, sorted(mine, lane), p.K - 1));
    if (high > ref + 64.f || ref == -INFINITY) {  // the first value; later only where the sum could overflow
      sum *= high < INFINITY && ref > -INFINITY ? expf(ref - high) : 0.f;
      ref = high;
    }
    if (ref > -INFINITY) {
      float g[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float h[E];
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = sm100::ex2((f[i][e] - ref) * kLog2e);
#pragma unroll
        for (int n = E / 2; n > 0; n /= 2)
#pragma unroll
          for (int e = 0; e < n; ++e) h[e] += h[e + n];
        g[i] = h[0];
      }
#pragma unroll
      for (int n = N / 2; n > 0; n /= 2)
#pragma unroll
        for (int i = 0; i < n; ++i) g[i] += g[i + n];
      sum += g[0];
    }
    if (high < cut) continue;
    int n = 0;  // granules collected, in the order of their elements
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned who = __ballot_sync(~0u, most[i] >= cut && v0 + i * 32 * E < p.V);
      if (who >> lane & 1) {
        const int at = n + __popc(who & ((1u << lane) - 1));
        c.granule[at] = make_uint4(f[i].w[0], f[i].w[1], f[i].w[2], f[i].w[3]);
        c.index[at] = v0 + i * 32 * E;
      }
      n += __popc(who);
    }
    __syncwarp();
#pragma unroll 1
    for (int q0 = 0; q0 < n * E; q0 += 32) {
      const int q = q0 + lane, v = q < n * E ? c.index[q / E] + q % E : p.V;
      float a = -INFINITY;
      if (v < p.V) a = static_cast<float>(reinterpret_cast<const T *>(c.granule)[q]);
      const unsigned who = __ballot_sync(~0u, a >= cut && v < p.V);
      if (who >> lane & 1) c.key[count + __popc(who & ((1u << lane) - 1))] = (u64)ordered(a + 0.f) << 32 | ~static_cast<unsigned>(v);
      count += __popc(who);
      if (count < 32) continue;
      // a warpful into the list
      __syncwarp();
      best = merged(best, sorted(c.key[lane], lane), lane);
      count -= 32;
      const u64 rest = lane < count ? c.key[32 + lane] : 0;
      __syncwarp();
      if (lane < count) c.key[lane] = rest;
      // what comes now has higher indexes than all this: no use for a value equal to the K-th
      const u64 kth = __shfl_sync(~0u, best, p.K - 1);
      if (kth) cut = fmaxf(cut, unordered(min(static_cast<unsigned>(kth >> 32) + 1, ordered(INFINITY))));
    }
    __syncwarp();
  }
  __syncwarp();
  if (count) best = merged(best, sorted(lane < count ? c.key[lane] : 0, lane), lane);
  if (lane < p.K) keys[(size_t)id * p.K + lane] = best;
  double all = sum;
#pragma unroll 1
  for (int d = 16; d > 0; d /= 2) all += __shfl_xor_sync(~0u, all, d);
  const bool bad = __any_sync(~0u, isnan(top) || top == INFINITY);
  if (lane == 0) part[id] = {bad || ref == -INFINITY ? 0. : all, ref, bad};
}

__device__ __forceinline__ u64 ordered(double x) {
  const long long b = __double_as_longlong(x);
  return static_cast<u64>(b ^ (b >> 63 & 0x7fffffffffffffffll)) ^ 0x8000000000000000ull;
}
__device__ __forceinline__ double unordered(u64 u) {
  const long long b = static_cast<long long>(u ^ 0x8000000000000000ull);
  return __longlong_as_double(b ^ (b >> 63 & 0x7fffffffffffffffll));
}

// The natural logarithm of a sum, to about 1e-11: x = 2^k m, 1 <= m < 2, and with c the middle of m's 32nd of that
// range log m = log c + log1p(m / c - 1), a series in |r| <= 1/64. Few 64-bit instructions, which are slow on this
// chip. kLogs holds 1 / c and -log(1 / c).
__constant__ double2 kLogs[32] = {
    {0.9846153846153847, 0.015504186535965199}, {0.9552238805970149, 0.04580953603129422}, {0.927536231884058, 0.07522342123758752},
    {0.9014084507042254, 0.10379679368164355}, {0.8767123287671232, 0.13157635778871932}, {0.8533333333333334, 0.15860503017663852},
    {0.8311688311688312, 0.18492233849401193}, {0.810126582278481, 0.21056476910734964}, {0.7901234567901234, 0.23556607131276697},
    {0.7710843373493976, 0.259957524436926}, {0.7529411764705882, 0.2837681731306446}, {0.735632183908046, 0.3070250352949119},
    {0.7191011235955056, 0.32975328637246804}, {0.7032967032967034, 0.3519764231571781}, {0.6881720430107527, 0.373716409793584},
    {0.6736842105263158, 0.394993808240869}, {0.6597938144329897, 0.415827895143711}, {0.6464646464646465, 0.43623676677491796},
    {0.6336633663366337, 0.4562374334815876}, {0.6213592233009708, 0.475845904869964}, {0.6095238095238096, 0.4950772667978514},
    {0.5981308411214953, 0.5139457511022344}, {0.5871559633027523, 0.5324647988694717}, {0.5765765765765766, 0.5506471179526623},
    {0.5663716814159292, 0.5685047353526688}, {0.5565217391304348, 0.5860490450035782}, {0.5470085470085471, 0.6032908514380841},
    {0.5378151260504201, 0.6202404097518576}, {0.5289256198347108, 0.6369074622370692}, {0.5203252032520326, 0.6533012720127456},
    {0.512, 0.6694306539426292}, {0.5039370078740157, 0.6853040030989195}};
__device__ __forceinline__ double log_of(double x) {
  const long long b = __double_as_longlong(x);
  const int k = static_cast<int>(b >> 52) - 1023, i = static_cast<int>(b >> 47) & 31;
  const double m = __longlong_as_double((b & 0xfffffffffffffll) | 0x3ff0000000000000ll);
  const double r = fma(m, kLogs[i].x, -1.0);
  const float s = static_cast<float>(r);
  const float tail = s * s * fmaf(s, fmaf(s, fmaf(s, 0.2f, -0.25f), 1.f / 3), -0.5f);
  return fma(k, 0.69314718055994531, kLogs[i].y) + (r + tail);
}

constexpr int kSelectThreads = 256, kSelectWarps = kSelectThreads / 32;
constexpr int kHeld = 2048;  // candidates that are held in shared memory
constexpr int kList = 256;   // candidates that the bound may leave

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const BeamSelect p, int parts, const FastDiv by_parts,
                                                                const FastDiv by_each, const FastDiv by_V,
                                                                const Part *part, const u64 *keys) {
  __shared__ double logs[kMaxBeams];  // of each beam's sum of exp(x - top); NaN: its candidates have no value
  __shared__ double totals[kMaxBeams];
  __shared__ float tops[kMaxBeams];
  __shared__ u64 bounds[kSelectWarps];
  __shared__ Key128 list[kList];
  __shared__ u64 held[kHeld];
  __shared__ int count;
  wait_for_stream();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float *scores = p.scores + b * p.W;
  const unsigned char *done = p.done ? p.done + b * p.W : nullptr;
  const int each = parts * p.K, lists = p.W * parts, all = p.W * each;
  const u64 *mine = keys + (size_t)b * all;
  if (tid == 0) count = 0;
  if (all <= kHeld)
    for (int i = tid; i < all; i += kSelectThreads) held[i] = mine[i];  // (an ended beam's are not looked at)
  for (int w = warp; w < p.W; w += kSelectWarps) {
    if (done && done[w]) continue;
    const Part *s = part + (size_t)(b * p.W + w) * parts;
    float m = -INFINITY;
    bool bad = false;
    for (int i = lane; i < parts; i += 32) {
      if (s[i].sum > 0) m = fmaxf(m, s[i].ref);
      bad |= s[i].bad != 0;
    }
#pragma unroll 1
    for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
    double sum = 0;
    if (!__any_sync(~0u, bad) && m > -INFINITY) {
      for (int i = lane; i < parts; i += 32)
        if (s[i].sum > 0) sum += s[i].sum * expf(s[i].ref - m);
#pragma unroll 1
      for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(~0u, sum, d);
    }
    if (lane == 0) {
      totals[w] = sum;
      tops[w] = m;
    }
  }
  __syncthreads();
  if (tid < p.W) {
    const bool value = !(done && done[tid]) && totals[tid] > 0 && isfinite(scores[tid]);
    logs[tid] = value ? log_of(totals[tid]) : CUDART_NAN;
  }
  __syncthreads();
  const u64 none = ordered(-(double)INFINITY);
  // candidate at = j * K + r of beam w, the r-th of part j; each part's come in descending order
  auto candidate = [&](int w, int at) -> Key128 {
    if (done && done[w]) {
      // eos, and the first tokens besides it without a value
      if (at == 0) return {isfinite(scores[w]) ? ordered((double)scores[w]) : none, ~static_cast<unsigned>(w * p.V + p.eos)};
      if (at < p.K && at < p.V) return {none, ~static_cast<unsigned>(w * p.V + at - (at <= p.eos))};
      return {0, 0};
    }
    if (isnan(logs[w])) return at < p.K && at < p.V ? Key128{none, ~static_cast<unsigned>(w * p.V + at)} : Key128{0, 0};
    const u64 c = all <= kHeld ? held[w * each + at] : mine[w * each + at];
    if (!c) return {0, 0};
    // (not x - (top + log): a top near the type's limits would swallow the log)
    const double x = (double)scores[w] + (((double)unordered(static_cast<unsigned>(c >> 32)) - tops[w]) - logs[w]);
    return {ordered(x), ~(static_cast<unsigned>(w * p.V) + ~static_cast<unsigned>(c))};
  };
  // as in a part: the K-th of the lists' first candidates bounds what can be among the K best
  u64 head = 0;
  for (int i = tid; i < lists; i += kSelectThreads) {
    unsigned w, j;
    by_parts.split(i, w, j);
    head = max(head, candidate(w, j * p.K).score);
  }
  const u64 order = sorted(head, lane);
  if (lane == p.K - 1) bounds[warp] = order;
  __syncthreads();
  u64 low = 1;
#pragma unroll
  for (int i = 0; i < kSelectWarps; ++i) low = max(low, bounds[i]);
  for (int i = tid; i < lists; i += kSelectThreads) {
    unsigned w, j;
    by_parts.split(i, w, j);
    for (int r = 0; r < p.K; ++r) {
      const Key128 k = candidate(w, j * p.K + r);
      if (k.score < low) break;
      const int at = atomicAdd(&count, 1);
      if (at < kList) list[at] = k;
    }
  }
  __syncthreads();
  const int n = count;
  // these, or all where there are too many
  Key128 best = {0, 0};
  const int some = n > kList ? all : n;
#pragma unroll 1
  for (int i0 = warp * 32; i0 < some; i0 += kSelectThreads) {
    const int i = i0 + lane;
    Key128 k = {0, 0};
    if (i < some && n > kList) {
      unsigned w, at;
      by_each.split(i, w, at);
      k = candidate(w, at);
    } else if (i < some) {
      k = list[i];
    }
    k = sorted(k, lane);
    best = i0 < kSelectThreads ? k : merged(best, k, lane);
  }
#pragma unroll 1
  for (int half = kSelectWarps / 2; half > 0; half /= 2) {
    if (n <= half * 32) continue;  // (nothing in those warps)
    __syncthreads();
    if (warp >= half && warp < 2 * half) list[tid - half * 32] = best;
    __syncthreads();
    if (warp < half) best = merged(best, list[tid], lane);
  }
  if (tid < p.K) {
    unsigned w, v;
    by_V.split(~best.rank, w, v);
    const size_t out = (size_t)b * p.K + tid;
    p.scores_out[out] = static_cast<float>(unordered(best.score));
    p.parent[out] = w;
    p.token[out] = v;
  }
}

// How the rows are cut: granules of a lane, parts of a row, tiles of a part.
struct Cut {
  int n, parts, tiles;
};
// Parts for all the warps that the SMs hold (20 each), of small tiles where there is less; but no more than kLists for
// a request, which the second kernel goes through.
constexpr int kLists = 512;
Cut cut_of(const BeamSelect &p) {
  const long long rows = (long long)p.B * p.W, e = p.f32 ? 4 : 8, warps = 20ll * std::max(sm_count(), 1);
  Cut c = {4, 0, 0};
  while (c.n > 1 && rows * (p.V / (32 * c.n * e)) < warps) c.n /= 2;
  const long long all = (p.V - 1) / (32 * c.n * e) + 1;  // tiles of a row
  c.tiles = static_cast<int>(std::max(1ll, (rows * all + warps - 1) / warps));
  c.tiles = static_cast<int>(std::max<long long>(c.tiles, (all * p.W - 1) / kLists + 1));
  c.tiles = static_cast<int>(std::min<long long>(c.tiles, all));
  c.parts = static_cast<int>((all - 1) / c.tiles + 1);
  return c;
}

template <typename T, int N>
cudaError_t launch_n(const BeamSelect &p, const Cut &c, Part *part, u64 *keys, cudaStream_t stream) {
  const int total = p.B * p.W * c.parts;
  const dim3 grid((total - 1) / kWarps + 1);
  const bool wide = (reinterpret_cast<uintptr_t>(p.logits) & 15) == 0 && p.ld * sizeof(T) % 16 == 0;
  return launch_early(wide ? part_kernel<T, N, false> : part_kernel<T, N, true>, grid, kThreads, 0, stream, p, total, c.parts,
                      c.tiles, part, keys);
}

template <typename T> cudaError_t launch(const BeamSelect &p, const Cut &c, Part *part, u64 *keys, cudaStream_t stream) {
  return c.n == 1   ? launch_n<T, 1>(p, c, part, keys, stream)
         : c.n == 2 ? launch_n<T, 2>(p, c, part, keys, stream)
                    : launch_n<T, 4>(p, c, part, keys, stream);
}

int fail(const char *what, cudaError_t e) {
  set_error("la_beam_select: %s: %s", what, cudaGetErrorString(e));
  return LA_ERR_CUDA;
}

}  // namespace

int launch_beam_select(const BeamSelect &p, cudaStream_t stream) {
  const Cut c = cut_of(p);
  const size_t parts = (size_t)p.B * p.W * c.parts;
  uint8_t *ws = nullptr;
  cudaMemPool_t pool = library_pool();
  if (!pool) return fail("could not create the workspace pool", cudaGetLastError());
  cudaError_t e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), parts * (sizeof(Part) + sizeof(u64) * p.K), pool,
                                          stream);
  if (e != cudaSuccess) return fail("workspace allocation failed", e);
  Part *part = reinterpret_cast<Part *>(ws);
  u64 *keys = reinterpret_cast<u64 *>(part + parts);
  e = p.f32 ? launch<float>(p, c, part, keys, stream) : launch<__nv_bfloat16>(p, c, part, keys, stream);
  if (e == cudaSuccess)
    e = launch_early(select_kernel, dim3(p.B), kSelectThreads, 0, stream, p, c.parts, FastDiv(c.parts), FastDiv(c.parts * p.K),
                     FastDiv(p.V), part, keys);
  const cudaError_t f = cudaFreeAsync(ws, stream);
  if (e == cudaSuccess) e = f;
  return e == cudaSuccess ? LA_OK : fail("launch failed", e);
}

}  // namespace la
