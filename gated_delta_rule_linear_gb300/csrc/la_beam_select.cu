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
//
// Code. Both kernels are short, and what they run once or twice is rolled up:
// fetching straight-line code takes longer than running it (with all sorts
// unrolled the first kernel stalled for instructions four times as often as for
// memory).
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>

#include "la_serve_internal.h"
#include "la_sm100.cuh"

namespace la {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 128, kWarps = kThreads / 32;  // of the first kernel
constexpr int kStages = 3;                             // tiles of a warp that are on their way or being read
constexpr float kLog2e = 1.44269504f;

// What the first kernel leaves of a part; its K keys are in an array of their own.
struct Part {
  double sum;   // of exp(x - ref); 0: no value in the part, or a bad one
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

// Bitonic exchange with the lane j away; `top` keeps the larger one.
template <typename Word>
__device__ __forceinline__ Word exchange(Word k, int j, bool top) {
  const Word o = __shfl_xor_sync(~0u, k, j);
  return (o > k) == top ? o : k;
}
// A warp's keys in descending order over its lanes.
template <typename Word>
__device__ __forceinline__ Word sorted(Word k, int lane) {
#pragma unroll 1
  for (int n = 2; n <= 32; n *= 2)
#pragma unroll 1
    for (int j = n / 2; j > 0; j /= 2) k = exchange(k, j, ((lane & n) == 0) == ((lane & j) == 0));
  return k;
}
// The 32 largest of two such lists, as one.
__device__ __forceinline__ u64 merged(u64 a, u64 b, int lane) {
  a = max(a, __shfl_xor_sync(~0u, b, 31));
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
  static constexpr unsigned kNone = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -infinity
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
  // The 16 bytes `off` behind *at; `left` elements of it are in the row, the others become -infinity.
  __device__ __forceinline__ void load(const uint4 *at, int off, int left) {
    uint4 a = *at;
    if (off) {
      uint4 b = at[1];
      if (off & 8) a = make_uint4(a.z, a.w, b.x, b.y), b = make_uint4(b.z, b.w, b.z, b.w);
      if (off & 4) a = make_uint4(a.y, a.z, a.w, b.x), b.x = b.y;
      if (off & 2)
        a = make_uint4(__funnelshift_r(a.x, a.y, 16), __funnelshift_r(a.y, a.z, 16), __funnelshift_r(a.z, a.w, 16),
                       __funnelshift_r(a.w, b.x, 16));
    }
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    if (left < E) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int inside = left - i * E / 4;  // elements of this word
        if (inside <= 0) w[i] = kNone;
        else if (sizeof(T) == 2 && inside == 1) w[i] = (w[i] & 0xffffu) | (kNone & 0xffff0000u);
      }
    }
  }
};

// A warp's shared memory: tiles as they are in memory (one granule more than a tile, for rows that start anywhere),
// which of a tile's granules have an element above the cut, and such elements' keys.
template <int N> struct Work {
  uint4 tile[kStages][32 * N + 1];
  u64 key[64];
  unsigned char index[32 * N];
};

// A warp, one part: `tiles` tiles of 32 * N granules.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads) part_kernel(const BeamSelect p, int total, int parts, int tiles, Part *part,
                                                        u64 *keys) {
  constexpr int E = Granule<T>::E, kTile = 32 * N * E;
  __shared__ Work<N> works[kWarps];
  wait_for_stream();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int id = blockIdx.x * kWarps + warp;
  if (id >= total) return;
  const int row = id / parts;
  if (p.done && p.done[row]) return;
  Work<N> &c = works[warp];
  const T *x = static_cast<const T *>(p.logits) + row * p.ld;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15);
  const int first = id % parts * tiles * kTile, n_tiles = min(tiles, (p.V - first + kTile - 1) / kTile);
  const char *lo = static_cast<const char *>(p.logits), *end = reinterpret_cast<const char *>(x + p.V);
  auto fetch = [&](int t) {  // whole granules of memory, but nothing in front of the first row or behind this one
    if (t < n_tiles) {
      const char *src = reinterpret_cast<const char *>(x + first + t * kTile) - off;
      uint4 *dst = c.tile[t % kStages];
#pragma unroll 1
      for (int i = lane; i < 32 * N + (off != 0); i += 32) {
        const char *at = src + i * 16;
        const int there = static_cast<int>(min(max((long long)(end - at), 0ll), 16ll));
        if (at >= lo) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(dst + i)), "l"(there ? at : lo),
                       "r"(there)
                       : "memory");
        } else {
#pragma unroll 1
          for (int e = off / (int)sizeof(T); e * (int)sizeof(T) < there; ++e)
            reinterpret_cast<T *>(dst + i)[e] = reinterpret_cast<const T *>(at)[e];
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int t = 0; t < kStages - 1; ++t) fetch(t);
  u64 best = 0;                      // lane i: the i-th of the list
  int count = 0;                     // keys collected
  float cut = -INFINITY, top = -INFINITY, ref = -INFINITY, sum = 0.f;
#pragma unroll 1
  for (int t = 0; t < n_tiles; ++t) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();
    fetch(t + kStages - 1);
    const uint4 *tile = c.tile[t % kStages];
    const int v0 = first + t * kTile;  // element e of the lane's i-th granule is v0 + (i * 32 + lane) * E + e
    Granule<T> f[N];
    float most[N], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      f[i].load(tile + i * 32 + lane, off, p.V - v0 - (i * 32 + lane) * E);
      most[i] = f[i].max();
      m = max_nan(m, most[i]);
    }
    top = max_nan(top, m);
    const unsigned mine = ordered(isnan(m) ? INFINITY : m + 0.f);  // (+ 0: one zero)
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
      const unsigned who = __ballot_sync(~0u, most[i] >= cut && v0 + (i * 32 + lane) * E < p.V);
      if (who >> lane & 1) c.index[n + __popc(who & ((1u << lane) - 1))] = static_cast<unsigned char>(i * 32 + lane);
      n += __popc(who);
    }
    __syncwarp();
#pragma unroll 1
    for (int q0 = 0; q0 < n * E; q0 += 32) {
      const int q = q0 + lane, j = q < n * E ? c.index[q / E] * E + q % E : kTile, v = v0 + j;
      const bool in = j < kTile && v < p.V;
      float a = -INFINITY;
      if (in) a = static_cast<float>(reinterpret_cast<const T *>(tile)[j + off / (int)sizeof(T)]);
      const unsigned who = __ballot_sync(~0u, in && a >= cut);
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

// A candidate: its score in the order of unsigned integers, then the order of w * V + v, reversed. 0, 0: none.
struct Candidate {
  u64 score;
  unsigned rank;  // ~(w * V + v)
};
__device__ __forceinline__ bool above(const Candidate &a, const Candidate &b) {
  return a.score > b.score || (a.score == b.score && a.rank > b.rank);
}
__device__ __forceinline__ u64 ordered(double x) {
  const long long b = __double_as_longlong(x);
  return static_cast<u64>(b ^ (b >> 63 & 0x7fffffffffffffffll)) ^ 0x8000000000000000ull;
}
__device__ __forceinline__ double unordered(u64 u) {
  const long long b = static_cast<long long>(u ^ 0x8000000000000000ull);
  return __longlong_as_double(b ^ (b >> 63 & 0x7fffffffffffffffll));
}

// The natural logarithm of a sum, to about 1e-9: x = 2^k m, 1/sqrt2 < m < sqrt2, and with s = (m - 1) / (m + 1)
// log m = 2 (s + s^3 / 3 + s^5 / 5 + ..), |s| < 0.172. s is two float32 parts, the quotient and its remainder; the
// other terms are below 0.002 of it and float32. (64-bit instructions are few on this chip.)
__device__ __forceinline__ double log_of(double x) {
  long long b = __double_as_longlong(x);
  int k = static_cast<int>(b >> 52) - 1023;
  const bool upper = (b >> 32 & 0xfffff) >= 0x6a09e;  // m >= sqrt2: halved
  k += upper;
  const double m = __longlong_as_double((b & 0xfffffffffffffll) | (upper ? 0x3fe0000000000000ll : 0x3ff0000000000000ll));
  const float hi = static_cast<float>(m), lo = static_cast<float>(m - hi);
  const float num = hi - 1.f, den = hi + 1.f;  // num exact; den's rounding is carried along
  const float den_lo = (hi - (den - 1.f)) + lo;
  const float s = num / den, s_lo = (fmaf(-s, den, num) + lo - s * den_lo) / den;
  const float z = s * s;
  const float tail = s * z * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 11, 1.f / 9), 1.f / 7), 1.f / 5), 1.f / 3);
  return fma((double)k, 0.69314718055994531, 2 * ((double)s + (s_lo + tail)));
}

constexpr int kSelectThreads = 256, kSelectWarps = kSelectThreads / 32;
constexpr int kHeld = 2048;  // candidates that are held in shared memory
constexpr int kList = 256;   // candidates that the bound may leave

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const BeamSelect p, int parts, const FastDiv by_each,
                                                                const FastDiv by_V, const Part *part, const u64 *keys) {
  __shared__ double logs[kMaxBeams];  // of each beam's sum of exp(x - top)
  __shared__ float tops[kMaxBeams];
  __shared__ float base[kMaxBeams];   // about score - log; NaN: its candidates have no value, infinity: it has ended
  __shared__ float bounds[kSelectWarps];
  __shared__ Candidate list[kList];
  __shared__ u64 held[kHeld];
  __shared__ int count;
  wait_for_stream();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float *scores = p.scores + b * p.W;
  const int each = parts * p.K, all = p.W * each;
  const u64 *mine = keys + (size_t)b * all;
  if (all <= kHeld)
#pragma unroll 1
    for (int i = tid; i < all; i += kSelectThreads) held[i] = mine[i];  // (those of ended and worthless beams are not used)
#pragma unroll 1
  for (int w = warp; w < p.W; w += kSelectWarps) {
    const Part *s = part + (size_t)(b * p.W + w) * parts;
    const bool done = p.done && p.done[b * p.W + w];
    const float score = scores[w];
    float m = -INFINITY;
    double sum = 0;
    bool bad = false;
#pragma unroll 1
    for (int i = lane; i < parts && !done; i += 32) {  // sums to their largest reference so far
      const Part a = s[i];
      bad |= a.bad != 0;
      if (!(a.sum > 0)) continue;
      const float top = fmaxf(m, a.ref);
      sum = sum * expf(m - top) + a.sum * expf(a.ref - top);
      m = top;
    }
    bad = __any_sync(~0u, bad);
#pragma unroll 1
    for (int d = 16; d > 0; d /= 2) {
      const float o = __shfl_xor_sync(~0u, m, d), top = fmaxf(m, o);
      const double theirs = __shfl_xor_sync(~0u, sum, d);
      if (top > -INFINITY) sum = (m == top ? sum : sum * expf(m - top)) + (o == top ? theirs : theirs * expf(o - top));
      m = top;
    }
    if (lane == 0) {
      const bool value = !bad && sum > 0 && isfinite(score);
      const double log = value ? log_of(sum) : 0;
      logs[w] = log;
      tops[w] = m;
      base[w] = done ? INFINITY : value ? static_cast<float>(score - log) : CUDART_NAN_F;
    }
  }
  if (tid == 0) count = 0;
  __syncthreads();
  // Candidate at = j * K + r of beam w is the r-th of part j; an ended beam's first one is eos, its others and those of a
  // beam without values the first tokens, without a value.
  auto key = [&](int w, int at) { return all <= kHeld ? held[w * each + at] : mine[w * each + at]; };
  auto rough = [&](int w, int at) -> float {  // its score, to float32; NaN: none
    const float c = base[w];
    if (c == INFINITY) return at == 0 && isfinite(scores[w]) ? scores[w] : at < p.K && at < p.V ? -INFINITY : CUDART_NAN_F;
    if (isnan(c)) return at < p.K && at < p.V ? -INFINITY : CUDART_NAN_F;
    const u64 k = key(w, at);
    return k ? c + (unordered(static_cast<unsigned>(k >> 32)) - tops[w]) : CUDART_NAN_F;
  };
  auto candidate = [&](int w, int at) -> Candidate {
    const u64 none = ordered(-(double)INFINITY);
    const unsigned first = static_cast<unsigned>(w * p.V);
    if (base[w] == INFINITY && at == 0) return {isfinite(scores[w]) ? ordered((double)scores[w]) : none, ~(first + p.eos)};
    if (base[w] == INFINITY) return {none, ~(first + at - (at <= p.eos))};
    if (isnan(base[w])) return {none, ~(first + at)};
    const u64 k = key(w, at);
    // (not x - (top + log): a top near the type's limits would swallow the log)
    const double x = (double)scores[w] + (((double)unordered(static_cast<unsigned>(k >> 32)) - tops[w]) - logs[w]);
    return {ordered(x), ~(first + ~static_cast<unsigned>(k))};
  };
  // As in a part: the K-th largest of a warp's lanes bounds what can be among the K best. Lanes take the parts' first
  // candidates; all in float32, with what that may be off taken from the bound.
  float head = -INFINITY;
  bool any = false;
#pragma unroll 1
  for (int i = tid; i < p.W * parts; i += kSelectThreads) {
    unsigned w, at;
    by_each.split(i * p.K, w, at);
    const float c = rough(w, at);
    if (!isnan(c)) head = fmaxf(head, c), any = true;
  }
  const unsigned order = sorted(any ? ordered(head) : 0u, lane);
  if (lane == p.K - 1) bounds[warp] = order ? unordered(order) : -INFINITY;
  __syncthreads();
  float low = bounds[0], size = 0.f;
#pragma unroll 1
  for (int i = 1; i < kSelectWarps; ++i) low = fmaxf(low, bounds[i]);
#pragma unroll 1
  for (int w = 0; w < p.W; ++w)
    if (isfinite(base[w])) size = fmaxf(size, fabsf(base[w]));
  low -= 1e-6f * (fabsf(low) + size);  // (three roundings of up to 2^-24)
#pragma unroll 1
  for (int i = tid; i < all; i += kSelectThreads) {
    unsigned w, at;
    by_each.split(i, w, at);
    if (!(rough(w, at) >= low)) continue;
    const int n = atomicAdd(&count, 1);
    if (n < kList) list[n] = candidate(w, at);
  }
  __syncthreads();
  const int n = count;
  auto put = [&](int r, const Candidate &k) {
    unsigned w, v;
    by_V.split(~k.rank, w, v);
    const size_t out = (size_t)b * p.K + r;
    p.scores_out[out] = static_cast<float>(unordered(k.score));
    p.parent[out] = w;
    p.token[out] = v;
  };
  if (n <= kList) {  // a candidate's rank: how many are above it
    if (tid < n) {
      const Candidate k = list[tid];
      int r = 0;
#pragma unroll 4
      for (int i = 0; i < n; ++i) r += above(list[i], k);
      if (r < p.K) put(r, k);
    }
    return;
  }
  // too many that are equal: the next one below the last, K times
  Candidate last = {~0ull, ~0u};
#pragma unroll 1
  for (int r = 0; r < p.K; ++r) {
    Candidate k = {0, 0};
#pragma unroll 1
    for (int i = tid; i < all; i += kSelectThreads) {
      unsigned w, at;
      by_each.split(i, w, at);
      if (isnan(rough(w, at))) continue;
      const Candidate o = candidate(w, at);
      if (above(last, o) && above(o, k)) k = o;
    }
#pragma unroll 1
    for (int d = 16; d > 0; d /= 2) {
      const Candidate o = {__shfl_xor_sync(~0u, k.score, d), __shfl_xor_sync(~0u, k.rank, d)};
      if (above(o, k)) k = o;
    }
    __syncthreads();
    if (lane == 0) list[warp] = k;
    __syncthreads();
    last = list[0];
#pragma unroll 1
    for (int i = 1; i < kSelectWarps; ++i)
      if (above(list[i], last)) last = list[i];
    if (tid == 0) put(r, last);
  }
}

// How the rows are cut: granules of a lane, parts of a row, tiles of a part.
struct Cut {
  int n, parts, tiles;
};
// Parts for all the warps that the SMs hold (20 each), of small tiles where there is less; but no more than kLists for
// a request, which the second kernel goes through.
constexpr int kLists = 256;
Cut cut_of(const BeamSelect &p) {
  const long long rows = (long long)p.B * p.W, e = p.f32 ? 4 : 8, warps = 20ll * std::max(sm_count(), 1);
  Cut c = {4, 0, 0};
  while (c.n > 1 && rows * (p.V / (32 * c.n * e)) < warps) c.n /= 2;
  const long long all = (p.V - 1) / (32 * c.n * e) + 1;  // tiles of a row
  long long tiles = std::max({1ll, (rows * all + warps - 1) / warps, (all * p.W - 1) / kLists + 1});
  c.tiles = static_cast<int>(std::min(tiles, all));
  c.parts = static_cast<int>((all - 1) / c.tiles + 1);
  return c;
}

template <typename T, int N>
cudaError_t launch_n(const BeamSelect &p, const Cut &c, Part *part, u64 *keys, cudaStream_t stream) {
  const int total = p.B * p.W * c.parts;
  const dim3 grid((total - 1) / kWarps + 1);
  return launch_early(part_kernel<T, N>, grid, kThreads, 0, stream, p, total, c.parts, c.tiles, part, keys);
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
    e = launch_early(select_kernel, dim3(p.B), kSelectThreads, 0, stream, p, c.parts, FastDiv(c.parts * p.K), FastDiv(p.V),
                     part, keys);
  const cudaError_t f = cudaFreeAsync(ws, stream);
  if (e == cudaSuccess) e = f;
  return e == cudaSuccess ? LA_OK : fail("launch failed", e);
}

}  // namespace la
