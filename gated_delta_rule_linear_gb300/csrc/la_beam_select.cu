// Beam search's selection: of W beams with V continuations each, the K best by
// c(w, v) = scores[w] + x[w][v] - log sum_u exp x[w][u].
//
// Bound by reading the logits once. Two kernels. In the first a warp takes a part
// of a row: the K best of it, by logits (inside a row the order of c is that of
// x), and the part's share of the sum. The second takes a request: the log of
// each beam's sum, the parts' candidates' scores in 64 bits, and their K best.
//
// K best of a part. No element below the K-th largest of the lanes' largest can be
// among the K best, which leaves little more than K of them: the warp goes over
// its part once for the lanes' largest and the sum, collects what passes this cut,
// and sorts it. The part stays in shared memory meanwhile. Keys are value and
// index together, so that the order is right for equal logits (bfloat16 has
// many). Warps do not wait for one another.
//
// The sum. exp(x - r) with the largest value so far as the reference r (an
// exponent is rounded to 2^-24 of itself: of those that count, none may be
// large). In pairs inside a lane's 16 bytes, in two float32 across lanes. Which
// elements meet in which order depends on their index alone, not on where a row
// lies, so that two beams with the same logits get the same sum; rows that do not
// start at 16 bytes are shifted into place for this.
//
// Code. Both kernels are short, and what they run once or twice is rolled up:
// fetching straight-line code takes longer than running it (with all sorts
// unrolled the first kernel waited for instructions more than for memory).
//
// 32 requests of 8 beams of 50257 bfloat16 logits (25.7 MB, rows at odd places):
// 18.5 us, the first kernel 12.5 and bound by its instructions (the shifts, exp2 and
// what a part costs besides), the second 6 and bound by the latency of its steps;
// one request of 4 beams of 32000 float32 logits 9 us.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>

#include "la_f32x2.cuh"
#include "la_serve_internal.h"
#include "la_sm100.cuh"

namespace la {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 64, kWarps = kThreads / 32;  // of the first kernel
constexpr int kCoarse = 16;          // up to so many of a part by the lanes' largest values alone
constexpr float kLog2e = 1.44269504f;

// What the first kernel leaves of a part; its K keys are in an array of their own.
struct Part {
  float2 sum;   // of exp(x - ref), as two float32; 0: no value in the part, or a bad one
  float ref;
  int bad;      // it has a NaN or +infinity
};

// Sums of two float32 each (Knuth's two-sum and a renormalisation).
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  const float s = a.x + b.x, t = s - a.x;
  const float e = ((a.x - (s - t)) + (b.x - t)) + (a.y + b.y), r = s + e;
  return make_float2(r, e - (r - s));
}
__device__ __forceinline__ float2 mul2(float2 a, float f) {
  const float s = a.x * f;
  return make_float2(s, fmaf(a.x, f, -s) + a.y * f);
}

// The order of floats (no NaN) as that of unsigned integers.
__device__ __forceinline__ unsigned ordered(float x) {
  const int b = __float_as_int(x);
  return static_cast<unsigned>(b ^ (b >> 31 & 0x7fffffff)) ^ 0x80000000u;
}
__device__ __forceinline__ float unordered(unsigned u) {
  const int b = static_cast<int>(u ^ 0x80000000u);
  return __int_as_float(b ^ (b >> 31 & 0x7fffffff));
}

// A candidate: its score in the order of unsigned integers, then the order of w * V + v, reversed. 0, 0: none.
struct Candidate {
  u64 score;
  unsigned rank;  // ~(w * V + v)
};
__device__ __forceinline__ bool operator>(const Candidate &a, const Candidate &b) {
  return a.score > b.score || (a.score == b.score && a.rank > b.rank);
}

template <typename Word> __device__ __forceinline__ Word of_lane(Word k, int x) { return __shfl_xor_sync(~0u, k, x); }
__device__ __forceinline__ Candidate of_lane(const Candidate &k, int x) { return {of_lane(k.score, x), of_lane(k.rank, x)}; }

// Bitonic exchange with the lane j away; `top` keeps the larger one.
template <typename Word>
__device__ __forceinline__ Word exchange(Word k, int j, bool top) {
  const Word o = of_lane(k, j);
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
template <typename Word>
__device__ __forceinline__ Word merged(Word a, Word b, int lane) {
  const Word o = of_lane(b, 31);
  if (o > a) a = o;
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

__device__ __forceinline__ void copy16(uint4 *dst, const char *src, int bytes) {  // the rest becomes zero
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
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
  // -infinity for the elements behind the first `left`.
  __device__ __forceinline__ void end(int left) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int inside = left - i * E / 4;  // elements of this word
      if (inside <= 0) w[i] = kNone;
      else if (sizeof(T) == 2 && inside == 1) w[i] = (w[i] & 0xffffu) | (kNone & 0xffff0000u);
    }
  }
};

// U granules 32 apart, each the 16 bytes `OFF` behind at[32 * i].
template <typename T, int U, int OFF> __device__ __forceinline__ void load_at(Granule<T> (&f)[U], const uint4 *at) {
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint4 a = at[32 * i], b = OFF ? at[32 * i + 1] : a;
    const unsigned in[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      f[i].w[k] = OFF & 2 ? __funnelshift_r(in[k + OFF / 4], in[k + OFF / 4 + 1], 16) : in[k + OFF / 4];
  }
}
template <typename T, int U> __device__ __forceinline__ void load_off(Granule<T> (&f)[U], const uint4 *at, int off) {
  switch (off) {
    case 0: load_at<T, U, 0>(f, at); break;
    case 4: load_at<T, U, 4>(f, at); break;
    case 8: load_at<T, U, 8>(f, at); break;
    case 12: load_at<T, U, 12>(f, at); break;
    default:
      if constexpr (sizeof(T) == 2) {
        if (off == 2) load_at<T, U, 2>(f, at);
        else if (off == 6) load_at<T, U, 6>(f, at);
        else if (off == 10) load_at<T, U, 10>(f, at);
        else load_at<T, U, 14>(f, at);
      }
  }
}

// A warp's shared memory: its part as it is in memory (one granule more, for rows that start anywhere), each granule's
// largest value, which granules pass the cut, and keys.
template <int G> struct Work {
  uint4 data[32 * G + 1];
  float most[32 * G];
  unsigned short index[32 * G];
  u64 key[64];
};

// A warp, one part: 32 * G granules of a row.
template <typename T, int G>
__global__ void __launch_bounds__(kThreads) part_kernel(const BeamSelect p, int total, int parts, Part *part, u64 *keys) {
  constexpr int E = Granule<T>::E, kPart = 32 * G * E, U = G < 4 ? G : 4;  // granules of a lane at a time
  extern __shared__ __align__(16) uint8_t smem[];
  wait_for_stream();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int id = blockIdx.x * kWarps + warp;
  if (id >= total) return;
  const int row = id / parts;
  if (p.done && p.done[row]) return;
  Work<G> &c = reinterpret_cast<Work<G> *>(smem)[warp];
  const T *x = static_cast<const T *>(p.logits) + row * p.ld;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15);
  const int v0 = id % parts * kPart;  // element e of granule i of the part is v0 + i * E + e
  const char *src = reinterpret_cast<const char *>(x + v0) - off;
  const char *lo = static_cast<const char *>(p.logits), *end = reinterpret_cast<const char *>(x + p.V);
  // whole granules of memory, but nothing in front of the first row or behind this one
  if (src >= lo && src + (32 * G + 1) * 16 <= end) {
    if (off && lane == 0) copy16(c.data + 32 * G, src + 32 * G * 16, 16);
#pragma unroll
    for (int i = 0; i < G; ++i) copy16(c.data + i * 32 + lane, src + (i * 32 + lane) * 16, 16);
  } else {
#pragma unroll 1
    for (int i = lane; i <= 32 * G; i += 32) {
      const char *at = src + i * 16;
      const int there = static_cast<int>(min(max((long long)(end - at), 0ll), 16ll));
      if (there == 0) {  // (no copy of zero bytes: its source would have to be aligned all the same)
        c.data[i] = make_uint4(0, 0, 0, 0);
      } else if (at >= lo) {
        copy16(c.data + i, at, there);
      } else {
#pragma unroll 1
        for (int e = off / (int)sizeof(T); e * (int)sizeof(T) < there; ++e)
          reinterpret_cast<T *>(c.data + i)[e] = reinterpret_cast<const T *>(at)[e];
      }
    }
  }
  float top = -INFINITY, ref = -INFINITY;
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int j = 0; j < G / U; ++j) {
    // all of it: the granule that follows the last lane's is of the next round
    if (j == 0) asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    Granule<T> f[U];
    float m = -INFINITY;
    const int g0 = j * U * 32 + lane;
    load_off<T, U>(f, c.data + g0, off);
    if (p.V - v0 < (j + 1) * U * 32 * E)
#pragma unroll
      for (int i = 0; i < U; ++i) f[i].end(p.V - v0 - (g0 + i * 32) * E);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float most = f[i].max();
      c.most[g0 + i * 32] = most;
      m = max_nan(m, most);
    }
    if (isnan(m)) m = INFINITY;
    top = fmaxf(top, m);
    const float high = unordered(__reduce_max_sync(~0u, ordered(m + 0.f)));  // (+ 0: one zero)
    if (high > ref) {
      sum = mul2(sum, high < INFINITY && ref > -INFINITY ? expf(ref - high) : 0.f);
      ref = high;
    }
    if (ref > -INFINITY) {
      const uint64_t r = f32x2::pair(-ref, -ref), l = f32x2::pair(kLog2e, kLog2e);
      uint64_t g[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        uint64_t h[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          float t[2];
          f32x2::split(f32x2::mul(f32x2::add(f32x2::pair(f[i][2 * e], f[i][2 * e + 1]), r), l), t);
          h[e] = f32x2::pair(sm100::ex2(t[0]), sm100::ex2(t[1]));
        }
#pragma unroll
        for (int n = E / 4; n > 0; n /= 2)
#pragma unroll
          for (int e = 0; e < n; ++e) h[e] = f32x2::add(h[e], h[e + n]);
        g[i] = h[0];
      }
#pragma unroll
      for (int n = U / 2; n > 0; n /= 2)
#pragma unroll
        for (int i = 0; i < n; ++i) g[i] = f32x2::add(g[i], g[i + n]);
      float t[2];
      f32x2::split(g[0], t);
      sum = add2(sum, make_float2(t[0] + t[1], 0.f));
    }
  }
  // the K-th largest of the lanes': the largest again and again for few (8 best as above: 12.5 us, sorted 12.8)
  float cut;
  unsigned order = ordered(top + 0.f), high = 0;
  if (p.K <= 8) {
    unsigned m;
#pragma unroll 1
    for (int gone = 0; gone < p.K;) {
      m = __reduce_max_sync(~0u, order);
      const bool is = order == m;
      gone += __popc(__ballot_sync(~0u, is));
      if (is) order = 0;
      high = max(high, m);
    }
    cut = unordered(m);
  } else {
    order = sorted(order, lane);
    high = __shfl_sync(~0u, order, 0);
    unsigned low = __shfl_sync(~0u, order, p.K - 1);
    // near 32 that is the least of the lanes' and leaves some hundred: from there up by halving while K granules pass (18 x
    // 16 rows of 43624, 32 best: this kernel 28 us without, 19 with; 18 x 12, 24 best 13.6 and 12.9; 32 x 8 of 50257, 16
    // best 14.3 and 16; small parts 22 x 16 of 3830, 32 best, the call: 24 and 27)
#pragma unroll 1
    for (unsigned up = high; G == 8 && p.K > kCoarse && low < up;) {
      const unsigned mid = up - (up - low) / 2;
      const float at = unordered(mid);
      int pass = 0;
#pragma unroll
      for (int i = 0; i < G; ++i) pass += c.most[i * 32 + lane] >= at;
      pass = __reduce_add_sync(~0u, pass);
      if (pass >= p.K) low = mid;
      else up = mid - 1;
      if (pass >= p.K && pass <= p.K + 4) break;
    }
    cut = unordered(low);
  }
  const bool bad = unordered(high) == INFINITY;
  int n = 0;  // granules that pass, in the order of their elements
#pragma unroll 1
  for (int i = 0; i < G && !bad; ++i) {
    const int g = i * 32 + lane;
    const unsigned who = __ballot_sync(~0u, c.most[g] >= cut && v0 + g * E < p.V);
    if (who >> lane & 1) c.index[n + __popc(who & ((1u << lane) - 1))] = static_cast<unsigned short>(g);
    n += __popc(who);
  }
  __syncwarp();
  u64 best = 0;   // lane i: the i-th of the list
  int count = 0;  // keys collected
  bool listed = false;
#pragma unroll 1
  for (int q0 = 0; q0 < n * E; q0 += 32) {
    const int q = q0 + lane, at = q < n * E ? c.index[q / E] * E + q % E : kPart, v = v0 + at;
    const bool in = at < kPart && v < p.V;
    float a = -INFINITY;
    if (in) a = static_cast<float>(reinterpret_cast<const T *>(c.data)[at + off / (int)sizeof(T)]);
    const unsigned who = __ballot_sync(~0u, in && a >= cut);
    if (who >> lane & 1) c.key[count + __popc(who & ((1u << lane) - 1))] = (u64)ordered(a + 0.f) << 32 | ~static_cast<unsigned>(v);
    count += __popc(who);
    if (count <= 32) continue;
    // a warpful into the list
    __syncwarp();
    best = merged(best, sorted(lane < count ? c.key[lane] : 0, lane), lane);
    const u64 rest = 32 + lane < count ? c.key[32 + lane] : 0;
    __syncwarp();
    c.key[lane] = rest;
    count -= 32;
    listed = true;
    __syncwarp();
    // what comes now has higher indexes than all this: no use for a value equal to the K-th
    const u64 kth = __shfl_sync(~0u, best, p.K - 1);
    if (kth) cut = fmaxf(cut, unordered(min(static_cast<unsigned>(kth >> 32) + 1, ordered(INFINITY))));
    if (cut > unordered(high)) break;  // (all equal, or none allowed)
  }
  __syncwarp();
  const u64 mine = lane < count ? c.key[lane] : 0;
  u64 *out = keys + (size_t)id * p.K;
  if (listed) {
    best = merged(best, sorted(mine, lane), lane);
    if (lane < p.K) out[lane] = best;
  } else {  // few, as mostly: a key's rank is the number above it (32 x 8 of 50257, 8 best: this kernel 12.8 us, sorted 14)
    int r = 0;
#pragma unroll 1
    for (int i = 0; i < count; ++i) r += c.key[i] > mine;
    if (lane >= count) r = lane;
    if (r < p.K) out[r] = mine;
  }
#pragma unroll 1
  for (int d = 16; d > 0; d /= 2) sum = add2(sum, make_float2(__shfl_xor_sync(~0u, sum.x, d), __shfl_xor_sync(~0u, sum.y, d)));
  if (lane == 0) part[id] = {bad || ref == -INFINITY ? make_float2(0.f, 0.f) : sum, ref, bad};
}

__device__ __forceinline__ u64 ordered(double x) {
  const long long b = __double_as_longlong(x + 0.0);  // (one zero: scores of ended beams may be either)
  return static_cast<u64>(b ^ (b >> 63 & 0x7fffffffffffffffll)) ^ 0x8000000000000000ull;
}
__device__ __forceinline__ double unordered(u64 u) {
  const long long b = static_cast<long long>(u ^ 0x8000000000000000ull);
  return __longlong_as_double(b ^ (b >> 63 & 0x7fffffffffffffffll));
}

// The natural logarithm of a sum of two float32, to about 1e-8: x = 2^k m, 1/sqrt2 < m < sqrt2, and with
// s = (m - 1) / (m + 1) log m = 2 (s + s^3 / 3 + s^5 / 5 + ..), |s| < 0.172. s is two float32, the quotient and its
// remainder; the other terms are below 0.002 of it and one. (64-bit instructions are few on this chip.)
__device__ __forceinline__ double log_of(float2 x) {
  const int b = __float_as_int(x.x);
  const int k = (b - 0x3f3504f3) >> 23;  // the exponent that leaves m in (1/sqrt2, sqrt2)
  const float unit = __int_as_float((127 - k) << 23), hi = x.x * unit, lo = x.y * unit;
  const float num = hi - 1.f, den = hi + 1.f;  // num exact; den's rounding is carried along
  const float den_lo = (hi - (den - 1.f)) + lo;
  const float s = num / den, s_lo = (fmaf(-s, den, num) + lo - s * den_lo) / den;
  const float z = s * s;
  const float tail = s * z * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 11, 1.f / 9), 1.f / 7), 1.f / 5), 1.f / 3);
  // k ln 2 in two float32, the first with a product that is exact (the pair of Moshier's Cephes library)
  const float ln = k * 0.693359375f, ln_lo = fmaf(k, -2.12194440e-4f, 2.f * (s_lo + tail));
  return (double)ln + ((double)(2.f * s) + ln_lo);
}

constexpr int kSelectThreads = 256, kSelectWarps = kSelectThreads / 32;
constexpr int kList = kSelectThreads;  // parts and candidates that the bound may leave

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const BeamSelect p, int parts, const FastDiv by_parts,
                                                                const FastDiv by_K, const FastDiv by_V, const Part *part,
                                                                const u64 *keys) {
  __shared__ double logs[kMaxBeams];  // of each beam's sum of exp(x - top)
  __shared__ float tops[kMaxBeams];
  __shared__ float base[kMaxBeams];   // about score - log; NaN: its candidates have no value, infinity: it has ended, with a score
  __shared__ unsigned heads[kSelectThreads];
  __shared__ Candidate list[kList];
  __shared__ int passed[kList];
  __shared__ int passing, count;
  wait_for_stream();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float *scores = p.scores + b * p.W;
  const int lists = p.W * parts, all = lists * p.K;
  const u64 *mine = keys + (size_t)b * all;
  // Threads look at each list's first candidate, or at 2^deep of each: while no more than the threads are looked at, and
  // where all K may come from one beam of fewer than 2 K parts (18 x 16 rows of 43624, 32 best: this kernel 84 us without, 28).
  int deep = 0;
  while ((lists << (deep + 1) <= kSelectThreads || parts << deep < 2 * p.K) && 2 << deep <= p.K) ++deep;
  const int looks = lists << deep, mask = (1 << deep) - 1;
  auto key_of = [&](int i) { return mine[(i >> deep) * p.K + (i & mask)]; };
  const u64 first = tid < looks ? key_of(tid) : 0;  // (that of an ended beam is not used)
  auto look = [&](int i) { return i == tid ? first : key_of(i); };
#pragma unroll 1
  for (int w = warp; w < p.W; w += kSelectWarps) {
    const Part *s = part + (size_t)(b * p.W + w) * parts;
    const bool done = p.done && p.done[b * p.W + w];
    const float score = scores[w];
    float m = -INFINITY;
    float2 sum = make_float2(0.f, 0.f);
    bool bad = false;
#pragma unroll 1
    for (int i = lane; i < parts && !done; i += 32) {  // sums to their largest reference so far
      const Part a = s[i];
      bad |= a.bad != 0;
      if (!(a.sum.x > 0.f)) continue;
      const float top = fmaxf(m, a.ref);
      sum = add2(mul2(sum, expf(m - top)), mul2(a.sum, expf(a.ref - top)));
      m = top;
    }
    bad = __any_sync(~0u, bad);
    const float top = unordered(__reduce_max_sync(~0u, ordered(m)));
    if (m > -INFINITY) sum = mul2(sum, expf(m - top));
#pragma unroll 1
    for (int d = 16; d > 0; d /= 2) sum = add2(sum, make_float2(__shfl_xor_sync(~0u, sum.x, d), __shfl_xor_sync(~0u, sum.y, d)));
    if (lane == 0) {
      const bool value = !bad && sum.x > 0.f && isfinite(score);
      const double log = value ? log_of(sum) : 0;
      logs[w] = log;
      tops[w] = top;
      base[w] = done && isfinite(score) ? INFINITY : value ? score - static_cast<float>(log) : CUDART_NAN_F;
    }
  }
  if (tid == 0) passing = count = 0;
  __syncthreads();
  // Candidate at = j * K + r of beam w is the r-th of part j, with key k; an ended beam's first one is eos, its others and
  // those of a beam without values (an ended one without a score too) the first tokens, without a value. Inside a part they fall.
  auto rough = [&](int w, int at, u64 k) -> float {  // its score, to float32; NaN: none
    const float c = base[w];
    if (c == INFINITY) return at == 0 ? scores[w] : at < p.K && at < p.V ? -INFINITY : CUDART_NAN_F;
    if (isnan(c)) return at < p.K && at < p.V ? -INFINITY : CUDART_NAN_F;
    return k ? c + (unordered(static_cast<unsigned>(k >> 32)) - tops[w]) : CUDART_NAN_F;
  };
  auto candidate = [&](int w, int at, u64 k) -> Candidate {
    const u64 none = ordered(-(double)INFINITY);
    const unsigned first = static_cast<unsigned>(w * p.V);
    if (base[w] == INFINITY && at == 0) return {ordered((double)scores[w]), ~(first + p.eos)};
    if (base[w] == INFINITY) return {none, ~(first + at - (at <= p.eos))};
    if (isnan(base[w])) return {none, ~(first + at)};
    // The log last: what is in front of it is exact, so that equal candidates of beams with the same sum stay equal.
    // (And not x - (top + log): a top near the type's limits would swallow the log.)
    const double x = ((double)scores[w] + ((double)unordered(static_cast<unsigned>(k >> 32)) - tops[w])) - logs[w];
    return {ordered(x), ~(first + ~static_cast<unsigned>(k))};
  };
  // As in a part: the K-th largest of the threads' bounds what can be among the K best, and so does that of a warp's. For few
  // the best of the warps' is near enough (1 x 4: 9.5 us, with all threads' 10.2); for many it leaves most candidates (2 x 16
  // rows of 27787, 32 of each: 65 us, with all threads' 27). All in float32, with what that may be off taken from the bound.
  float head = -INFINITY;
  bool any = false;
#pragma unroll 1
  for (int i = tid; i < looks; i += kSelectThreads) {
    unsigned w, j;
    by_parts.split(i >> deep, w, j);
    const float c = rough(w, j * p.K + (i & mask), look(i));
    if (!isnan(c)) head = fmaxf(head, c), any = true;
  }
  unsigned order = sorted(any ? ordered(head) : 0u, lane);
  heads[tid] = order;
  __syncthreads();
  unsigned bound = 0;
  if (p.K <= 8) {
#pragma unroll
    for (int i = 0; i < kSelectWarps; ++i) bound = max(bound, heads[i * 32 + p.K - 1]);
  } else {  // the 32 best of two warps, until one has those of all
#pragma unroll 1
    for (int half = kSelectWarps / 2; half > 0; half /= 2) {
      if (warp < half) heads[tid] = order = merged(order, heads[tid + half * 32], lane);
      __syncthreads();
    }
    bound = heads[p.K - 1];
  }
  float low = bound ? unordered(bound) : -INFINITY, size = 0.f;
  if (lane < p.W && isfinite(base[lane])) size = fabsf(base[lane]) + fabsf(static_cast<float>(logs[lane]));
  size = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(size)));
  // 2^-24 each of the log, of base, of x - top (|base| + |low| at most) and of their sum, for the bound and for what it is held
  // against: below 2^-22 (|low| + |base| + log). (base alone is not enough: it is small where a score is near the log.)
  low -= 1e-6f * (fabsf(low) + size);
  // the parts whose first candidate passes, then their candidates that pass
#pragma unroll 1
  for (int i = tid; i < looks; i += kSelectThreads) {
    unsigned w, j;
    by_parts.split(i >> deep, w, j);
    if (i & mask || !(rough(w, j * p.K, look(i)) >= low)) continue;
    const int n = atomicAdd(&passing, 1);
    if (n < kList) passed[n] = i >> deep;
  }
  __syncthreads();
  const bool few = passing <= kList;
#pragma unroll 1
  for (int i = tid; i < passing * p.K && few; i += kSelectThreads) {
    unsigned n, r, w, j;
    by_K.split(i, n, r);
    by_parts.split(passed[n], w, j);
    const u64 k = mine[passed[n] * p.K + r];
    if (!(rough(w, j * p.K + r, k) >= low)) continue;
    const int c = atomicAdd(&count, 1);
    if (c < kList) list[c] = candidate(w, j * p.K + r, k);
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
  if (few && n <= kList) {  // a candidate's rank: how many are above it, counted by eight threads
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kSelectThreads / 8) {
      const int i = min(i0 + tid / 8, n - 1);
      const Candidate k = list[i];
      int r = 0;
      for (int o = tid % 8; o < n; o += 8) r += list[o] > k;
#pragma unroll
      for (int d = 4; d > 0; d /= 2) r += __shfl_xor_sync(~0u, r, d);
      if (tid % 8 == 0 && i0 + tid / 8 < n && r < p.K) put(r, k);
    }
    return;
  }
  // Too many that are equal, or fewer than K with a value among those looked at: warps keep the best 32 that they meet, in
  // order, and are joined two by two. (2 x 16 bfloat16 rows of 50257 zeros, 32 best: 48 us for both
  // kernels; one more candidate of the falling lists at a time 82.)
  Candidate best = {0, 0};
  u64 next = tid < all ? mine[tid] : 0;
#pragma unroll 1
  for (int i = tid; i - lane < all; i += kSelectThreads) {
    Candidate o = {0, 0};
    const u64 k = next;
    if (i + kSelectThreads < all) next = mine[i + kSelectThreads];
    if (i < all) {
      unsigned l, r, w, j;
      by_K.split(i, l, r);
      by_parts.split(l, w, j);
      if (rough(w, j * p.K + r, k) >= low) o = candidate(w, j * p.K + r, k);
    }
    const Candidate last = {__shfl_sync(~0u, best.score, p.K - 1), __shfl_sync(~0u, best.rank, p.K - 1)};
    if (__any_sync(~0u, o > last)) best = merged(best, sorted(o, lane), lane);
  }
#pragma unroll 1
  for (int half = kSelectWarps / 2; half > 0; half /= 2) {
    __syncthreads();
    if (warp >= half) list[tid] = best;
    __syncthreads();
    if (warp < half) best = merged(best, list[tid + half * 32], lane);
  }
  if (tid < p.K) put(tid, best);
}

// Granules of a lane: few for short rows, so that all SMs have some, but not so few that the second kernel has more than
// some hundred parts to look through (4 beams of 32000, both kernels: 500 parts 14.4 us, 125 parts 9.1). No more than 8:
// with 16 the SMs hold fewer warps (32 x 8 rows of 50257: 22.5 us, with 8 20.1).
int granules(const BeamSelect &p) {
  const long long rows = (long long)p.B * p.W, e = p.f32 ? 4 : 8;
  int g = 8;
  while (g > 2 && rows * (p.V / (32 * g * e)) < 8ll * std::max(sm_count(), 1) && p.W * (p.V / (16 * g * e)) <= 160) g /= 2;
  return g;
}

template <typename T, int G>
cudaError_t launch_g(const BeamSelect &p, int parts, Part *part, u64 *keys, cudaStream_t stream) {
  const int total = p.B * p.W * parts;
  return launch_early(part_kernel<T, G>, dim3((total - 1) / kWarps + 1), kThreads, kWarps * sizeof(Work<G>), stream, p, total,
                      parts, part, keys);
}

template <typename T>
cudaError_t launch(const BeamSelect &p, int g, int parts, Part *part, u64 *keys, cudaStream_t stream) {
  return g == 2   ? launch_g<T, 2>(p, parts, part, keys, stream)
         : g == 4 ? launch_g<T, 4>(p, parts, part, keys, stream)
                  : launch_g<T, 8>(p, parts, part, keys, stream);
}

int fail(const char *what, cudaError_t e) {
  set_error("la_beam_select: %s: %s", what, cudaGetErrorString(e));
  return LA_ERR_CUDA;
}

}  // namespace

int launch_beam_select(const BeamSelect &p, cudaStream_t stream) {
  const int g = granules(p), parts = (p.V - 1) / (32 * g * (p.f32 ? 4 : 8)) + 1;
  const size_t total = (size_t)p.B * p.W * parts;
  uint8_t *ws = nullptr;
  cudaMemPool_t pool = library_pool();
  if (!pool) return fail("could not create the workspace pool", cudaGetLastError());
  cudaError_t e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), total * (sizeof(Part) + sizeof(u64) * p.K), pool,
                                          stream);
  if (e != cudaSuccess) return fail("workspace allocation failed", e);
  Part *part = reinterpret_cast<Part *>(ws);
  u64 *keys = reinterpret_cast<u64 *>(part + total);
  e = p.f32 ? launch<float>(p, g, parts, part, keys, stream) : launch<__nv_bfloat16>(p, g, parts, part, keys, stream);
  if (e == cudaSuccess)
    e = launch_early(select_kernel, dim3(p.B), kSelectThreads, 0, stream, p, parts, FastDiv(parts), FastDiv(p.K), FastDiv(p.V),
                     part, keys);
  const cudaError_t f = cudaFreeAsync(ws, stream);
  if (e == cudaSuccess) e = f;
  return e == cudaSuccess ? LA_OK : fail("launch failed", e);
}

}  // namespace la
