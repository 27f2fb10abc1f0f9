// New tokens into a paged key-value cache, keys and queries turned by their
// positions on the way: K[place] = R(pos) k, V[place] = v, q_out = R(pos) q.
//
// Bound by memory traffic: q, k and v once in, q_out and the cache's rows once
// out; with few tokens by the chain of loads cu_seqlens and lens -> table -> row.
// A CTA takes up to 8 tokens. Its threads look through the sequences for them
// once; from there on a token has warps of its own, which form its cosines and
// sines while the table entry and the rows (asked into L2 first) are on their way.
//
// 32768 tokens of 16 + 4 + 4 heads of 128, bfloat16: 68 us, 5.9 TB/s (a CTA's
// tokens together, with cosines read across banks: 75.7 us); 128 single tokens:
// 5 us, a chain of four loads from memory and the launch.
#include <climits>
#include <type_traits>

#include "la_rotary.cuh"
#include "la_serve_internal.h"
#include "la_sm100.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;  // and most tokens of a CTA

constexpr int kBatch = 2;              // items of a lane whose loads are in flight together

// W elements as they are loaded: 16 bytes, or W = 1, 2 one by one.
template <typename T, int W> struct Row {
  static constexpr bool kWide = W * sizeof(T) == 16;
  std::conditional_t<kWide, uint4, T> u[kWide ? 1 : W];
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (kWide) {
      u[0] = *reinterpret_cast<const uint4 *>(p);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) u[i] = p[i];
    }
  }
  __device__ __forceinline__ void store(T *p) const {
    if constexpr (kWide) {
      *reinterpret_cast<uint4 *>(p) = u[0];
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) p[i] = u[i];
    }
  }
  __device__ __forceinline__ void load_one(const T *p) {
    if constexpr (!kWide) u[0] = *p;
  }
  __device__ __forceinline__ void store_one(T *p) const {
    if constexpr (!kWide) *p = u[0];
  }
  __device__ __forceinline__ void get(float *f) const {
    if constexpr (kWide) {
      Vec<T, W>::load(reinterpret_cast<const T *>(u), f);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) f[i] = static_cast<float>(u[i]);
    }
  }
  __device__ __forceinline__ void set(const float *f) {
    if constexpr (kWide) {
      Vec<T, W>::store(reinterpret_cast<T *>(u), f);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) u[i] = T(f[i]);
    }
  }
};

struct AppendDiv {
  FastDiv items, page;
};

// packed_range without its read-only loads: this kernel is in flight before what writes cu_seqlens may be done.
__device__ __forceinline__ void range_of(const AppendParams &p, int s, int *a, int *b) {
  const int lo = min(max(p.cu[s], 0), p.total);
  *a = lo;
  *b = min(max(p.cu[s + 1], lo), p.total);
}
// The place of a token with `behind` - 1 ones behind it.
__device__ __forceinline__ int place_of(int len, int behind) {
  return static_cast<int>(max((long long)len - behind, (long long)INT_MIN));
}

// V elements at a time (16 bytes), or 1 where sizes or addresses do not allow
// it. Work items of a row as in rotary_kernel: interleaved, vectors of V/2 pairs
// (V = 1: one pair); halves, V channels with their V partners; the channels
// behind the pairs are copied.
template <typename T, int V, bool IL>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p, const AppendDiv by, int tokens) {
  extern __shared__ float2 turns[];  // [warps][P] cos, sin
  __shared__ unsigned long long found[kWarps];  // sequence and place of a token
  const int P = p.s0 + p.s1 + p.s2, n0 = blockIdx.x * tokens, m = min(tokens, p.total - n0);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hd = p.Hk * p.d;
  wait_for_stream();
  if (V > 1 && tid < 3 * m) {  // a token's heads are one run of bytes
    const int n = n0 + tid / 3, which = tid % 3;
    if (which || p.H)
      sm100::bulk_prefetch_l2(static_cast<const T *>(which == 0 ? p.q : which == 1 ? p.k : p.v) +
                                  n * (which == 0 ? p.ldq : which == 1 ? p.ldk : p.ldv),
                              (which == 0 ? p.H * p.d : hd) * static_cast<int>(sizeof(T)));
  }
  const int each = kWarps / tokens, i = warp / each, sub = warp % each;  // (tokens is a power of two)
  const int n = n0 + i;
  int s, place;
  if (p.cu) {  // all sequences are looked at: the unused end of cu_seqlens may hold anything
    if (tid < kWarps) found[tid] = ~0ull;
    __syncthreads();
    for (int q = tid; q < p.n_seq; q += kThreads) {
      const int len = p.at.lens[q];
      int a, b;
      range_of(p, q, &a, &b);
      for (int t = max(a - n0, 0); t < min(b - n0, m); ++t)  // the first sequence that has it
        atomicMin(&found[t], (unsigned long long)q << 32 | static_cast<unsigned>(place_of(len, b - n0 - t)));
    }
    __syncthreads();
    if (i >= m || found[i] == ~0ull) return;
    s = static_cast<int>(found[i] >> 32);
    place = static_cast<int>(found[i]);
  } else {
    if (i >= m) return;
    s = n;
    place = place_of(p.at.lens[s], 1);
  }
  long long row = -1;  // element of the token's row in the caches, -1: it has none
  if (place >= 0) {
    uint32_t page, r;
    by.page.split(place, page, r);
    if ((int)page < p.at.max_pages) {
      const int g = p.at.table[s * p.at.ld_table + page];
      if (g >= 0 && g < p.at.n_pages) row = g * p.at.ld_page + (long long)r * hd;
    }
  }
  constexpr int W = V == 1 && IL ? 2 : V;    // channels of one load
  constexpr int R = IL ? W / 2 : V;          // pairs of an item
  const int pairs = IL ? 2 * P / W : P / W;  // rotating items of a row
  float2 *turn = turns + warp * P;           // pair e of item i at e * pairs + i: lanes are neighbouring items
  for (int c = lane; c < P; c += 32) {
    const int axis = c < p.s0 ? 0 : c < p.s0 + p.s1 ? 1 : 2;
    turn[c % R * pairs + c / R] = rotary_turn(p.freq[c], p.pos ? p.pos[(size_t)n * p.n_axes + axis] : place, false);
  }
  __syncwarp();
  // rows, kBatch loads of a lane in front of their stores
  const int lanes = each * 32, at = sub * 32 + lane;
  if (row >= 0) {
    const T *src = static_cast<const T *>(p.v) + n * p.ldv;
    T *dst = static_cast<T *>(p.v_cache) + row;
    for (int c0 = at; c0 < hd / V; c0 += kBatch * lanes) {
      using Unit = std::conditional_t<V == 1, T, uint4>;
      Unit u[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int c = c0 + k * lanes;
        if (c < hd / V) u[k] = reinterpret_cast<const Unit *>(src)[c];
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int c = c0 + k * lanes;
        if (c < hd / V) reinterpret_cast<Unit *>(dst)[c] = u[k];
      }
    }
  }
  const int rest = (p.d - 2 * P) / V, items = pairs + rest;
  const int first = row < 0 ? p.Hk * items : 0, all = (p.Hk + p.H) * items;  // keys, then queries
  for (int j0 = first + at; j0 < all; j0 += kBatch * lanes) {
    Row<T, W> a[kBatch], b[kBatch];
    T *dst[kBatch];
    int which[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int j = j0 + k * lanes;
      if (j >= all) continue;
      uint32_t head, item;
      by.items.split(j, head, item);
      const int it = item;
      const bool turns = it < pairs;
      const int c = turns ? it * W : 2 * P + (it - pairs) * V;
      which[k] = it;
      const T *src;
      if ((int)head < p.Hk) {
        src = static_cast<const T *>(p.k) + n * p.ldk + head * p.d + c;
        dst[k] = static_cast<T *>(p.k_cache) + row + head * p.d + c;
      } else {
        src = static_cast<const T *>(p.q) + n * p.ldq + (head - p.Hk) * p.d + c;
        dst[k] = static_cast<T *>(p.q_out) + ((long long)n * p.H + head - p.Hk) * p.d + c;
      }
      if (W > V && !turns) a[k].load_one(src);
      else a[k].load(src);
      if (!IL && turns) b[k].load(src + P);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int j = j0 + k * lanes;
      if (j >= all) continue;
      const int it = which[k];
      if (it >= pairs) {
        if (W > V) a[k].store_one(dst[k]);
        else a[k].store(dst[k]);
        continue;
      }
      float x[W], y[W];
      a[k].get(x);
      if constexpr (IL) {
#pragma unroll
        for (int e = 0; e < W / 2; ++e) {
          const float2 t = turn[e * pairs + it];
          const float u = x[2 * e], w = x[2 * e + 1];
          x[2 * e] = u * t.x - w * t.y;
          x[2 * e + 1] = w * t.x + u * t.y;
        }
        a[k].set(x);
        a[k].store(dst[k]);
      } else {
        b[k].get(y);
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const float2 t = turn[e * pairs + it];
          const float u = x[e], w = y[e];
          x[e] = u * t.x - w * t.y;
          y[e] = w * t.x + u * t.y;
        }
        a[k].set(x);
        a[k].store(dst[k]);
        b[k].set(y);
        b[k].store(dst[k] + P);
      }
    }
  }
}

template <typename T>
cudaError_t launch(const AppendParams &p, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  const int P = p.s0 + p.s1 + p.s2;
  const void *all[] = {p.q, p.q_out, p.k, p.v, p.k_cache, p.v_cache};
  bool wide = p.d % V == 0 && (p.interleaved ? 2 * P : P) % V == 0 && (!p.H || p.ldq % V == 0) && p.ldk % V == 0 &&
              p.ldv % V == 0 && p.at.ld_page % V == 0;
  for (const void *t : all) wide = wide && (reinterpret_cast<uintptr_t>(t) & 15) == 0;
  // tokens of a CTA: few enough warps for each that a lane has some items, but all SMs busy
  const int W = wide ? V : p.interleaved ? 2 : 1;
  const int items = (p.interleaved ? 2 * P / W : P / W) + (p.d - 2 * P) / (wide ? V : 1);
  const long long sms = sm_count() > 0 ? sm_count() : 1;
  const long long work = (long long)(p.H + p.Hk) * items + p.Hk * p.d / (wide ? V : 1);
  int tokens = kWarps;
  while (tokens > 1 && (work * tokens > 8 * kThreads || p.total / tokens < 2 * sms)) tokens /= 2;
  const AppendDiv by = {FastDiv(items), FastDiv(p.at.page_size)};
  const int grid = (p.total - 1) / tokens + 1;
  return launch_early(wide ? (p.interleaved ? append_kernel<T, V, true> : append_kernel<T, V, false>)
                           : (p.interleaved ? append_kernel<T, 1, true> : append_kernel<T, 1, false>),
                      dim3(grid), kThreads, (size_t)kWarps * P * sizeof(float2), stream, p, by, tokens);
}

}  // namespace

int launch_cache_append(const AppendParams &p, cudaStream_t stream) {
  const cudaError_t e = p.f32 ? launch<float>(p, stream) : launch<__nv_bfloat16>(p, stream);
  if (e != cudaSuccess) {
    set_error("la_cache_append: launch failed: %s", cudaGetErrorString(e));
    return LA_ERR_CUDA;
  }
  return LA_OK;
}

}  // namespace la
