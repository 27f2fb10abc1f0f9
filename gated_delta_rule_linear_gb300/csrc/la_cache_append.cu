// New tokens into a paged key-value cache, keys and queries turned by their
// positions on the way: K[place] = R(pos) k, V[place] = v, q_out = R(pos) q.
//
// Bound by memory traffic: q, k and v once in, q_out and the cache's rows once
// out; with few tokens by the chain lens -> table -> row. As in la_rotary.cu a
// CTA takes a few tokens: it looks up where each of them goes and forms the
// cosines and sines once, under which the rows are on their way into L2.
#include "la_rotary.cuh"
#include "la_serve_internal.h"
#include "la_sm100.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 8;  // most tokens of a CTA

struct AppendDiv {
  FastDiv items, heads, P, values, page;
};

// V elements at a time (16 bytes), or 1 where sizes or addresses do not allow
// it. Work items of a row as in rotary_kernel: interleaved, vectors of V/2 pairs
// (V = 1: one pair); halves, V channels with their V partners; the channels
// behind the pairs are copied.
template <typename T, int V, bool IL>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p, const AppendDiv by, int tokens) {
  extern __shared__ float2 turn[];  // [tokens][P] cos, sin
  __shared__ int seq[kTokens], place[kTokens];
  __shared__ long long row[kTokens];  // element of the token's row in the caches, -1: it has none
  const int P = p.s0 + p.s1 + p.s2, n0 = blockIdx.x * tokens, m = min(tokens, p.total - n0), tid = threadIdx.x;
  const int hd = p.Hk * p.d;
  if (V > 1 && tid < 3 * m) {  // a token's heads are one run of bytes
    const int n = n0 + tid / 3, which = tid % 3;
    if (which || p.H)
      sm100::bulk_prefetch_l2(static_cast<const T *>(which == 0 ? p.q : which == 1 ? p.k : p.v) +
                                  n * (which == 0 ? p.ldq : which == 1 ? p.ldk : p.ldv),
                              (which == 0 ? p.H * p.d : hd) * static_cast<int>(sizeof(T)));
  }
  if (tid < kTokens) seq[tid] = p.cu ? INT_MAX : n0 + tid;
  if (p.cu) {  // the sequences of these tokens: all are looked at, the unused end of cu_seqlens may hold anything
    __syncthreads();
    for (int s = tid; s < p.n_seq; s += kThreads) {
      int a, b;
      packed_range(p.cu, s, p.total, &a, &b);
      for (int i = max(a - n0, 0); i < min(b - n0, m); ++i) atomicMin(&seq[i], s);
    }
    __syncthreads();
  }
  if (tid < m) {
    const int s = seq[tid];
    long long at = -1;
    int where = 0;
    if (s != INT_MAX) {
      int a = n0 + tid, b = a + 1;
      if (p.cu) packed_range(p.cu, s, p.total, &a, &b);
      const long long pl = (long long)__ldg(p.at.lens + s) - (b - n0 - tid);
      where = static_cast<int>(pl);
      if (pl >= 0) {
        uint32_t page, r;
        by.page.split(where, page, r);
        if ((int)page < p.at.max_pages) {
          const int g = __ldg(p.at.table + s * p.at.ld_table + page);
          if (g >= 0 && g < p.at.n_pages) at = g * p.at.ld_page + (long long)r * hd;
        }
      }
    }
    place[tid] = where;
    row[tid] = at;
  }
  __syncthreads();
  for (int i = tid; i < m * P; i += kThreads) {
    uint32_t n, c;
    by.P.split(i, n, c);
    const int axis = (int)c < p.s0 ? 0 : (int)c < p.s0 + p.s1 ? 1 : 2;
    turn[i] = rotary_turn(__ldg(p.freq + c), p.pos ? __ldg(p.pos + (size_t)(n0 + n) * p.n_axes + axis) : place[n], false);
  }
  // values meanwhile
  const int vitems = hd / V;
#pragma unroll 2
  for (int i = tid; i < m * vitems; i += kThreads) {
    uint32_t n, c;
    by.values.split(i, n, c);
    if (row[n] < 0) continue;
    const T *src = static_cast<const T *>(p.v) + (n0 + n) * p.ldv + c * V;
    T *dst = static_cast<T *>(p.v_cache) + row[n] + c * V;
    if constexpr (V == 1) *dst = *src;
    else *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(src);
  }
  __syncthreads();
  constexpr int W = V == 1 && IL ? 2 : V;    // channels of one load
  const int pairs = IL ? 2 * P / W : P / W;  // rotating items of a row
  const int rest = (p.d - 2 * P) / V, items = pairs + rest, heads = p.H + p.Hk;
#pragma unroll 4
  for (int i = tid; i < m * heads * items; i += kThreads) {
    uint32_t q, n, head, item;
    by.items.split(i, q, item);
    by.heads.split(q, n, head);
    const int it = item;
    const bool is_k = (int)head >= p.H;
    if (is_k ? row[n] < 0 : seq[n] == INT_MAX) continue;
    const T *src;
    T *dst;
    if (is_k) {
      const int c = (head - p.H) * p.d;
      src = static_cast<const T *>(p.k) + (n0 + n) * p.ldk + c;
      dst = static_cast<T *>(p.k_cache) + row[n] + c;
    } else {
      src = static_cast<const T *>(p.q) + (n0 + n) * p.ldq + head * p.d;
      dst = static_cast<T *>(p.q_out) + ((long long)(n0 + n) * p.H + head) * p.d;
    }
    const float2 *cs = turn + n * P;
    float a[W], b[W];
    if (it >= pairs) {
      const int c = 2 * P + (it - pairs) * V;
      Vec<T, V>::load(src + c, a);
      Vec<T, V>::store(dst + c, a);
    } else if (IL) {
      const int c = it * W;
      if (V == 1) {
        Vec<T, 1>::load(src + c, a);
        Vec<T, 1>::load(src + c + 1, a + (W > 1 ? 1 : 0));
      } else {
        Vec<T, V>::load(src + c, a);
      }
#pragma unroll
      for (int j = 0; j < W / 2; ++j) {
        const float2 t = cs[c / 2 + j];
        const float u = a[2 * j], w = a[2 * j + 1];
        a[2 * j] = u * t.x - w * t.y;
        a[2 * j + 1] = w * t.x + u * t.y;
      }
      if (V == 1) {
        Vec<T, 1>::store(dst + c, a);
        Vec<T, 1>::store(dst + c + 1, a + (W > 1 ? 1 : 0));
      } else {
        Vec<T, V>::store(dst + c, a);
      }
    } else {
      const int c = it * V;
      Vec<T, V>::load(src + c, a);
      Vec<T, V>::load(src + c + P, b);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float2 t = cs[c + j];
        const float u = a[j], w = b[j];
        a[j] = u * t.x - w * t.y;
        b[j] = w * t.x + u * t.y;
      }
      Vec<T, V>::store(dst + c, a);
      Vec<T, V>::store(dst + c + P, b);
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
  // tokens of a CTA: enough rows that its loads overlap, not so many that the grid leaves SMs idle
  const int W = wide ? V : p.interleaved ? 2 : 1;
  const int items = (p.interleaved ? 2 * P / W : P / W) + (p.d - 2 * P) / (wide ? V : 1), heads = p.H + p.Hk;
  const long long sms = sm_count() > 0 ? sm_count() : 1;
  int tokens = 1;
  while (tokens < kTokens && (long long)tokens * items * heads < 8 * kThreads && p.total / (2 * tokens) >= 8 * sms)
    tokens *= 2;
  const AppendDiv by = {FastDiv(items), FastDiv(heads), FastDiv(P > 0 ? P : 1), FastDiv(p.Hk * p.d / (wide ? V : 1)),
                        FastDiv(p.at.page_size)};
  const int grid = (p.total - 1) / tokens + 1;
  const size_t smem = (size_t)tokens * P * sizeof(float2);
  if (wide && p.interleaved) append_kernel<T, V, true><<<grid, kThreads, smem, stream>>>(p, by, tokens);
  else if (wide) append_kernel<T, V, false><<<grid, kThreads, smem, stream>>>(p, by, tokens);
  else if (p.interleaved) append_kernel<T, 1, true><<<grid, kThreads, smem, stream>>>(p, by, tokens);
  else append_kernel<T, 1, false><<<grid, kThreads, smem, stream>>>(p, by, tokens);
  return cudaGetLastError();
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
