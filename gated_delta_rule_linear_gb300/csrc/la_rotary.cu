// Rotary positions with one to three axes on queries and keys.
//
// Bound by HBM traffic: every row once in and once out. A CTA takes a few
// tokens, forms their cosines and sines once in shared memory and turns all
// query and key heads with them; the rows are asked into L2 first, so that
// their way from HBM passes under the sines (0.219 -> 0.189 ms, 5.7 TB/s, on
// 65536 tokens of 16 + 16 heads of 128, bf16).
//
// Angles: see rotary_turn.
#include "la_layer_internal.h"
#include "la_rotary.cuh"
#include "la_sm100.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;

// Offset of row (n, h) of a tensor with `heads` heads: token-major (T = 0) or head-major.
__device__ __forceinline__ size_t row_at(int n, int h, int heads, int d, int T, const FastDiv &by_T, long long ld) {
  if (T == 0) return (size_t)n * ld + (size_t)h * d;
  uint32_t b, t;
  by_T.split(n, b, t);
  return (((size_t)b * heads + h) * T + t) * d;
}

struct RotaryDiv {
  FastDiv items, heads, T_in, T_out, P;
};

// V channels at a time (16 bytes), or 1 where sizes or addresses do not allow it.
// Work items of a row: interleaved, V = vector of V/2 pairs (V = 1: one pair);
// halves, V channels of the first half with their V partners. Channels behind
// the pairs are copied, V at a time.
template <typename T, int V, bool IL>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p, const RotaryDiv by, int tokens) {
  extern __shared__ float2 turn[];  // [tokens][P] cos, sin
  const int P = p.s0 + p.s1 + p.s2, n0 = blockIdx.x * tokens, m = min(tokens, p.N - n0);
  // the rows into L2 under the sines; a token's heads are one run of bytes
  if (V > 1 && p.T_in == 0 && (int)threadIdx.x < 2 * m) {
    const bool is_k = threadIdx.x & 1;
    if (!is_k || p.k)
      sm100::bulk_prefetch_l2(static_cast<const T *>(is_k ? p.k : p.q) +
                                  (size_t)(n0 + (threadIdx.x >> 1)) * (is_k ? p.ldk : p.ldq),
                              (is_k ? p.Hk : p.H) * p.d * static_cast<int>(sizeof(T)));
  }
  for (int i = threadIdx.x; i < m * P; i += kThreads) {
    uint32_t n, c;
    by.P.split(i, n, c);
    const int axis = (int)c < p.s0 ? 0 : (int)c < p.s0 + p.s1 ? 1 : 2;
    turn[i] = rotary_turn(__ldg(p.freq + c), __ldg(p.pos + (size_t)(n0 + n) * p.n_axes + axis), p.inverse);
  }
  __syncthreads();
  constexpr int W = V == 1 && IL ? 2 : V;             // channels of one load
  const int pairs = IL ? 2 * P / W : P / W;           // rotating items of a row
  const int rest = (p.d - 2 * P) / V, items = pairs + rest;
  const int heads = p.H + (p.k ? p.Hk : 0);
#pragma unroll 4
  for (int i = threadIdx.x; i < m * heads * items; i += kThreads) {
    uint32_t q, n, head, item;
    by.items.split(i, q, item);
    by.heads.split(q, n, head);
    const int hh = head, it = item;
    const bool is_k = hh >= p.H;
    const int h = is_k ? hh - p.H : hh, nh = is_k ? p.Hk : p.H;
    const T *src = static_cast<const T *>(is_k ? p.k : p.q) +
                   row_at(n0 + n, h, nh, p.d, p.T_in, by.T_in, is_k ? p.ldk : p.ldq);
    T *dst = static_cast<T *>(is_k ? p.k_out : p.q_out) + row_at(n0 + n, h, nh, p.d, p.T_out, by.T_out, (long long)nh * p.d);
    const float scale = is_k ? p.scale_k : p.scale_q;
    const float2 *cs = turn + n * P;
    float a[W], b[W];
    if (it >= pairs) {
      const int c = 2 * P + (it - pairs) * V;
      Vec<T, V>::load(src + c, a);
#pragma unroll
      for (int j = 0; j < V; ++j) a[j] *= scale;
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
        a[2 * j] = (u * t.x - w * t.y) * scale;
        a[2 * j + 1] = (w * t.x + u * t.y) * scale;
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
        a[j] = (u * t.x - w * t.y) * scale;
        b[j] = (w * t.x + u * t.y) * scale;
      }
      Vec<T, V>::store(dst + c, a);
      Vec<T, V>::store(dst + c + P, b);
    }
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T>
cudaError_t launch(const RotaryParams &p, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  const int P = p.s0 + p.s1 + p.s2;
  const bool wide = p.d % V == 0 && (p.interleaved ? 2 * P : P) % V == 0 && aligned16(p.q) && aligned16(p.q_out) &&
                    aligned16(p.k) && aligned16(p.k_out) && (p.T_in > 0 || (p.ldq % V == 0 && p.ldk % V == 0));
  // tokens of a CTA: enough rows that its loads overlap, not so many that the grid leaves SMs idle
  const int W = wide ? V : p.interleaved ? 2 : 1;
  const int items = (p.interleaved ? 2 * P / W : P / W) + (p.d - 2 * P) / (wide ? V : 1), heads = p.H + (p.k ? p.Hk : 0);
  const long long sms = sm_count() > 0 ? sm_count() : 1;
  int tokens = 1;
  while (tokens < 8 && (long long)tokens * items * heads < 8 * kThreads && p.N / (2 * tokens) >= 8 * sms) tokens *= 2;
  const RotaryDiv by = {FastDiv(items), FastDiv(heads), FastDiv(p.T_in > 0 ? p.T_in : 1),
                        FastDiv(p.T_out > 0 ? p.T_out : 1), FastDiv(P)};
  const int grid = (p.N - 1) / tokens + 1;  // N >= 1, up to INT_MAX
  const size_t smem = (size_t)tokens * P * sizeof(float2);
  if (wide && p.interleaved) rotary_kernel<T, V, true><<<grid, kThreads, smem, stream>>>(p, by, tokens);
  else if (wide) rotary_kernel<T, V, false><<<grid, kThreads, smem, stream>>>(p, by, tokens);
  else if (p.interleaved) rotary_kernel<T, 1, true><<<grid, kThreads, smem, stream>>>(p, by, tokens);
  else rotary_kernel<T, 1, false><<<grid, kThreads, smem, stream>>>(p, by, tokens);
  return cudaGetLastError();
}

}  // namespace

int launch_rotary(const RotaryParams &p, cudaStream_t stream) {
  const cudaError_t e = p.f32 ? launch<float>(p, stream) : launch<__nv_bfloat16>(p, stream);
  if (e != cudaSuccess) {
    set_error("la_rotary: launch failed: %s", cudaGetErrorString(e));
    return LA_ERR_CUDA;
  }
  return LA_OK;
}

}  // namespace la
