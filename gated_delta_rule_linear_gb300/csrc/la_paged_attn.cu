// Attention of one new token of each sequence over a paged cache:
// o_h = sum_p softmax_p(scale q_h . k_p) v_p.
//
// One CTA takes a (sequence, query head); each warp walks every fourth place
// with a running maximum and sum, a lane holding d / 32 channels.
#include <cuda_bf16.h>

#include "la_serve_internal.h"

namespace la {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attn_kernel(const PagedAttn p, const FastDiv by_page) {
  constexpr int C = D / 32;
  __shared__ float so[kWarps][D], sm[kWarps], sl[kWarps];
  const int s = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / (p.H / p.Hk);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int len = min((long long)max(__ldg(p.at.lens + s), 0), (long long)p.at.max_pages * p.at.page_size);
  const int first = p.window > 0 ? max(len - p.window, 0) : 0;
  const T *q = static_cast<const T *>(p.q) + s * p.ldq + h * D;
  float qf[C], o[C], m = -INFINITY, l = 0.f;
  for (int c = 0; c < C; ++c) {
    qf[c] = static_cast<float>(q[lane + 32 * c]);
    o[c] = 0.f;
  }
  for (int i = first + warp; i < len; i += kWarps) {
    uint32_t pg, r;
    by_page.split(i, pg, r);
    const int g = __ldg(p.at.table + s * p.at.ld_table + pg);
    if (g < 0 || g >= p.at.n_pages) continue;
    const long long at = g * p.at.ld_page + ((long long)r * p.Hk + hk) * D + lane;
    const T *k = static_cast<const T *>(p.k_cache) + at, *v = static_cast<const T *>(p.v_cache) + at;
    float x = 0.f;
    for (int c = 0; c < C; ++c) x = fmaf(qf[c], static_cast<float>(k[32 * c]), x);
    for (int d = 16; d > 0; d /= 2) x += __shfl_xor_sync(~0u, x, d);
    x *= p.scale;
    const float next = fmaxf(m, x), keep = expf(m - next), e = expf(x - next);
    l = l * keep + e;
    for (int c = 0; c < C; ++c) o[c] = o[c] * keep + e * static_cast<float>(v[32 * c]);
    m = next;
  }
  for (int c = 0; c < C; ++c) so[warp][lane + 32 * c] = o[c];
  if (lane == 0) { sm[warp] = m; sl[warp] = l; }
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  if (top == -INFINITY) top = 0.f;
  for (int w = 0; w < kWarps; ++w) sum += sl[w] * expf(sm[w] - top);
  for (int c = threadIdx.x; c < D; c += kThreads) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += so[w][c] * expf(sm[w] - top);
    static_cast<T *>(p.o)[((size_t)s * p.H + h) * D + c] = T(sum > 0.f ? x / sum : 0.f);
  }
  if (p.lse && threadIdx.x == 0) p.lse[(size_t)s * p.H + h] = sum > 0.f ? top + logf(sum) : -INFINITY;
}

template <typename T>
void launch(const PagedAttn &p, cudaStream_t stream) {
  const FastDiv by(p.at.page_size);
  const unsigned grid = static_cast<unsigned>(p.n) * p.H;
  if (p.d == 64) attn_kernel<T, 64><<<grid, kThreads, 0, stream>>>(p, by);
  else if (p.d == 128) attn_kernel<T, 128><<<grid, kThreads, 0, stream>>>(p, by);
  else attn_kernel<T, 256><<<grid, kThreads, 0, stream>>>(p, by);
}

}  // namespace

int launch_paged_attn(const PagedAttn &p, cudaStream_t stream) {
  if (p.f32) launch<float>(p, stream);
  else launch<__nv_bfloat16>(p, stream);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("la_paged_attn: launch failed: %s", cudaGetErrorString(e));
    return LA_ERR_CUDA;
  }
  return LA_OK;
}

}  // namespace la
