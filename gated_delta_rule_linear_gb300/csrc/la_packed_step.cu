// One token for each of n requests on a pool of retention states:
// S <- gamma_h S + k v^T in place, o = S^T q ("Talk Linear Attention" section
// 2.1, the recurrent form), float32 state.
//
// Bound by the states' HBM traffic, 2*dk*dv*4 bytes a row and head. One CTA of
// 256 threads takes one (row, head): its states are dk rows of dv floats, a
// thread holds 4 neighbouring columns of every (1024/dv)-th row, all loads of
// the thread (16 of 16 bytes at 128 x 128) in flight before the first use. A
// thread adds up o over its rows, the CTA over its row groups in shared memory.
// 128 rows of 16 heads of 128 x 128: 45 us, 6.0 TB/s (88% of the measured copy).
#include <cuda_bf16.h>

#include "la_layer_internal.h"

namespace la {
namespace {

constexpr int kThreads = 256;

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(kThreads) packed_step_kernel(const PackedStep p) {
  constexpr int kQuads = DV / 4, kGroups = kThreads / kQuads, kRows = DK / kGroups;
  __shared__ float sq[DK], sk[DK];
  __shared__ __align__(16) float so[kGroups][DV];
  const int h = blockIdx.x % p.H, row = blockIdx.x / p.H, tid = threadIdx.x;
  const int cq = tid % kQuads, rg = tid / kQuads;
  const int slot = p.slots ? __ldg(p.slots + row) : row;
  T *o = static_cast<T *>(p.o);
  if (slot < 0 || slot >= p.n_slots) {  // padding row
    for (int c = tid; c < DV; c += kThreads) o[((size_t)row * p.H + h) * DV + c] = T(0.f);
    return;
  }
  float4 S[kRows];
  float4 *base = reinterpret_cast<float4 *>(p.S + ((size_t)slot * p.H + h) * DK * DV) + cq;
#pragma unroll
  for (int i = 0; i < kRows; ++i) S[i] = __ldcs(base + (size_t)(i * kGroups + rg) * kQuads);
  // rows that share a slot are one chain, walked by the CTA of its first row
  int next = p.n;
  if (p.slots) {
    int seen = 0;
    for (int j = tid; j < p.n; j += kThreads)
      if (j != row && __ldg(p.slots + j) == slot) seen |= j < row ? 1 : 2;
    seen = __syncthreads_or(seen);  // non-zero if any: which, by a second look
    if (seen) {
      int before = 0, mine = p.n;
      for (int j = tid; j < p.n; j += kThreads)
        if (__ldg(p.slots + j) == slot) {
          if (j < row) before = 1;
          if (j > row) mine = min(mine, j);
        }
      if (__syncthreads_or(before)) return;
      __shared__ int nearest;
      if (tid == 0) nearest = p.n;
      __syncthreads();
      atomicMin(&nearest, mine);
      __syncthreads();
      next = nearest;
    }
  }
  const Decay decay(p.g ? __ldg(p.g + h) : 0.f, 1);
  const size_t hk = (size_t)(h / (p.H / p.Hk)) * DK;
  for (int r = row; r < p.n;) {
    for (int c = tid; c < DK; c += kThreads) {
      sq[c] = static_cast<float>(static_cast<const T *>(p.q)[r * p.ldq + hk + c]);
      sk[c] = static_cast<float>(static_cast<const T *>(p.k)[r * p.ldk + hk + c]);
    }
    float v[4];
    const T *vr = static_cast<const T *>(p.v) + r * p.ldv + (size_t)h * DV + cq * 4;
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = static_cast<float>(vr[c]);
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float k = sk[i * kGroups + rg], q = sq[i * kGroups + rg];
      S[i].x = fmaf(k, v[0], decay(S[i].x));
      S[i].y = fmaf(k, v[1], decay(S[i].y));
      S[i].z = fmaf(k, v[2], decay(S[i].z));
      S[i].w = fmaf(k, v[3], decay(S[i].w));
      acc.x = fmaf(q, S[i].x, acc.x);
      acc.y = fmaf(q, S[i].y, acc.y);
      acc.z = fmaf(q, S[i].z, acc.z);
      acc.w = fmaf(q, S[i].w, acc.w);
    }
    *reinterpret_cast<float4 *>(&so[rg][cq * 4]) = acc;
    __syncthreads();
    for (int c = tid; c < DV; c += kThreads) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) t += so[i][c];
      o[((size_t)r * p.H + h) * DV + c] = T(t);
    }
    if (next >= p.n) break;
    r = next;
    __syncthreads();
    for (next = r + 1; next < p.n && __ldg(p.slots + next) != slot;) ++next;
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) __stcs(base + (size_t)(i * kGroups + rg) * kQuads, S[i]);
}

template <typename T>
void launch(const PackedStep &p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.n) * p.H;  // the caller keeps n * H below 2^31
  if (p.dk == 128 && p.dv == 128) packed_step_kernel<T, 128, 128><<<grid, kThreads, 0, stream>>>(p);
  else if (p.dk == 128) packed_step_kernel<T, 128, 64><<<grid, kThreads, 0, stream>>>(p);
  else if (p.dv == 128) packed_step_kernel<T, 64, 128><<<grid, kThreads, 0, stream>>>(p);
  else packed_step_kernel<T, 64, 64><<<grid, kThreads, 0, stream>>>(p);
}

}  // namespace

int launch_packed_step(const PackedStep &p, cudaStream_t stream) {
  if (p.f32) launch<float>(p, stream);
  else launch<__nv_bfloat16>(p, stream);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("la_packed_step: launch failed: %s", cudaGetErrorString(e));
    return LA_ERR_CUDA;
  }
  return LA_OK;
}

}  // namespace la
