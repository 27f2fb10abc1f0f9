// Packed retention, token by token on the CUDA cores in float32: the float32
// path of la_packed_fwd and la_packed_bwd, and either type's calls without a
// token, which take states over and read nothing else.
//
// One CTA of 128 threads owns 32 value columns of one (sequence, head) and
// walks its tokens, the state slice da x 32 in registers: thread (w, l) holds
// the rows w*da/4 .. of column l. Tokens come 16 at a time through shared
// memory; every warp's partial of out_t over its rows goes to shared memory and
// is added up once per block of tokens. The walk is bound by its own serial
// chain, about da/2 FMAs a token and warp, not by memory (4 x 16384 tokens of 16
// heads of 128: 6.9 ms, 0.42 us a token; the backward's three walks over 8 x 4096
// tokens: 6.9 ms).
#include <cuda_bf16.h>

#include "la_layer_internal.h"

namespace la {
namespace {

constexpr int kTok = 16, kCols = 32;

template <int DA>
__global__ void __launch_bounds__(128) packed_walk_kernel(const PackedPass p) {
  __shared__ __align__(16) float sx[kTok][DA], sy[kTok][DA];
  __shared__ float sz[kTok][kCols], part[kTok][4][kCols];
  constexpr int R = DA / 4;
  const int s = blockIdx.x, h = blockIdx.y, v0 = blockIdx.z * kCols;
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31, c0 = w * R, col = v0 + l;
  int a, b;
  packed_range(p.cu, s, p.total, &a, &b);
  const int slot = packed_slot(p.slots, s, p.n_slots);
  const size_t sbase = ((size_t)max(slot, 0) * p.H + h) * p.sized;
  float S[R];
#pragma unroll
  for (int c = 0; c < R; ++c) {
    const size_t at = p.in_t ? (size_t)col * DA + c0 + c : (size_t)(c0 + c) * p.db + col;
    S[c] = (p.S_in && slot >= 0) ? p.S_in[sbase + at] : 0.f;
  }
  const float *px = static_cast<const float *>(p.x), *py = static_cast<const float *>(p.y),
              *pz = static_cast<const float *>(p.z);
  const Decay decay(p.g ? __ldg(p.g + h) : 0.f, 1);
  const size_t xh = (size_t)(h / p.rx) * DA, yh = (size_t)(h / p.ry) * DA, zh = (size_t)(h / p.rz) * p.db;

  for (int done = 0; done < b - a; done += kTok) {
    const int m = min(kTok, b - a - done);
    auto token = [&](int i) { return (size_t)(p.reverse ? b - 1 - done - i : a + done + i); };
    __syncthreads();
    for (int i = threadIdx.x; i < m * DA; i += 128) {
      const size_t t = token(i / DA);
      sx[i / DA][i % DA] = px[t * p.ldx + xh + i % DA];
      sy[i / DA][i % DA] = py[t * p.ldy + yh + i % DA];
    }
    for (int i = threadIdx.x; i < m * kCols; i += 128)
      sz[i / kCols][i % kCols] = pz[token(i / kCols) * p.ldz + zh + v0 + i % kCols];
    __syncthreads();
    for (int i = 0; i < m; ++i) {
      const float z = sz[i][l];
      float o = 0.f;
#pragma unroll
      for (int c = 0; c < R; ++c) {
        const float y = sy[i][c0 + c], x = sx[i][c0 + c];
        S[c] = fmaf(y, z, p.reverse ? S[c] : decay(S[c]));
        o = fmaf(x, S[c], o);
        if (p.reverse) S[c] = decay(S[c]);
      }
      part[i][w][l] = o;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < m * kCols; i += 128) {
      const int t = i / kCols, c = i % kCols;
      const float o = (part[t][0][c] + part[t][1][c]) + (part[t][2][c] + part[t][3][c]);
      static_cast<float *>(p.out)[token(t) * p.ldo + (size_t)h * p.db + v0 + c] = o;
    }
  }
  if (p.S_out && slot >= 0)
#pragma unroll
    for (int c = 0; c < R; ++c) p.S_out[sbase + (size_t)(c0 + c) * p.db + col] = S[c];
}

// Gradients of shared heads: the float32 parts of the heads that use one. Tokens of no sequence have
// no parts, and their rows stay as they are. The sequences in use are one run of tokens, and what is
// behind them empty, a padded batch's zeros included: cu_seqlens does not fall before the last of
// them. Where it does, every sequence is summed for itself.
template <typename T>
__global__ void __launch_bounds__(256) head_sum_kernel(const float *__restrict__ src0, T *__restrict__ dst0,
                                                       const float *__restrict__ src1, T *__restrict__ dst1,
                                                       const int *__restrict__ cu, int n_seq, int total,
                                                       int heads, int share, int d) {
  const float *src = blockIdx.y ? src1 : src0;
  T *dst = blockIdx.y ? dst1 : dst0;
  const int dq = d / 4;
  const long long row = (long long)heads * dq;
  auto sum = [&](int a, int b) {
    for (long long i = a * row + blockIdx.x * 256LL + threadIdx.x; i < b * row; i += gridDim.x * 256LL) {
      const long long at = i / dq;  // (token, shared head)
      const int c = static_cast<int>(i % dq);
      const float4 *s = reinterpret_cast<const float4 *>(src + at * share * d) + c;
      float4 t = __ldcs(s);
      for (int j = 1; j < share; ++j) {
        const float4 u = __ldcs(s + (size_t)j * dq);
        t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
      }
      if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(dst)[i] = t;
      } else {
        __nv_bfloat162 u[2] = {__floats2bfloat162_rn(t.x, t.y), __floats2bfloat162_rn(t.z, t.w)};
        reinterpret_cast<uint2 *>(dst)[i] = *reinterpret_cast<uint2 *>(u);
      }
    }
  };
  __shared__ int falls, last;  // the first bound behind which they fall, the last sequence with a token
  if (threadIdx.x == 0) falls = n_seq, last = -1;
  __syncthreads();
  auto bound = [&](int s) { return min(max(__ldg(cu + s), 0), total); };
  for (int s = threadIdx.x; s < n_seq; s += 256) {
    const int a = bound(s), b = bound(s + 1);
    if (b < a) atomicMin(&falls, s);
    if (b > a) atomicMax(&last, s);
  }
  __syncthreads();
  if (last < falls) {
    sum(bound(0), bound(falls));
  } else {
    for (int s = 0; s <= last; ++s) sum(bound(s), max(bound(s), bound(s + 1)));
  }
}

}  // namespace

int launch_packed_walk(const PackedPass &p, cudaStream_t stream) {
  const dim3 grid(p.n_seq, p.H, p.db / kCols);
  if (p.da == 64) packed_walk_kernel<64><<<grid, 128, 0, stream>>>(p);
  else packed_walk_kernel<128><<<grid, 128, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("packed retention: launch failed: %s", cudaGetErrorString(e));
    return LA_ERR_CUDA;
  }
  return LA_OK;
}

int launch_head_sums(const float *const src[2], void *const dst[2], int f32, const int *cu, int n_seq, int total,
                     int Hk, int share, int d, cudaStream_t stream) {
  const long long quads = (long long)total * Hk * (d / 4);
  if (quads == 0) return LA_OK;
  // as many CTAs as are resident, eight a SM: each looks through the bounds once
  const long long want = (quads + 255) / 256, most = 4LL * (sm_count() > 0 ? sm_count() : 1);
  const dim3 grid(static_cast<unsigned>(want < most ? want : most), 2);
  if (f32)
    head_sum_kernel<<<grid, 256, 0, stream>>>(src[0], static_cast<float *>(dst[0]), src[1], static_cast<float *>(dst[1]),
                                              cu, n_seq, total, Hk, share, d);
  else
    head_sum_kernel<<<grid, 256, 0, stream>>>(src[0], static_cast<__nv_bfloat16 *>(dst[0]), src[1],
                                              static_cast<__nv_bfloat16 *>(dst[1]), cu, n_seq, total, Hk, share, d);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("la_packed_bwd: head sum launch failed: %s", cudaGetErrorString(e));
    return LA_ERR_CUDA;
  }
  return LA_OK;
}

}  // namespace la
