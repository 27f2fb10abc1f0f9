// The end of a block in one pass over memory, forward and backward: RMS norm of
// x over d channels, gate, residual scale, residual, and the next block's norm.
//
//   n = x r, r = 1/sqrt(mean(x^2) + eps); y = n w; out = res + scale y a(gate)
//   next = m w_next, m = out r', r' = 1/sqrt(mean(out^2) + eps)
//
// With e = d_next w_next and tot = d_out + r' (e - m mean(e m)) (the norm's
// gradient: the part of e along m does not change a normalised row), the rest
// follows by the product rule: dres = tot, dscale = sum tot y a,
// dgate = tot scale y a', dw = sum tot scale a n, and dx = r (f - n mean(f n))
// with f = tot scale a w.
//
// Bound by HBM: every tensor once. A row of d channels stays in the registers
// of TPR threads (a power of two, as few as hold it at 16 bytes a load, up to
// 512), so the statistics, the products and both norms need no second read;
// rows are taken in a grid stride and the weights stay in registers across
// them. The backward adds its weight gradients up in registers over the rows a
// thread sees, writes one partial a CTA, and a second kernel adds the partials
// in order: no atomics, the same sums every run.
#include <cuda_bf16.h>

#include "la_layer_internal.h"

namespace la {
namespace {

template <typename T, int V>
__device__ __forceinline__ void load(const T *p, float *f) {
  if constexpr (V == 1) {
    f[0] = static_cast<float>(*p);
  } else {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        f[i] = __uint_as_float(w[i]);
      } else {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void store(T *p, const float *f) {
  if constexpr (V == 1) {
    *p = T(f[0]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<uint4 *>(h);
  }
}
template <int V>
__device__ __forceinline__ void load_w(const float *p, float *f) {
  if constexpr (V == 1) {
    f[0] = __ldg(p);
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 t = __ldg(reinterpret_cast<const float4 *>(p) + i);
      f[4 * i] = t.x; f[4 * i + 1] = t.y; f[4 * i + 2] = t.z; f[4 * i + 3] = t.w;
    }
  }
}

// Sum over the tpr threads of a row; every one of them gets it. Rows wider than
// a warp own the whole CTA: `red` alternates between two halves so that one
// barrier a sum is enough.
__device__ __forceinline__ float row_sum(float v, int tpr, float *red, int &turn) {
  const int lanes = tpr < 32 ? tpr : 32;
  for (int o = lanes >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (tpr <= 32) return v;
  const int warps = tpr >> 5, per = blockDim.x >> 5;
  float *r = red + (turn ? 16 : 0);
  turn ^= 1;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) r[warp] = v;
  __syncthreads();
  // rows of 64 threads share a CTA of 128 with another row: each adds up its own warps
  const int w0 = per > warps ? warp / warps * warps : 0;
  float s = 0.f;
  for (int i = 0; i < warps; ++i) s += r[w0 + i];
  return s;
}

// The gate's activation and its slope.
template <bool EXACT>
__device__ __forceinline__ void activate(float a, int act, float *value, float *slope) {
  const float e = EXACT ? expf(-a) : __expf(-a);
  const float s = EXACT ? 1.f / (1.f + e) : __fdividef(1.f, 1.f + e);
  if (act == LA_ACT_SIGMOID) {
    *value = s;
    *slope = s * (1.f - s);
  } else {
    *value = a * s;
    *slope = s * (1.f + a * (1.f - s));
  }
}

__device__ __forceinline__ size_t x_at(const EpilogueParams &p, int row) {
  if (p.T == 0) return (size_t)row * p.d;
  const int n = row / p.G, g = row % p.G;
  return (((size_t)(n / p.T) * p.G + g) * p.T + n % p.T) * p.d;
}

template <typename T, int V, int NV, bool BWD>
__global__ void __launch_bounds__(512) epilogue_kernel(const EpilogueParams p, int tpr, float *part) {
  constexpr bool exact = sizeof(T) == 4;
  __shared__ float red[32];
  const int d = p.d, rows = p.N * p.G, lane = threadIdx.x % tpr, sub = threadIdx.x / tpr, rpb = blockDim.x / tpr;
  const float inv_d = 1.f / static_cast<float>(d);
  int turn = 0;
  float w[NV * V], sc[NV * V], wn[NV * V];
  float aw[BWD ? NV * V : 1], as[BWD ? NV * V : 1], an[BWD ? NV * V : 1];
  auto col = [&](int i) { return (i * tpr + lane) * V; };
  const bool with_next = BWD ? p.d_next != nullptr : p.next != nullptr;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      w[i * V + j] = sc[i * V + j] = wn[i * V + j] = 1.f;
      if (BWD) aw[i * V + j] = as[i * V + j] = an[i * V + j] = 0.f;
    }
    if (col(i) < d) {
      if (p.w) load_w<V>(p.w + col(i), w + i * V);
      if (p.scale) load_w<V>(p.scale + col(i), sc + i * V);
      if (p.w_next) load_w<V>(p.w_next + col(i), wn + i * V);
    }
  }
  // every thread of the CTA makes the same number of turns: the sums have barriers
  for (int first = blockIdx.x * rpb; first < rows; first += gridDim.x * rpb) {
    const int row = first + sub;
    const bool live = row < rows;
    const size_t at = (size_t)row * d, xat = live ? x_at(p, row) : 0;
    float x[NV * V], a[NV * V], slope[BWD ? NV * V : 1], o[NV * V];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = live && col(i) < d;
#pragma unroll
      for (int j = 0; j < V; ++j) x[i * V + j] = a[i * V + j] = o[i * V + j] = 0.f;
      if (in) {
        load<T, V>(static_cast<const T *>(p.x) + xat + col(i), x + i * V);
        if (p.gate) load<T, V>(static_cast<const T *>(p.gate) + at + col(i), a + i * V);
        if (p.res && (!BWD || with_next)) load<T, V>(static_cast<const T *>(p.res) + at + col(i), o + i * V);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(x[i * V + j], x[i * V + j], ss);
    }
    float g[BWD ? NV * V : 1], gn[BWD ? NV * V : 1];  // d_out, d_next
    if constexpr (BWD) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j) g[i * V + j] = gn[i * V + j] = 0.f;
        if (live && col(i) < d) {
          if (p.d_out) load<T, V>(static_cast<const T *>(p.d_out) + at + col(i), g + i * V);
          if (p.d_next) load<T, V>(static_cast<const T *>(p.d_next) + at + col(i), gn + i * V);
        }
      }
    }
    const float r = rsqrtf(row_sum(ss, tpr, red, turn) * inv_d + p.eps);
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV * V; ++i) {
      x[i] *= r;  // n
      float value = 1.f, sl = 0.f;
      if (p.gate) activate<exact>(a[i], p.act, &value, &sl);
      a[i] = value;
      if constexpr (BWD) slope[i] = sl;
      o[i] = fmaf(sc[i] * (x[i] * w[i]), value, o[i]);
      ss = fmaf(o[i], o[i], ss);
    }
    if constexpr (!BWD) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (live && col(i) < d) store<T, V>(static_cast<T *>(p.out) + at + col(i), o + i * V);
      if (with_next) {
        // columns behind d and rows behind the last hold zeros
        const float r2 = rsqrtf(row_sum(ss, tpr, red, turn) * inv_d + p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
          for (int j = 0; j < V; ++j) o[i * V + j] *= r2 * wn[i * V + j];
          if (live && col(i) < d) store<T, V>(static_cast<T *>(p.next) + at + col(i), o + i * V);
        }
      }
    } else {
      if (with_next) {
        const float r2 = rsqrtf(row_sum(ss, tpr, red, turn) * inv_d + p.eps);
        float c = 0.f;
#pragma unroll
        for (int i = 0; i < NV * V; ++i) {
          o[i] *= r2;  // m
          an[i] = fmaf(gn[i], o[i], an[i]);
          gn[i] *= wn[i];
          c = fmaf(gn[i], o[i], c);
        }
        c = row_sum(c, tpr, red, turn) * inv_d;
#pragma unroll
        for (int i = 0; i < NV * V; ++i) g[i] = fmaf(r2, gn[i] - o[i] * c, g[i]);
      }
      float c = 0.f;
      float dg[NV * V];
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (p.dres && live && col(i) < d) store<T, V>(static_cast<T *>(p.dres) + at + col(i), g + i * V);
#pragma unroll
      for (int i = 0; i < NV * V; ++i) {
        const float y = x[i] * w[i];
        as[i] = fmaf(g[i], y * a[i], as[i]);
        const float t = g[i] * sc[i];
        dg[i] = t * y * slope[i];
        const float ta = t * a[i];
        aw[i] = fmaf(ta, x[i], aw[i]);
        g[i] = ta * w[i];
        c = fmaf(g[i], x[i], c);
      }
      c = row_sum(c, tpr, red, turn) * inv_d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!(live && col(i) < d)) continue;
        if (p.dgate) store<T, V>(static_cast<T *>(p.dgate) + at + col(i), dg + i * V);
        if (p.dx) {
          float t[V];
#pragma unroll
          for (int j = 0; j < V; ++j) t[j] = r * (g[i * V + j] - x[i * V + j] * c);
          store<T, V>(static_cast<T *>(p.dx) + xat + col(i), t);
        }
      }
    }
  }
  if constexpr (BWD) {
    // this CTA's partials, [3][gridDim.x][d]; rows that shared the CTA first
    __shared__ float fold[NV == 1 ? 128 * V : 1];
    const float *acc[3] = {aw, as, an};
    const bool want[3] = {p.dw != nullptr, p.dscale != nullptr, p.dw_next != nullptr};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (!want[k]) continue;
      float *dst = part + ((size_t)k * gridDim.x + blockIdx.x) * d;
      if (rpb == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (col(i) < d) dst[col(i) + j] = acc[k][i * V + j];
      } else if constexpr (NV == 1) {  // several rows a CTA: one load a thread and 128 threads
        __syncthreads();
#pragma unroll
        for (int j = 0; j < V; ++j) fold[threadIdx.x * V + j] = acc[k][j];
        __syncthreads();
        for (int c = threadIdx.x; c < d; c += blockDim.x) {
          float t = 0.f;
          for (int s = 0; s < rpb; ++s) t += fold[s * tpr * V + c];
          dst[c] = t;
        }
      }
    }
  }
}

// Column sums of the CTAs' partials, always in the same order.
__global__ void __launch_bounds__(256) partial_sum_kernel(const float *__restrict__ part, int blocks, int d,
                                                          float *dw, float *dscale, float *dw_next) {
  __shared__ float red[8][32];
  float *dst = blockIdx.y == 0 ? dw : blockIdx.y == 1 ? dscale : dw_next;
  if (!dst) return;
  const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float t = 0.f;
  if (c < d)
    for (int b = strand; b < blocks; b += 8) t += part[((size_t)blockIdx.y * blocks + b) * d + c];
  red[strand][lane] = t;
  __syncthreads();
  if (strand == 0 && c < d) {
    for (int s = 1; s < 8; ++s) t += red[s][lane];
    dst[c] = t;
  }
}

struct Shape {
  int tpr, nv, threads, blocks;
  bool wide;
};

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// As few threads a row as hold it with one load each, up to 512; rows of up to
// 64 threads share a CTA of 128.
Shape shape_of(const EpilogueParams &p) {
  Shape s;
  const int V = p.f32 ? 4 : 8;
  s.wide = p.d % V == 0;
  const void *all[] = {p.x, p.gate, p.res, p.d_out, p.d_next, p.w, p.scale, p.w_next, p.out, p.next, p.dx, p.dgate,
                       p.dres};
  for (const void *q : all) s.wide = s.wide && aligned16(q);
  const int loads = s.wide ? p.d / V : p.d;
  s.tpr = 1;
  while (s.tpr < loads && s.tpr < 512) s.tpr *= 2;
  s.nv = 1;
  while (s.tpr * s.nv < loads) s.nv *= 2;
  s.threads = s.tpr < 128 ? 128 : s.tpr;
  const long long rows = (long long)p.N * p.G, rpb = s.threads / s.tpr;
  const long long most = (long long)sm_count() * (1024 / s.threads);
  const long long want = (rows + rpb - 1) / rpb;
  s.blocks = static_cast<int>(want < most ? want : most);
  return s;
}

template <typename T, bool BWD>
cudaError_t launch(const EpilogueParams &p, const Shape &s, float *part, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
#define LA_GO(v, n) epilogue_kernel<T, v, n, BWD><<<s.blocks, s.threads, 0, stream>>>(p, s.tpr, part)
  if (s.wide) {
    if (s.nv == 1) LA_GO(V, 1);
    else if (s.nv == 2) LA_GO(V, 2);
    else if (s.nv == 4) LA_GO(V, 4);
    else LA_GO(V, 8);
  } else {
    if (s.nv == 1) LA_GO(1, 1);
    else if (s.nv <= 8) LA_GO(1, 8);
    else LA_GO(1, 32);
  }
#undef LA_GO
  return cudaGetLastError();
}

int fail(const char *fn, const char *what, cudaError_t e) {
  set_error("%s: %s: %s", fn, what, cudaGetErrorString(e));
  return LA_ERR_CUDA;
}

}  // namespace

int launch_epilogue(const EpilogueParams &p, cudaStream_t stream) {
  const Shape s = shape_of(p);
  const cudaError_t e = p.f32 ? launch<float, false>(p, s, nullptr, stream)
                              : launch<__nv_bfloat16, false>(p, s, nullptr, stream);
  return e == cudaSuccess ? LA_OK : fail("la_epilogue", "launch failed", e);
}

int launch_epilogue_bwd(const EpilogueParams &p, cudaStream_t stream) {
  const char *fn = "la_epilogue_bwd";
  const Shape s = shape_of(p);
  void *part = nullptr;
  cudaError_t e;
  const bool sums = p.dw || p.dscale || p.dw_next;
  if (sums) {
    cudaMemPool_t pool = library_pool();
    if (!pool) return fail(fn, "could not create the workspace pool", cudaGetLastError());
    e = cudaMallocFromPoolAsync(&part, (size_t)3 * s.blocks * p.d * 4, pool, stream);
    if (e != cudaSuccess) return fail(fn, "workspace allocation failed", e);
  }
  e = p.f32 ? launch<float, true>(p, s, static_cast<float *>(part), stream)
            : launch<__nv_bfloat16, true>(p, s, static_cast<float *>(part), stream);
  if (sums) {
    if (e == cudaSuccess) {
      partial_sum_kernel<<<dim3((p.d + 31) / 32, 3), 256, 0, stream>>>(static_cast<float *>(part), s.blocks, p.d,
                                                                      p.dw, p.dscale, p.dw_next);
      e = cudaGetLastError();
    }
    const cudaError_t f = cudaFreeAsync(part, stream);
    if (e == cudaSuccess) e = f;
  }
  return e == cudaSuccess ? LA_OK : fail(fn, "launch failed", e);
}

}  // namespace la
