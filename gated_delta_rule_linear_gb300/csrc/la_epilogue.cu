// The end of a block in one pass over memory, forward and backward: RMS norm of
// x over d channels, gate, residual scale, residual, and the next block's norm.
//
//   n = x r, r = 1/sqrt(mean(x^2) + eps); y = n w; out = res + scale y a(gate)
//   next = m w_next, m = out r', r' = 1/sqrt(mean(out^2) + eps)
//
// With e = d_next w_next and tot = d_out + r' (e - m mean(e m)) (the norm's
// gradient: the part of e along m does not change a normalised row), the rest
// follows by the product rule: dres = tot, dgate = tot scale y a', dscale = w A
// and dw = scale A with the one sum A = sum tot a n over all rows, and
// dx = r (f - n mean(f n)) with f = tot scale a w.
//
// Bound by HBM: every tensor once. A row of d channels stays in the registers
// of TPR threads (a power of two, as few as hold it at 16 bytes a load, up to
// 512), so the statistics, the products and both norms need no second read;
// rows are taken in a grid stride and the weights stay in registers across
// them. The backward adds its weight gradients up in registers over the rows a
// thread sees, writes one partial a CTA, and a second kernel adds the partials
// in order: no atomics, the same sums every run.
//
// At one load a thread (bf16 up to 4096 channels, float32 up to 2048) a row and
// the next one's loads fit the registers. Wider rows take up to 8 loads a thread
// and the backward then spills, up to 7 KB a thread; rows that cannot go 16
// bytes at a time have too little in flight for memory.
//
// Measured on GB300 (6.78 TB/s copy): per-head norm and silu gate of 65536 x 16
// heads of 128, bf16, head-major x: 0.156 ms, 5.15 TB/s; with the 96 registers a
// thread that the compiler takes unasked, 0.193 (too few threads a SM to cover
// memory: hence 64 at one load a thread). Backward with residual, scale, sigmoid
// gate and next norm on 32768 x 2048: 0.252 ms, 4.26 TB/s, at 53% of the issue
// slots and 47% of memory: neither is full, 512 threads a SM at 128 registers do
// not cover memory's latency. The same work on 2^26 elements of other widths,
// us forward / backward (five and eight tensors: 99 / 158 at the copy's rate in
// bf16, 198 / 317 in float32):
//   d       2048       4096       5120       8192        16384       2047         5001
//   bf16    128 / 255  134 / 288  174 / 908  122 / 589   218 / 1298  531 / 1557   1701 / 5656
//   float32 211 / 432  222 / 633  396 / 1355 335 / 1031  541 / 2847  623 / 1543   1566 / 6527
#include <cuda_bf16.h>

#include <algorithm>

#include "la_f32x2.cuh"
#include "la_layer_internal.h"

namespace la {
namespace {

using f32x2::vdot;
using f32x2::vfma;
using f32x2::vmul;

constexpr int kSums = 5;  // at most this many sums at once

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

// K sums over the tpr threads of a row; every one of them gets them. Rows wider
// than a warp meet in shared memory: `red` alternates between two halves, so
// that one barrier a call is enough.
template <int K>
__device__ __forceinline__ void row_sums(float (&v)[K], int tpr, float *red, int &turn) {
  const int lanes = tpr < 32 ? tpr : 32;
  for (int o = lanes >> 1; o; o >>= 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
  if (tpr <= 32) return;
  const int warps = tpr >> 5, per = blockDim.x >> 5, warp = threadIdx.x >> 5;
  float *r = red + (turn ? 16 * kSums : 0);
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) r[16 * k + warp] = v[k];
  }
  __syncthreads();
  // rows of 64 threads share a CTA of 128 with another row: each adds up its own warps
  const int w0 = per > warps ? warp / warps * warps : 0;
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = r[16 * k + w0 + (threadIdx.x & (warps - 1))];
  for (int o = warps >> 1; o; o >>= 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
}

// The gate's activation and its slope, in place: a becomes the value. float32
// tensors take the accurate exponential and division; for bfloat16 ones 2^x and
// 1/x of the special function unit (2^-22 each) are far below their rounding.
template <bool EXACT, bool SILU, int E, int ES>
__device__ __forceinline__ void activate(float (&a)[E], float (&slope)[ES]) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    float s;
    if constexpr (EXACT) {
      s = 1.f / (1.f + expf(-a[i]));
    } else {
      float e;
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a[i] * -1.4426950408889634f));
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
    }
    if constexpr (ES == E) slope[i] = SILU ? s * (1.f + a[i] * (1.f - s)) : s * (1.f - s);
    a[i] = SILU ? a[i] * s : s;
  }
}

// Where row (n, g) of x is: token-major (T = 0) or head-major.
struct XRows {
  FastDiv groups, tokens;
  int T, G;
};
__device__ __forceinline__ size_t x_at(const XRows &xr, int d, int row) {
  if (xr.T == 0) return (size_t)row * d;
  uint32_t n, g, b, t;
  xr.groups.split(row, n, g);
  xr.tokens.split(n, b, t);
  return (((size_t)b * xr.G + g) * xr.T + t) * d;
}

// 16 bytes (V channels) of a row as they lie in memory, so that the next row's loads can be in
// flight under this row's sums.
template <typename T, int V> struct Raw {
  uint4 u;
  __device__ __forceinline__ void load(const T *p) { u = __ldcs(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void get(float *f) const {
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
  __device__ __forceinline__ void clear() { u = make_uint4(0, 0, 0, 0); }
};
template <typename T> struct Raw<T, 1> {
  T u;
  __device__ __forceinline__ void load(const T *p) { u = *p; }
  __device__ __forceinline__ void get(float *f) const { f[0] = static_cast<float>(u); }
  __device__ __forceinline__ void clear() { u = T(0.f); }
};

template <typename T, int V, int NV, bool BWD>
__global__ void __launch_bounds__(512, !BWD && NV == 1 ? 2 : 1) epilogue_kernel(const EpilogueParams p, const XRows xr, int tpr, float *part) {
  constexpr bool exact = sizeof(T) == 4;
  constexpr int E = NV * V;
  __shared__ __align__(16) float red[2 * 16 * kSums];
  const int d = p.d, rows = p.N * p.G, lane = threadIdx.x % tpr, sub = threadIdx.x / tpr, rpb = blockDim.x / tpr;
  const float inv_d = 1.f / static_cast<float>(d);
  int turn = 0;
  float w[E], sc[E], wn[E];
  float as[BWD ? E : 1], an[BWD ? E : 1];
  auto col = [&](int i) { return (i * tpr + lane) * V; };
  const bool with_next = BWD ? p.d_next != nullptr : p.next != nullptr;
  const bool with_res = p.res && (!BWD || with_next);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      w[i * V + j] = sc[i * V + j] = wn[i * V + j] = 1.f;
      if (BWD) as[i * V + j] = an[i * V + j] = 0.f;
    }
    if (col(i) < d) {
      if (p.w) load_w<V>(p.w + col(i), w + i * V);
      if (p.scale) load_w<V>(p.scale + col(i), sc + i * V);
      if (p.w_next) load_w<V>(p.w_next + col(i), wn + i * V);
    }
  }
  vmul(w, w, sc);
  Raw<T, V> rx[NV], ra[NV], ro[NV], rg[BWD ? NV : 1], rn[BWD ? NV : 1];
  // rows and columns that are not there hold zeros
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    rx[i].clear(); ra[i].clear(); ro[i].clear();
    if constexpr (BWD) { rg[i].clear(); rn[i].clear(); }
  }
  size_t xat = 0;
  auto fetch = [&](int row) {
    if (row >= rows) return;
    xat = x_at(xr, d, row);
    const size_t at = (size_t)row * d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (col(i) >= d) continue;
      rx[i].load(static_cast<const T *>(p.x) + xat + col(i));
      if (p.gate) ra[i].load(static_cast<const T *>(p.gate) + at + col(i));
      if (with_res) ro[i].load(static_cast<const T *>(p.res) + at + col(i));
      if constexpr (BWD) {
        if (p.d_out) rg[i].load(static_cast<const T *>(p.d_out) + at + col(i));
        if (p.d_next) rn[i].load(static_cast<const T *>(p.d_next) + at + col(i));
      }
    }
  };
  // the widest rows need their registers for themselves
  constexpr bool kAhead = NV <= 2;
  const int stride = gridDim.x * rpb;
  if (kAhead) fetch(blockIdx.x * rpb + sub);
  // every thread of the CTA makes the same number of turns: the sums have barriers
  for (int first = blockIdx.x * rpb; first < rows; first += stride) {
    const int row = first + sub;
    const bool live = row < rows;
    if (!kAhead) fetch(row);
    const size_t at = (size_t)row * d, xrow = xat;
    float x[E], a[E], slope[BWD ? E : 1], o[E] = {}, g[BWD ? E : 1], gn[BWD ? E : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      rx[i].get(x + i * V);
      ra[i].get(a + i * V);
      if (with_res) ro[i].get(o + i * V);
      if constexpr (BWD) {
        rg[i].get(g + i * V);
        rn[i].get(gn + i * V);
      }
    }
    if (kAhead) fetch(row + stride);
    float sum[1] = {vdot(x, x)};
    row_sums(sum, tpr, red, turn);
    const float r = rsqrtf(sum[0] * inv_d + p.eps);
    if (!p.gate) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        a[i] = 1.f;
        if constexpr (BWD) slope[i] = 0.f;
      }
    } else if (p.act == LA_ACT_SILU) {
      activate<exact, true>(a, slope);
    } else {
      activate<exact, false>(a, slope);
    }
    vmul(x, x, r);  // n
    if constexpr (!BWD) {
      if (p.gate) vmul(x, x, a);
      if (with_res) vfma(o, x, w, o);  // w is w * scale here
      else vmul(o, x, w);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (live && col(i) < d) store<T, V>(static_cast<T *>(p.out) + at + col(i), o + i * V);
      if (with_next) {
        sum[0] = vdot(o, o);
        row_sums(sum, tpr, red, turn);
        vmul(o, o, rsqrtf(sum[0] * inv_d + p.eps));
        vmul(o, o, wn);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (live && col(i) < d) store<T, V>(static_cast<T *>(p.next) + at + col(i), o + i * V);
      }
    } else {
      // a thread without a row keeps its last one's values: they must not be added up again
      if (!live) {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = g[i] = gn[i] = o[i] = 0.f;
      }
      // With k = scale a w n: mean(f n) = mean(k tot), and tot = d_out + r' e - r'^2 mean(e m) out. So
      // all sums that are left are over products of k, out, e and d_out, and meet at one barrier.
      float y[E], k[E], c;
      vmul(y, x, w);
      vmul(k, y, a);
      if (with_next) {
        vfma(o, y, a, o);  // out
        float e[E];
        vmul(e, gn, wn);
        float s5[kSums] = {vdot(o, o), vdot(e, o), vdot(k, g), vdot(k, e), vdot(k, o)};
        row_sums(s5, tpr, red, turn);
        const float r2 = rsqrtf(s5[0] * inv_d + p.eps), em = r2 * s5[1] * inv_d, back = r2 * r2 * em;
        c = (s5[2] + (r2 * s5[3] - back * s5[4])) * inv_d;
        vfma(g, e, r2, g);
        vfma(g, o, -back, g);
        vmul(o, o, r2);  // m
        vfma(an, gn, o, an);
      } else {
        sum[0] = vdot(k, g);
        row_sums(sum, tpr, red, turn);
        c = sum[0] * inv_d;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (p.dres && live && col(i) < d) store<T, V>(static_cast<T *>(p.dres) + at + col(i), g + i * V);
      float dg[E];
      vmul(dg, g, y);
      vmul(dg, dg, slope);
      vmul(g, g, a);
      vfma(as, g, x, as);
      vmul(g, g, w);
      vfma(g, x, -c, g);
      vmul(g, g, r);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!(live && col(i) < d)) continue;
        if (p.dgate) store<T, V>(static_cast<T *>(p.dgate) + at + col(i), dg + i * V);
        if (p.dx) store<T, V>(static_cast<T *>(p.dx) + xrow + col(i), g + i * V);
      }
    }
  }
  if constexpr (BWD) {
    // this CTA's partials, [2][gridDim.x][d]; rows that shared the CTA first
    __shared__ float fold[NV == 1 ? 128 * V : 1];
    const float *acc[2] = {as, an};
    const bool want[2] = {p.dw || p.dscale, p.dw_next != nullptr};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
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

// A pair of channels of a row of raw loads.
template <typename T, int V> __device__ __forceinline__ uint64_t pair_of(const Raw<T, V> &r, int j) {
  const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
  if constexpr (sizeof(T) == 4)
    return f32x2::pair(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
  else
    return f32x2::pair(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
}
// Pairs as they are stored: one word of bf16 pairs, two of float32.
template <typename T> __device__ __forceinline__ void put_pair(uint4 &u, int j, uint64_t p) {
  uint32_t *w = &u.x;
  float f[2];
  f32x2::split(p, f);
  if constexpr (sizeof(T) == 4) {
    w[2 * j] = __float_as_uint(f[0]);
    w[2 * j + 1] = __float_as_uint(f[1]);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[0], f[1]);
    w[j] = *reinterpret_cast<const uint32_t *>(&h);
  }
}

// The backward for 16-byte loads. As the kernel above, but a row is kept as it
// was loaded and every value is formed again, pair by pair, where it is needed
// (twice: for the sums, for the gradients): with the row's values in registers
// as float32 the next row's loads did not fit beside them, and without those in
// flight the kernel waited for memory (0.46 ms against 0.31 on 32768 x 2048).
// GATE: 0 none, 1 silu, 2 sigmoid; NEXT: with the next norm's gradient; -1 (more than one load a thread): as the
// arguments say.
template <typename T, int V, int NV, int GATE, int NEXT>
__global__ void __launch_bounds__(512, 1) epilogue_bwd_kernel(const EpilogueParams p, const XRows xr, int tpr,
                                                              float *part) {
  namespace q = f32x2;
  constexpr bool exact = sizeof(T) == 4, kAhead = NV <= 2;
  constexpr int P2 = V / 2, E2 = NV * P2;
  __shared__ __align__(16) float red[2 * 16 * kSums];
  const int d = p.d, rows = p.N * p.G, lane = threadIdx.x % tpr, sub = threadIdx.x / tpr, rpb = blockDim.x / tpr;
  const float inv_d = 1.f / static_cast<float>(d);
  int turn = 0;
  auto col = [&](int i) { return (i * tpr + lane) * V; };
  const bool with_next = NEXT < 0 ? p.d_next != nullptr : NEXT != 0, with_res = p.res && with_next;
  const bool gated = GATE < 0 ? p.gate != nullptr : GATE != 0, silu = GATE < 0 ? p.act == LA_ACT_SILU : GATE == 1;
  uint64_t ws[E2], wn[E2], as[E2], an[E2];  // w scale, w_next; sums of tot a n and d_next m
#pragma unroll
  for (int i = 0; i < E2; ++i) {
    ws[i] = wn[i] = q::pair(1.f, 1.f);
    as[i] = an[i] = 0;
    const int c = col(i / P2) + 2 * (i % P2);
    if (c < d) {
      if (p.w) ws[i] = *reinterpret_cast<const uint64_t *>(p.w + c);
      if (p.scale) ws[i] = q::mul(ws[i], *reinterpret_cast<const uint64_t *>(p.scale + c));
      if (p.w_next) wn[i] = *reinterpret_cast<const uint64_t *>(p.w_next + c);
    }
  }
  Raw<T, V> nx[NV], na[NV], no[NV], ng[NV], nn[NV];  // the next row
#pragma unroll
  for (int i = 0; i < NV; ++i) nx[i].clear(), na[i].clear(), no[i].clear(), ng[i].clear(), nn[i].clear();
  size_t xat = 0;
  auto fetch = [&](int row) {
    if (row >= rows) {  // a thread without a row adds nothing to the sums
#pragma unroll
      for (int i = 0; i < NV; ++i) nx[i].clear(), na[i].clear(), no[i].clear(), ng[i].clear(), nn[i].clear();
      return;
    }
    xat = x_at(xr, d, row);
    const size_t at = (size_t)row * d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (col(i) >= d) continue;
      nx[i].load(static_cast<const T *>(p.x) + xat + col(i));
      if (gated) na[i].load(static_cast<const T *>(p.gate) + at + col(i));
      if (with_res) no[i].load(static_cast<const T *>(p.res) + at + col(i));
      if (p.d_out) ng[i].load(static_cast<const T *>(p.d_out) + at + col(i));
      if (with_next) nn[i].load(static_cast<const T *>(p.d_next) + at + col(i));
    }
  };
  // value and slope of the gate
  auto gate = [&](uint64_t a2, uint64_t &slope) {
    if (!gated) {
      slope = 0;
      return q::pair(1.f, 1.f);
    }
    float a[2], sl[2];
    q::split(a2, a);
    if (silu) activate<exact, true>(a, sl);
    else activate<exact, false>(a, sl);
    slope = q::pair(sl[0], sl[1]);
    return q::pair(a[0], a[1]);
  };
  const int stride = gridDim.x * rpb;
  if (kAhead) fetch(blockIdx.x * rpb + sub);
  for (int first = blockIdx.x * rpb; first < rows; first += stride) {
    const int row = first + sub;
    const bool live = row < rows;
    if (!kAhead) fetch(row);
    const size_t at = (size_t)row * d, xrow = xat;
    Raw<T, V> rx[NV], ra[NV], ro[NV], rg[NV], rn[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) rx[i] = nx[i], ra[i] = na[i], ro[i] = no[i], rg[i] = ng[i], rn[i] = nn[i];
    if (kAhead) fetch(row + stride);
    uint64_t t = 0;
#pragma unroll
    for (int i = 0; i < E2; ++i) {
      const uint64_t x = pair_of(rx[i / P2], i % P2);
      t = q::fma(x, x, t);
    }
    float h[2], one[1];
    q::split(t, h);
    one[0] = h[0] + h[1];
    row_sums(one, tpr, red, turn);
    const float r = rsqrtf(one[0] * inv_d + p.eps);
    const uint64_t rr = q::pair(r, r);
    // With k = scale a w n: mean(f n) = mean(k tot), and tot = d_out + r' e - r'^2 mean(e m) out. So
    // all sums that are left are over products of k, out, e and d_out, and meet at one barrier.
    uint64_t t5[kSums] = {0, 0, 0, 0, 0};  // out out, e out, k d_out, k e, k out
#pragma unroll
    for (int i = 0; i < E2; ++i) {
      uint64_t slope;
      const uint64_t y = q::mul(q::mul(pair_of(rx[i / P2], i % P2), rr), ws[i]);
      const uint64_t k = q::mul(y, gate(pair_of(ra[i / P2], i % P2), slope));
      t5[2] = q::fma(k, pair_of(rg[i / P2], i % P2), t5[2]);
      if (with_next) {
        const uint64_t o = q::add(k, pair_of(ro[i / P2], i % P2)), e = q::mul(pair_of(rn[i / P2], i % P2), wn[i]);
        t5[0] = q::fma(o, o, t5[0]);
        t5[1] = q::fma(e, o, t5[1]);
        t5[3] = q::fma(k, e, t5[3]);
        t5[4] = q::fma(k, o, t5[4]);
      }
    }
    float c, r2 = 0.f, em = 0.f;
    if (with_next) {
      float s5[kSums];
#pragma unroll
      for (int i = 0; i < kSums; ++i) {
        q::split(t5[i], h);
        s5[i] = h[0] + h[1];
      }
      row_sums(s5, tpr, red, turn);
      r2 = rsqrtf(s5[0] * inv_d + p.eps);
      em = r2 * s5[1] * inv_d;
      c = (s5[2] + (r2 * s5[3] - r2 * r2 * em * s5[4])) * inv_d;
    } else {
      q::split(t5[2], h);
      one[0] = h[0] + h[1];
      row_sums(one, tpr, red, turn);
      c = one[0] * inv_d;
    }
    const uint64_t rr2 = q::pair(r2, r2), back = q::pair(-r2 * em, -r2 * em), cc = q::pair(-c, -c);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint4 dres, dgate, dx;
#pragma unroll
      for (int j = 0; j < P2; ++j) {
        const int e2 = i * P2 + j;
        uint64_t slope;
        const uint64_t n = q::mul(pair_of(rx[i], j), rr), a = gate(pair_of(ra[i], j), slope);
        const uint64_t y = q::mul(n, ws[e2]);
        uint64_t tot = pair_of(rg[i], j);
        if (with_next) {
          const uint64_t dn = pair_of(rn[i], j), m = q::mul(q::fma(y, a, pair_of(ro[i], j)), rr2);
          tot = q::fma(q::mul(dn, wn[e2]), rr2, tot);
          tot = q::fma(m, back, tot);
          an[e2] = q::fma(dn, m, an[e2]);
        }
        put_pair<T>(dres, j, tot);
        const uint64_t ta = q::mul(tot, a);
        as[e2] = q::fma(ta, n, as[e2]);
        put_pair<T>(dgate, j, q::mul(q::mul(tot, y), slope));
        put_pair<T>(dx, j, q::mul(q::fma(n, cc, q::mul(ta, ws[e2])), rr));
      }
      if (live && col(i) < d) {
        if (p.dres) *reinterpret_cast<uint4 *>(static_cast<T *>(p.dres) + at + col(i)) = dres;
        if (p.dgate) *reinterpret_cast<uint4 *>(static_cast<T *>(p.dgate) + at + col(i)) = dgate;
        if (p.dx) *reinterpret_cast<uint4 *>(static_cast<T *>(p.dx) + xrow + col(i)) = dx;
      }
    }
  }
  // this CTA's partials, [2][gridDim.x][d]; rows that shared the CTA first
  __shared__ __align__(16) float fold[NV == 1 ? 128 * V : 4];
  const uint64_t *acc[2] = {as, an};
  const bool want[2] = {p.dw || p.dscale, p.dw_next != nullptr};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!want[k]) continue;
    float *dst = part + ((size_t)k * gridDim.x + blockIdx.x) * d;
    if (rpb == 1) {
#pragma unroll
      for (int i = 0; i < E2; ++i) {
        const int c = col(i / P2) + 2 * (i % P2);
        if (c < d) *reinterpret_cast<uint64_t *>(dst + c) = acc[k][i];
      }
    } else if constexpr (NV == 1) {  // several rows a CTA: one load a thread and 128 threads
      __syncthreads();
#pragma unroll
      for (int i = 0; i < E2; ++i) *reinterpret_cast<uint64_t *>(fold + threadIdx.x * V + 2 * i) = acc[k][i];
      __syncthreads();
      for (int c = threadIdx.x; c < d; c += blockDim.x) {
        float t = 0.f;
        for (int s = 0; s < rpb; ++s) t += fold[s * tpr * V + c];
        dst[c] = t;
      }
    }
  }
}

// Column sums of the CTAs' partials, always in the same order.
__global__ void __launch_bounds__(256) partial_sum_kernel(const float *__restrict__ part, int blocks, int d,
                                                          const EpilogueParams p) {
  __shared__ float red[8][32];
  const bool second = blockIdx.y == 1;
  if (second ? !p.dw_next : !p.dw && !p.dscale) return;
  const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float t = 0.f;
  if (c < d)
    for (int b = strand; b < blocks; b += 8) t += part[((size_t)blockIdx.y * blocks + b) * d + c];
  red[strand][lane] = t;
  __syncthreads();
  if (strand == 0 && c < d) {
    for (int s = 1; s < 8; ++s) t += red[s][lane];
    if (second) {
      p.dw_next[c] = t;
    } else {  // dw = scale sum, dscale = w sum
      const float w = p.w ? p.w[c] : 1.f, sc = p.scale ? p.scale[c] : 1.f;
      if (p.dw) p.dw[c] = t * sc;
      if (p.dscale) p.dscale[c] = t * w;
    }
  }
}

// Threads of a SM's share of the grid: as many as its registers hold at once. More CTAs only load
// the weights again and, in the backward, leave more partials to add up (with 2048 threads their
// sum took 20 of 270 us on 32768 x 2048; with 512 it takes 10 of 252).
constexpr int kForward = 1024, kBackward = 512;

struct Shape {
  int tpr, nv, threads, blocks;
  bool wide;
};

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// As few threads a row as hold it with one load each, up to 512; rows of up to
// 64 threads share a CTA of 128.
Shape shape_of(const EpilogueParams &p, int resident) {
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
  const long long most = (long long)sm_count() * std::max(1, resident / s.threads);
  const long long want = (rows + rpb - 1) / rpb;
  s.blocks = static_cast<int>(want < most ? want : most);
  return s;
}

template <typename T, bool BWD>
cudaError_t launch(const EpilogueParams &p, const Shape &s, float *part, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  const XRows xr = {FastDiv(p.G), FastDiv(p.T > 0 ? p.T : 1), p.T, p.G};
#define LA_GO(v, n)                                                                              \
  do {                                                                                           \
    if constexpr (BWD && v > 1)                                                                  \
      epilogue_bwd_kernel<T, v, n, -1, -1><<<s.blocks, s.threads, 0, stream>>>(p, xr, s.tpr, part); \
    else                                                                                         \
      epilogue_kernel<T, v, n, BWD><<<s.blocks, s.threads, 0, stream>>>(p, xr, s.tpr, part);     \
  } while (0)
  if constexpr (BWD)
    if (s.wide && s.nv == 1) {
#define LA_BWD(g, n) epilogue_bwd_kernel<T, V, 1, g, n><<<s.blocks, s.threads, 0, stream>>>(p, xr, s.tpr, part)
      const int gate = !p.gate ? 0 : p.act == LA_ACT_SILU ? 1 : 2;
      if (p.d_next) {
        if (gate == 0) LA_BWD(0, 1);
        else if (gate == 1) LA_BWD(1, 1);
        else LA_BWD(2, 1);
      } else {
        if (gate == 0) LA_BWD(0, 0);
        else if (gate == 1) LA_BWD(1, 0);
        else LA_BWD(2, 0);
      }
#undef LA_BWD
      return cudaGetLastError();
    }
  if constexpr (!BWD)
    if (s.wide && s.nv == 1) {
      LA_GO(V, 1);
      return cudaGetLastError();
    }
  // up to 16384 channels: no bfloat16 row takes eight 16-byte loads a thread
  if (s.wide) {
    if (s.nv == 2) LA_GO(V, 2);
    else if (sizeof(T) == 2 || s.nv == 4) LA_GO(V, 4);
    else if constexpr (sizeof(T) == 4) LA_GO(V, 8);
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
  const Shape s = shape_of(p, kForward);
  const cudaError_t e = p.f32 ? launch<float, false>(p, s, nullptr, stream)
                              : launch<__nv_bfloat16, false>(p, s, nullptr, stream);
  return e == cudaSuccess ? LA_OK : fail("la_epilogue", "launch failed", e);
}

int launch_epilogue_bwd(const EpilogueParams &p, cudaStream_t stream) {
  const char *fn = "la_epilogue_bwd";
  const Shape s = shape_of(p, kBackward);
  void *part = nullptr;
  cudaError_t e;
  const bool sums = p.dw || p.dscale || p.dw_next;
  if (sums) {
    cudaMemPool_t pool = library_pool();
    if (!pool) return fail(fn, "could not create the workspace pool", cudaGetLastError());
    e = cudaMallocFromPoolAsync(&part, (size_t)2 * s.blocks * p.d * 4, pool, stream);
    if (e != cudaSuccess) return fail(fn, "workspace allocation failed", e);
  }
  e = p.f32 ? launch<float, true>(p, s, static_cast<float *>(part), stream)
            : launch<__nv_bfloat16, true>(p, s, static_cast<float *>(part), stream);
  if (sums) {
    if (e == cudaSuccess) {
      partial_sum_kernel<<<dim3((p.d + 31) / 32, 2), 256, 0, stream>>>(static_cast<float *>(part), s.blocks, p.d, p);
      e = cudaGetLastError();
    }
    const cudaError_t f = cudaFreeAsync(part, stream);
    if (e == cudaSuccess) e = f;
  }
  return e == cudaSuccess ? LA_OK : fail(fn, "launch failed", e);
}

}  // namespace la
