// Host side of include/la_layer.h: argument checks, the choice of kernel, and
// the workspaces of the layer operators.
#include <climits>
#include <cmath>

#include "la_check.h"
#include "la_layer_internal.h"

using namespace la;

namespace {

// LA_LINEAR or LA_RETNET, with or without LA_F32; heads and widths.
int check_packed(const char *fn, int mode, const float *g, int H, int Hk, int dk, int dv, long long ldq,
                 long long ldk, long long ldv) {
  const int kind = mode & 0xff;
  if ((mode & ~(0xff | LA_F32)) != 0 || kind > LA_OUTER_GATE) {
    set_error("%s: unknown mode 0x%x", fn, mode);
    return LA_ERR_INVALID_ARG;
  }
  if (kind != LA_LINEAR && kind != LA_RETNET) {
    set_error("%s: takes LA_LINEAR and LA_RETNET (got mode %d)", fn, kind);
    return LA_ERR_UNSUPPORTED;
  }
  if ((kind == LA_RETNET) != (g != nullptr)) return bad(fn, "g goes with LA_RETNET, and only with it");
  if (H < 1 || Hk < 1 || H % Hk != 0 || H > 65535) return bad(fn, "H must be a multiple of Hk, 1 <= H <= 65535");
  if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) {
    set_error("%s: dk and dv must be 64 or 128 (got %d, %d)", fn, dk, dv);
    return LA_ERR_UNSUPPORTED;
  }
  const int unit = (mode & LA_F32) ? 4 : 8;
  if (ldq < (long long)Hk * dk || ldk < (long long)Hk * dk || ldv < (long long)H * dv || ldq % unit || ldk % unit ||
      ldv % unit || ldq > INT_MAX || ldk > INT_MAX || ldv > INT_MAX)
    return bad(fn, "token strides must cover a token's heads, in multiples of 16 bytes below 2^31 elements");
  if (!at(g, 4)) return bad(fn, "g must be 4-byte aligned");
  return LA_OK;
}

int check_packing(const char *fn, const int *cu, const int *slots, int n_seq, int total, int max_len) {
  if (!cu) return bad(fn, "cu_seqlens is required");
  if (n_seq < 1 || total < 0 || max_len < 0) return bad(fn, "n_seq must be >= 1, total and max_len >= 0");
  if (!at(cu, 4) || !at(slots, 4)) return bad(fn, "cu_seqlens and slots must be 4-byte aligned");
  return LA_OK;
}

// float32 and calls without a token go to the walk, bfloat16 to the tensor cores.
int run_passes(const PackedPass *p, int passes, cudaStream_t stream) {
  if (!p->f32 && p->total > 0) return launch_packed_tc(p, passes, stream);
  int rc = LA_OK;
  for (int i = 0; i < passes && rc == LA_OK; ++i) rc = launch_packed_walk(p[i], stream);
  return rc;
}

}  // namespace

extern "C" {

int la_packed_fwd(const void *q, const void *k, const void *v, const float *g, void *o, const float *S0,
                  float *S_final, const int *cu_seqlens, const int *slots, int n_seq, int total, int max_len,
                  int n_slots, int H, int Hk, int dk, int dv, long long ldq, long long ldk, long long ldv,
                  int mode, la_stream_t stream) {
  NvtxRange nvtx_range("la_packed_fwd");
  const char *fn = "la_packed_fwd";
  set_error("%s", "");
  int rc = check_packed(fn, mode, g, H, Hk, dk, dv, ldq, ldk, ldv);
  if (rc) return rc;
  rc = check_packing(fn, cu_seqlens, slots, n_seq, total, max_len);
  if (rc) return rc;
  if (total > 0 && (!q || !k || !v || !o)) return bad(fn, "q, k, v and o are required");
  if (!at(q, 16) || !at(k, 16) || !at(v, 16) || !at(o, 16) || !at(S0, 16) || !at(S_final, 16))
    return bad(fn, "tensors must be 16-byte aligned");
  if ((S0 || S_final) && (n_slots < 0 || (!slots && n_slots < n_seq)))
    return bad(fn, "n_slots must be >= 0, and >= n_seq without slots");
  if (total > 0 && same({o}, {q, k, v})) return bad(fn, "o must not be an input");
  unsigned *status = status_word();
  if (!status) {
    set_error("%s: no CUDA device available (%s)", fn, cudaGetErrorString(cudaGetLastError()));
    return LA_ERR_CUDA;
  }
  PackedPass p = {};
  p.x = q; p.y = k; p.z = v; p.out = o;
  p.ldx = ldq; p.ldy = ldk; p.ldz = ldv; p.ldo = (long long)H * dv;
  p.rx = p.ry = H / Hk; p.rz = 1;
  p.da = dk; p.db = dv; p.sized = dk * dv;
  p.S_in = S0; p.S_out = S_final;
  p.cu = cu_seqlens; p.slots = slots; p.n_seq = n_seq; p.total = total; p.n_slots = n_slots; p.H = H;
  p.g = g; p.f32 = p.out_f32 = (mode & LA_F32) ? 1 : 0;
  p.status = status; p.max_len = max_len;
  return run_passes(&p, 1, reinterpret_cast<cudaStream_t>(stream));
}

int la_packed_bwd(const void *q, const void *k, const void *v, const float *g, const void *dO,
                  const float *S0, const float *dS_final, void *dq, void *dk_out, void *dv_out, float *dS0,
                  const int *cu_seqlens, int n_seq, int total, int max_len, int H, int Hk, int dk, int dv,
                  long long ldq, long long ldk, long long ldv, int mode, la_stream_t stream) {
  NvtxRange nvtx_range("la_packed_bwd");
  const char *fn = "la_packed_bwd";
  set_error("%s", "");
  int rc = check_packed(fn, mode, g, H, Hk, dk, dv, ldq, ldk, ldv);
  if (rc) return rc;
  rc = check_packing(fn, cu_seqlens, nullptr, n_seq, total, max_len);
  if (rc) return rc;
  if (total > 0 && (!q || !k || !v || !dO || !dq || !dk_out || !dv_out))
    return bad(fn, "q, k, v, dO, dq, dk_out and dv_out are required");
  const void *all[] = {q, k, v, dO, S0, dS_final, dq, dk_out, dv_out, dS0};
  for (const void *t : all)
    if (!at(t, 16)) return bad(fn, "tensors must be 16-byte aligned");
  if ((total > 0 && same({dq, dk_out, dv_out}, {q, k, v, dO})) || same({dS0}, {S0, dS_final}))
    return bad(fn, "outputs must not be inputs, nor one another");
  unsigned *status = status_word();
  if (!status) {
    set_error("%s: no CUDA device available (%s)", fn, cudaGetErrorString(cudaGetLastError()));
    return LA_ERR_CUDA;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int share = H / Hk, f32 = (mode & LA_F32) ? 1 : 0;
  // gradients of shared heads: one float32 part per head, then their sum
  float *parts = nullptr;
  if (share > 1 && total > 0) {
    cudaMemPool_t pool = library_pool();
    if (!pool) {
      set_error("%s: could not create the workspace pool: %s", fn, cudaGetErrorString(cudaGetLastError()));
      return LA_ERR_CUDA;
    }
    const size_t bytes = (size_t)2 * total * H * dk * 4;  // of dq and dk
    const cudaError_t e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&parts), bytes, pool, s);
    if (e != cudaSuccess) {
      set_error("%s: workspace allocation of %zu bytes failed: %s", fn, bytes, cudaGetErrorString(e));
      return LA_ERR_CUDA;
    }
  }
  const long long ldd = (long long)H * dv;
  PackedPass c = {};
  c.sized = dk * dv;
  c.cu = cu_seqlens; c.n_seq = n_seq; c.total = total; c.n_slots = n_seq; c.H = H;
  c.g = g; c.f32 = f32; c.status = status; c.max_len = max_len;
  float *parts_of[2] = {parts, parts ? parts + (size_t)total * H * dk : nullptr};
  void *summed[2] = {dq, dk_out};
  auto shared_out = [&](PackedPass &p, int i, void *dst) {
    p.out = parts ? parts_of[i] : dst;
    p.ldo = parts ? (long long)H * dk : (long long)Hk * dk;
    p.out_f32 = parts ? 1 : f32;
  };
  PackedPass p[3] = {c, c, c};
  p[0].x = dO; p[0].ldx = ldd; p[0].rx = 1;  // dq
  p[0].y = v; p[0].ldy = ldv; p[0].ry = 1;
  p[0].z = k; p[0].ldz = ldk; p[0].rz = share;
  p[0].da = dv; p[0].db = dk; p[0].S_in = S0; p[0].in_t = 1;
  shared_out(p[0], 0, dq);
  p[1].reverse = 1;  // dk
  p[1].x = v; p[1].ldx = ldv; p[1].rx = 1;
  p[1].y = dO; p[1].ldy = ldd; p[1].ry = 1;
  p[1].z = q; p[1].ldz = ldq; p[1].rz = share;
  p[1].da = dv; p[1].db = dk; p[1].S_in = dS_final; p[1].in_t = 1;
  shared_out(p[1], 1, dk_out);
  p[2].reverse = 1;  // dv and dS0
  p[2].x = k; p[2].ldx = ldk; p[2].rx = share;
  p[2].y = q; p[2].ldy = ldq; p[2].ry = share;
  p[2].z = dO; p[2].ldz = ldd; p[2].rz = 1;
  p[2].da = dk; p[2].db = dv; p[2].S_in = dS_final; p[2].S_out = dS0;
  p[2].out = dv_out; p[2].ldo = ldd; p[2].out_f32 = f32;
  rc = run_passes(p, 3, s);
  if (parts && rc == LA_OK) rc = launch_head_sums(parts_of, summed, f32, cu_seqlens, n_seq, total, Hk, share, dk, s);
  if (parts) {
    const cudaError_t e = cudaFreeAsync(parts, s);
    if (rc == LA_OK && e != cudaSuccess) {
      set_error("%s: workspace release failed: %s", fn, cudaGetErrorString(e));
      return LA_ERR_CUDA;
    }
  }
  return rc;
}

int la_packed_step(const void *q, const void *k, const void *v, const float *g, void *o, float *S,
                   const int *slots, int n, int n_slots, int H, int Hk, int dk, int dv, long long ldq,
                   long long ldk, long long ldv, int mode, la_stream_t stream) {
  NvtxRange nvtx_range("la_packed_step");
  const char *fn = "la_packed_step";
  set_error("%s", "");
  const int rc = check_packed(fn, mode, g, H, Hk, dk, dv, ldq, ldk, ldv);
  if (rc) return rc;
  if (n < 0 || n_slots < 0 || (!slots && n > n_slots)) return bad(fn, "n must be >= 0, and <= n_slots without slots");
  if ((long long)n * H > INT_MAX) return bad(fn, "n*H too large");
  if (n == 0) return LA_OK;
  if (!q || !k || !v || !o || !S) return bad(fn, "q, k, v, o and S are required");
  if (!at(q, 16) || !at(k, 16) || !at(v, 16) || !at(o, 16) || !at(S, 16) || !at(slots, 4))
    return bad(fn, "tensors must be 16-byte aligned, slots 4-byte aligned");
  if (same({o}, {q, k, v})) return bad(fn, "o must not be an input");
  const PackedStep p = {q, k, v, o, S, g, slots, n, n_slots, H, Hk, dk, dv, (mode & LA_F32) ? 1 : 0, ldq, ldk, ldv};
  return launch_packed_step(p, reinterpret_cast<cudaStream_t>(stream));
}

int la_rotary(const void *q, const void *k, void *q_out, void *k_out, const int *pos, const double *freq,
              int n_axes, int s0, int s1, int s2, int N, int H, int Hk, int d, int T_in, int T_out,
              long long ldq, long long ldk, float scale_q, float scale_k, int flags, la_stream_t stream) {
  NvtxRange nvtx_range("la_rotary");
  const char *fn = "la_rotary";
  set_error("%s", "");
  if (flags & ~(LA_F32 | LA_ROT_INTERLEAVED | LA_ROT_INVERSE)) return bad(fn, "unknown flag");
  if ((k != nullptr) != (k_out != nullptr)) return bad(fn, "k and k_out go together");
  if (N < 0 || H < 1 || (k && Hk < 1) || H > 65535 || Hk > 65535) return bad(fn, "N must be >= 0, H and Hk 1..65535");
  if (n_axes < 1 || n_axes > 3 || s0 < 0 || s1 < 0 || s2 < 0 || (n_axes < 2 && s1) || (n_axes < 3 && s2))
    return bad(fn, "n_axes must be 1..3, with s_a = 0 for the axes that are not there");
  if (d < 2 || d > 512) {
    set_error("%s: d must be 2..512 (got %d)", fn, d);
    return LA_ERR_UNSUPPORTED;
  }
  const long long P = (long long)s0 + s1 + s2;
  if (P < 1 || 2 * P > d) return bad(fn, "s0 + s1 + s2 pairs must be at least one and fit d");
  if (T_in < 0 || T_out < 0 || (T_in && N % T_in) || (T_out && N % T_out))
    return bad(fn, "N must be a multiple of T_in and of T_out");
  if (T_in == 0 && (ldq < (long long)H * d || (k && ldk < (long long)Hk * d)))
    return bad(fn, "token strides must cover a token's heads");
  if (!std::isfinite(scale_q) || !std::isfinite(scale_k)) return bad(fn, "scales must be finite");
  if (N == 0) return LA_OK;
  if (!q || !q_out || !pos || !freq) return bad(fn, "q, q_out, pos and freq are required");
  const size_t el = (flags & LA_F32) ? 4 : 2;
  if (!at(q, el) || !at(k, el) || !at(q_out, el) || !at(k_out, el) || !at(pos, 4) || !at(freq, 8))
    return bad(fn, "pointers must be aligned to their elements");
  // in place only where a row is written where it was read
  const bool same_q = T_in == T_out && (T_in || ldq == (long long)H * d);
  const bool same_k = T_in == T_out && (T_in || ldk == (long long)Hk * d);
  if ((q == q_out && !same_q) || (k && k == k_out && !same_k))
    return bad(fn, "an output may be its input only with the same layout and strides");
  if (same({q_out, k_out}, {}) || (k && (q_out == k || k_out == q)))
    return bad(fn, "q_out and k_out are two tensors, and not each other's input");
  RotaryParams p = {q, k, q_out, k_out, pos, freq, n_axes, s0, s1, s2, N, H, k ? Hk : 0, d, T_in, T_out,
                    ldq, k ? ldk : 0, scale_q, scale_k, (flags & LA_ROT_INTERLEAVED) ? 1 : 0,
                    (flags & LA_ROT_INVERSE) ? 1 : 0, (flags & LA_F32) ? 1 : 0};
  return launch_rotary(p, reinterpret_cast<cudaStream_t>(stream));
}

static int check_epilogue(const char *fn, const EpilogueParams &p, int flags) {
  if (flags & ~LA_F32) return bad(fn, "unknown flag");
  if (p.N < 0 || p.G < 1 || (long long)p.N * p.G > INT_MAX / 2) return bad(fn, "N must be >= 0, G >= 1, N*G below 2^30");
  if (p.d < 1 || p.d > 16384) {
    set_error("%s: d must be 1..16384 (got %d)", fn, p.d);
    return LA_ERR_UNSUPPORTED;
  }
  if (p.T < 0 || (p.T && p.N % p.T)) return bad(fn, "N must be a multiple of T");
  if (!(p.eps > 0.f) || !std::isfinite(p.eps)) return bad(fn, "eps must be finite and > 0");
  if (p.gate && p.act != LA_ACT_SILU && p.act != LA_ACT_SIGMOID) return bad(fn, "unknown act");
  const size_t el = (flags & LA_F32) ? 4 : 2;
  const void *t[] = {p.x, p.gate, p.res, p.d_out, p.d_next, p.out, p.next, p.dx, p.dgate, p.dres};
  const void *f[] = {p.w, p.scale, p.w_next, p.dw, p.dscale, p.dw_next};
  for (const void *q : t)
    if (!at(q, el)) return bad(fn, "pointers must be aligned to their elements");
  for (const void *q : f)
    if (!at(q, 4)) return bad(fn, "pointers must be aligned to their elements");
  return LA_OK;
}

int la_epilogue(const void *x, const float *w, const void *gate, int act, const void *res, const float *scale,
                const float *w_next, void *out, void *next, float eps, int N, int G, int d, int T, int flags,
                la_stream_t stream) {
  NvtxRange nvtx_range("la_epilogue");
  const char *fn = "la_epilogue";
  set_error("%s", "");
  EpilogueParams p = {};
  p.x = x; p.w = w; p.gate = gate; p.res = res; p.scale = scale; p.w_next = w_next; p.out = out; p.next = next;
  p.eps = eps; p.N = N; p.G = G; p.d = d; p.T = T; p.act = act; p.f32 = (flags & LA_F32) ? 1 : 0;
  const int rc = check_epilogue(fn, p, flags);
  if (rc) return rc;
  if (w_next && !next && N > 0) return bad(fn, "w_next goes with next");
  if (N == 0) return LA_OK;
  if (!x || !out) return bad(fn, "x and out are required");
  if (out == next || (T && (out == x || next == x))) return bad(fn, "out and next are two tensors, and not a head-major x");
  return launch_epilogue(p, reinterpret_cast<cudaStream_t>(stream));
}

int la_epilogue_bwd(const void *x, const float *w, const void *gate, int act, const void *res,
                    const float *scale, const float *w_next, const void *d_out, const void *d_next, void *dx,
                    void *dgate, void *dres, float *dw, float *dscale, float *dw_next, float eps, int N, int G,
                    int d, int T, int flags, la_stream_t stream) {
  NvtxRange nvtx_range("la_epilogue_bwd");
  const char *fn = "la_epilogue_bwd";
  set_error("%s", "");
  EpilogueParams p = {};
  p.x = x; p.w = w; p.gate = gate; p.res = res; p.scale = scale; p.w_next = w_next;
  p.d_out = d_out; p.d_next = d_next; p.dx = dx; p.dgate = dgate; p.dres = dres;
  p.dw = dw; p.dscale = dscale; p.dw_next = dw_next;
  p.eps = eps; p.N = N; p.G = G; p.d = d; p.T = T; p.act = act; p.f32 = (flags & LA_F32) ? 1 : 0;
  const int rc = check_epilogue(fn, p, flags);
  if (rc) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0) {  // no tokens: the sums over them are zero
    for (float *t : {dw, dscale, dw_next})
      if (t && cudaMemsetAsync(t, 0, (size_t)d * 4, s) != cudaSuccess) {
        set_error("%s: clearing the sums failed: %s", fn, cudaGetErrorString(cudaGetLastError()));
        return LA_ERR_CUDA;
      }
    return LA_OK;
  }
  if (!x || (!d_out && !d_next)) return bad(fn, "x and one of d_out and d_next are required");
  if (dgate && !gate) return bad(fn, "dgate needs gate");
  if ((dw_next || w_next) && !d_next) return bad(fn, "w_next and dw_next need d_next");
  if (same({dx, dgate, dres}, {x, gate, res, d_next}) || same({dx, dgate}, {d_out}) ||
      same({dw, dscale, dw_next}, {w, scale, w_next}))
    return bad(fn, "outputs must not be inputs, nor one another; dres may be d_out");
  return launch_epilogue_bwd(p, s);
}

}  // extern "C"
