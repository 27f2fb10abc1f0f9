// Internal declarations of the layer operators (include/la_layer.h): packed
// retention, block epilogue, rotary positions.
#pragma once

#include "../../include/la_layer.h"
#include "la_internal.h"

namespace la {

// n / d and n % d of 0 <= n < 2^31 by a multiplication, the division by an invariant
// of Granlund and Montgomery (1994): with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (mulhi(m, n) + n) >> s (the sum
// stays below 2^32 for n below 2^31).
struct FastDiv {
  uint32_t d, m, s;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div), s(0) {
    while ((1ull << s) < d) ++s;
    m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
  __device__ __forceinline__ void split(uint32_t n, uint32_t &q, uint32_t &r) const {
    q = (__umulhi(m, n) + n) >> s;
    r = n - q * d;
  }
};

// One pass of packed retention. All four products of the forward and backward
// are the same sum with other tensors in its three places:
//
//   out_i = sum_j gamma^|i-j| (x_i . y_j) z_j  (+ the entering state's part),
//
// over j <= i, or over j >= i with `reverse`, within a sequence:
//
//   o : x = q,  y = k,  z = v       dq: x = dO, y = v,  z = k
//   dk: x = v,  y = dO, z = q       dv: x = k,  y = q,  z = dO   (both reversed)
//
// with a state of da x db (da channels of x and y, db of z and out):
//   causal    S <- gamma S + y z^T, out = S^T x
//   reversed  G  = W + y z^T, out = G^T x, W <- gamma G
// so that W enters as dS_final and leaves as dS0.
struct PackedPass {
  const void *x, *y, *z;
  void *out;
  long long ldx, ldy, ldz, ldo;  // token strides in elements
  int rx, ry, rz;                // heads of the pass that share a head of x, y, z
  int da, db;
  const float *S_in;             // [slot][H][dk][dv], or null
  float *S_out;                  // likewise
  int in_t;                      // S_in is stored [db][da] (transposed for this pass)
  int sized;                     // da * db
  const int *cu, *slots;
  int n_seq, total, n_slots, H;
  const float *g;
  int reverse;
  int f32;                       // x, y, z are float32, else bfloat16
  int out_f32;                   // out is float32 (always with f32)
  unsigned *status;
  int max_len;
};

// The tokens of sequence s, clamped into [0, total].
__device__ __forceinline__ void packed_range(const int *cu, int s, int total, int *a, int *b) {
  const int lo = min(max(__ldg(cu + s), 0), total);
  *a = lo;
  *b = min(max(__ldg(cu + s + 1), lo), total);
}

// The state row of sequence s, or -1: without one, outside the pool, or taken
// by an earlier sequence. Called by all threads of the block.
__device__ __forceinline__ int packed_slot(const int *slots, int s, int n_slots) {
  const int slot = slots ? __ldg(slots + s) : s;
  if (slot < 0 || slot >= n_slots) return -1;
  if (!slots) return slot;
  int taken = 0;
  for (int j = threadIdx.x; j < s; j += blockDim.x) taken |= __ldg(slots + j) == slot;
  return __syncthreads_or(taken) ? -1 : slot;
}

// gamma^n of a natural-log decay, n >= 0 (gamma = 0: 1 at n = 0)
__device__ __forceinline__ float decay_power(float g, int n) { return n ? expf(g * static_cast<float>(n)) : 1.f; }


// S <- gamma^n S in float32 for decays near one: a rounded gamma^n would be off
// by up to 2^-25 at every application, always the same way, which a memory of
// thousands of tokens adds up; gamma^n - 1 carries its own 24 bits. Below one
// half the plain product is the more exact one.
struct Decay {
  float m;
  bool near;
  __device__ __forceinline__ Decay() {}
  __device__ __forceinline__ Decay(float g, int n) {
    const float e = n ? g * static_cast<float>(n) : 0.f;
    near = e > -0.6931472f;
    m = near ? expm1f(e) : expf(e);
  }
  __device__ __forceinline__ float operator()(float S) const { return fmaf(S, m, near ? S : 0.f); }
};

// float32 passes, or passes without a token
int launch_packed_walk(const PackedPass &p, cudaStream_t stream);
// Up to three passes that do not depend on each other.
int launch_packed_tc(const PackedPass *p, int passes, cudaStream_t stream);
// dst[i][n][hk][d] = sum over the `share` heads of src[i] float32 [n][hk * share][d], for both i
// and the tokens n of the sequences
int launch_head_sums(const float *const src[2], void *const dst[2], int f32, const int *cu, int n_seq, int total,
                     int Hk, int share, int d, cudaStream_t stream);

struct PackedStep {
  const void *q, *k, *v;
  void *o;
  float *S;
  const float *g;
  const int *slots;
  int n, n_slots, H, Hk, dk, dv, f32;
  long long ldq, ldk, ldv;
};
int launch_packed_step(const PackedStep &p, cudaStream_t stream);

struct RotaryParams {
  const void *q, *k;
  void *q_out, *k_out;
  const int *pos;
  const double *freq;
  int n_axes, s0, s1, s2;
  int N, H, Hk, d, T_in, T_out;
  long long ldq, ldk;
  float scale_q, scale_k;
  int interleaved, inverse, f32;
};
int launch_rotary(const RotaryParams &p, cudaStream_t stream);

struct EpilogueParams {
  const void *x, *gate, *res, *d_out, *d_next;
  const float *w, *scale, *w_next;
  void *out, *next;               // forward
  void *dx, *dgate, *dres;        // backward
  float *dw, *dscale, *dw_next;
  float eps;
  int N, G, d, T, act, f32;
};
int launch_epilogue(const EpilogueParams &p, cudaStream_t stream);
int launch_epilogue_bwd(const EpilogueParams &p, cudaStream_t stream);

}  // namespace la
