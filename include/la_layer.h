/*
 * la_layer.h -- the operators around the mixer of a retention layer, in
 * libla.so next to la.h: rotary positions in front of it (la_rotary), the
 * mixer itself over packed sequences (la_packed_fwd, la_packed_bwd,
 * la_packed_step) and the end of the block behind it (la_epilogue,
 * la_epilogue_bwd).
 *
 * Status codes, modes, LA_F32 and la_stream_t are la.h's; so are the
 * conventions: device pointers owned by the caller, calls asynchronous on
 * `stream`, float32 accumulation, natural-log decays, argument errors found on
 * the host before anything is launched, messages from la_last_error().
 *
 * Layouts. "Token-major" tensors are [N][heads][d], d fastest and the heads of
 * a token side by side; an input's token stride (ld*, in elements) may exceed
 * heads*d, so that a slice of a fused projection is read where it is.
 * "Head-major" tensors are la.h's dense [B][heads][T][d], with token n of the
 * N = B*T being (b, t) = (n / T, n % T).
 */
#ifndef LA_LAYER_H
#define LA_LAYER_H

#include "la.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * la_packed_fwd -- causal retention over sequences packed back to back: for
 * every sequence s, head h and token t of it,
 *
 *     S_t = gamma_h S_{t-1} + k_t v_t^T ,   o_t = S_t^T q_t
 *
 * (la_chunk_fwd's LA_RETNET and LA_LINEAR recurrence; "Talk Linear Attention"
 * sections 2.1 and 3.2), S_{-1} from S0 or zero.
 *
 *   q, k    [total][Hk][dk] token-major, token strides ldq, ldk
 *   v       [total][H][dv] token-major, token stride ldv; value head h uses
 *           query/key head h / (H / Hk) (H a multiple of Hk)
 *   g       float32 [H], log gamma_h (LA_RETNET), or NULL (LA_LINEAR)
 *   o       [total][H][dv], dense, overlaps no input; rows of tokens in no
 *           sequence are not written
 *   cu_seqlens  int32 [n_seq + 1], device: sequence s is the tokens
 *           cu_seqlens[s] .. cu_seqlens[s+1] - 1; non-decreasing within
 *           [0, total] (values outside are clamped, and a bound below the one
 *           before it ends an empty sequence: memory-safe, not an error).
 *           Sequences may be empty; the unused end of a padded batch may
 *           repeat the last bound or hold zeros.
 *   S0, S_final  float32 [n_slots][H][dk][dv] or NULL (zero / not written);
 *           S_final may be S0. An empty sequence's S_final is its S0.
 *   slots   int32 [n_seq], device: sequence s starts from S0[slots[s]] and
 *           leaves S_final[slots[s]]; NULL: row s. A slot outside
 *           [0, n_slots) means a zero start and no final state; so does a slot
 *           that an earlier sequence of the call has. Rows of no sequence are
 *           left as they are.
 *   max_len an upper bound of the lengths, 0: unknown. Only the split of the
 *           work goes by it, never the result's meaning.
 *   n_seq >= 1; total >= 0; dk, dv in {64, 128}; ld* >= heads*d, multiples of
 *           16 bytes; q, k, v, o, S0, S_final 16-byte aligned.
 *   mode    LA_LINEAR or LA_RETNET, bfloat16 q, k, v, o, or float32 with
 *           | LA_F32. Other modes of la.h: LA_ERR_UNSUPPORTED.
 *
 * bfloat16 runs chunkwise on the tensor cores, float32 token by token on the
 * CUDA cores in float32 throughout. In bfloat16 the state and all sums are
 * float32, and three operands of the products are not: the decayed values
 * gamma^n v that go into the state are two bfloat16 parts, good to 2^-16 of
 * each (S_final measured at 1.6e-6 relative, where float32 operands give about
 * 3e-7); the decayed scores inside a chunk of 128 tokens and the copy of the
 * state that o reads are rounded to bfloat16 once (o measured at 1.4 times the
 * error of its own rounding). A state that is carried from call to call is not
 * rounded on the way.
 *
 * Workspace from the library's pool where the heads and sequences
 * are more than the SMs or a sequence may be long (max_len unknown: as long as
 * total): 16 bytes a sequence, 4*n_slots with slots, and for the segments of
 * split sequences, however many sequences there are, up to 512*SMs*dk bytes
 * (dv if that is more; about 10 MB).
 *
 * Inputs are finite: a NaN or infinity at a token may reach every token of the
 * same sequence; never another sequence, whatever the neighbours hold.
 */
int la_packed_fwd(const void *q, const void *k, const void *v, const float *g, void *o, const float *S0,
                  float *S_final, const int *cu_seqlens, const int *slots, int n_seq, int total, int max_len,
                  int n_slots, int H, int Hk, int dk, int dv, long long ldq, long long ldk, long long ldv,
                  int mode, la_stream_t stream);

/*
 * la_packed_bwd -- the backward pass of la_packed_fwd: given dO = dL/do and
 * dS_final = dL/dS_final, per sequence of T tokens
 *
 *   dq_t = sum_{s<=t} gamma^(t-s) (dO_t . v_s) k_s + gamma^(t+1) S0 dO_t
 *   dk_s = sum_{t>=s} gamma^(t-s) (dO_t . v_s) q_t + gamma^(T-1-s) dS_final v_s
 *   dv_s = sum_{t>=s} gamma^(t-s) (q_t . k_s) dO_t + gamma^(T-1-s) dS_final^T k_s
 *   dS0  = sum_t gamma^(t+1) q_t dO_t^T + gamma^T dS_final
 *
 * with dq, dk summed over the value heads that share a query/key head.
 *
 *   q, k, v, g, cu_seqlens, max_len, ld*, mode  as la_packed_fwd
 *   dO      [total][H][dv], dense
 *   S0, dS_final  float32 [n_seq][H][dk][dv] or NULL (zero)
 *   dq, dk_out [total][Hk][dk]; dv_out [total][H][dv]: outputs, dense, input
 *           dtype; rows of tokens in no sequence are not written
 *   dS0     float32 [n_seq][H][dk][dv] or NULL (not computed)
 *   Outputs overlap no input and not each other. 16-byte alignment for every tensor.
 * Runs as three passes of la_packed_fwd's kernel with the tensors' places
 * exchanged (dk, dv: from the last token to the first), each with that
 * function's workspace, and with shared heads another 8*total*H*dk bytes. In
 * bfloat16 dq, dk and dv have o's accuracy there, dS0 that of S_final.
 */
int la_packed_bwd(const void *q, const void *k, const void *v, const float *g, const void *dO,
                  const float *S0, const float *dS_final, void *dq, void *dk_out, void *dv_out, float *dS0,
                  const int *cu_seqlens, int n_seq, int total, int max_len, int H, int Hk, int dk, int dv,
                  long long ldq, long long ldk, long long ldv, int mode, la_stream_t stream);

/*
 * la_packed_step -- one token for each of n requests on a pool of states:
 * row i takes S = S[slots[i]] through one step of the recurrence above, in
 * place, and o_i = S^T q_i.
 *
 *   q, k    [n][Hk][dk], v [n][H][dv] token-major (strides ldq, ldk, ldv);
 *   o       [n][H][dv] dense, overlaps no input
 *   S       float32 [n_slots][H][dk][dv], 16-byte aligned
 *   slots   int32 [n], device, or NULL (row i; then n <= n_slots). A slot
 *           outside [0, n_slots) is a padding row: o_i = 0, no state is
 *           touched. Rows with the same slot are applied in their order.
 *   dk, dv in {64, 128}; mode as la_packed_fwd; other alignments as there.
 */
int la_packed_step(const void *q, const void *k, const void *v, const float *g, void *o, float *S,
                   const int *slots, int n, int n_slots, int H, int Hk, int dk, int dv, long long ldq,
                   long long ldk, long long ldv, int mode, la_stream_t stream);

/*
 * la_rotary -- rotary positions with one to three axes on queries and keys:
 * the first 2*P channels of every row, P = s0 + s1 + s2, are P pairs; pair p
 * turns by the angle pos[n][axis(p)] * freq[p], the first s0 pairs with axis 0,
 * the next s1 with axis 1, the last s2 with axis 2:
 *
 *     (a, b) -> (a cos - b sin, b cos + a sin)
 *
 * and the whole row is multiplied by scale_q (scale_k). The other channels are
 * only scaled. LA_ROT_INVERSE turns by the negated angle: the backward pass.
 *
 *   q, q_out  N rows of H heads; k, k_out N rows of Hk heads, or both NULL
 *           T_in = 0: token-major inputs (token strides ldq, ldk);
 *           T_in > 0: head-major inputs [N/T_in][heads][T_in][d] (ld* ignored)
 *           T_out likewise for the dense outputs; N a multiple of T_in, T_out.
 *           An output may be its own input if both have the same layout and
 *           strides; outputs do not overlap otherwise.
 *   pos     int32 [N][n_axes], device; any int32 value
 *   freq    float64 [P], device: radians per position. Angles are formed in
 *           64-bit fixed point, so far positions keep float32 accuracy.
 *   n_axes  1..3; s_a >= 0 with s_a = 0 for a >= n_axes; 1 <= P, 2*P <= d <= 512
 *   flags   LA_F32 | LA_ROT_INTERLEAVED | LA_ROT_INVERSE. Pair p is the channels
 *           (2p, 2p+1) if interleaved, else (p, p + P).
 */
#define LA_ROT_INTERLEAVED 0x1
#define LA_ROT_INVERSE     0x2
int la_rotary(const void *q, const void *k, void *q_out, void *k_out, const int *pos, const double *freq,
              int n_axes, int s0, int s1, int s2, int N, int H, int Hk, int d, int T_in, int T_out,
              long long ldq, long long ldk, float scale_q, float scale_k, int flags, la_stream_t stream);

/*
 * la_epilogue -- the end of a block in one pass: norm, gate, residual scale,
 * residual and the next block's norm. For every token and each of its G groups
 * of d channels (G = heads after the mixer, 1 on the residual stream):
 *
 *     y    = x / sqrt(mean(x^2) + eps) * w
 *     out  = res + scale * y * act(gate)
 *     next = out / sqrt(mean(out^2) + eps) * w_next
 *
 *   x       token-major [N][G][d] (T = 0) or head-major [N/T][G][T][d] (T > 0,
 *           N a multiple of T: la_chunk_fwd's o); dense
 *   gate, res, out, next  [N][G][d] dense; gate NULL: no gate; res NULL: zero;
 *           next NULL: not computed. out may be x (T = 0), gate or res; next
 *           may be x (T = 0), gate or res too, but not out.
 *   w, scale, w_next  float32 [d], or NULL: ones. w_next only with next.
 *   act     LA_ACT_SILU or LA_ACT_SIGMOID (ignored without gate)
 *   eps > 0, finite; N >= 0; G >= 1; 1 <= d <= 16384
 *   flags   0 (bfloat16) or LA_F32
 *
 * next is formed from the float32 out, before its rounding. Tensors need the
 * alignment of their elements; 16-byte aligned ones with d a multiple of 16
 * bytes are read and written 16 bytes at a time.
 */
#define LA_ACT_SILU    0
#define LA_ACT_SIGMOID 1
int la_epilogue(const void *x, const float *w, const void *gate, int act, const void *res, const float *scale,
                const float *w_next, void *out, void *next, float eps, int N, int G, int d, int T, int flags,
                la_stream_t stream);

/*
 * la_epilogue_bwd -- the backward pass of la_epilogue from its inputs (nothing
 * is kept by the forward): given d_out and d_next (either may be NULL: zero,
 * not both), the gradients
 *
 *   dx (x's layout), dgate, dres [N][G][d] in the input dtype;
 *   dw, dscale, dw_next float32 [d], summed over all tokens and groups
 *
 * each NULL: not computed. dgate needs gate; dw_next needs d_next. res is needed with
 * d_next if the forward had it, and not read without d_next. Sums over tokens
 * run in a fixed order: the results do not change from run to run. Outputs may
 * not overlap inputs, except dres = d_out. Uses workspace from the library's pool
 * (up to 8*SMs*d*4 bytes) for dw, dscale and dw_next. Other arguments as la_epilogue.
 */
int la_epilogue_bwd(const void *x, const float *w, const void *gate, int act, const void *res,
                    const float *scale, const float *w_next, const void *d_out, const void *d_next, void *dx,
                    void *dgate, void *dres, float *dw, float *dscale, float *dw_next, float eps, int N, int G,
                    int d, int T, int flags, la_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* LA_LAYER_H */
