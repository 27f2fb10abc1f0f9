/*
 * la_serve.h -- decoding with paged caches and beams, in libla.so next to
 * la.h and la_layer.h: what a stack of linear-attention layers with a few
 * softmax-attention layers between them needs to answer requests. Appending
 * to a paged key-value cache with the position rotation on the way
 * (la_cache_append), attention of one new token over it (la_paged_attn), beam
 * search's selection (la_beam_select), and the reordering of states and pages
 * that follows it (la_beam_states, la_beam_cache).
 *
 * Status codes, LA_F32 and la_stream_t are la.h's, LA_ROT_INTERLEAVED is
 * la_layer.h's; so are the conventions: device pointers owned by the caller,
 * calls asynchronous on `stream`, float32 accumulation, argument errors found
 * on the host before anything is launched, messages from la_last_error().
 *
 * The cache. k_cache and v_cache are pools of n_pages pages,
 * [n_pages][page_size][Hk][d], a page dense and pages ld_page elements apart
 * (ld_page >= page_size*Hk*d: a layer's or the keys' part of a pool that
 * interleaves several is used where it is). Place p of sequence s is row
 * p % page_size of page table[s*ld_table + p / page_size], p / page_size <
 * max_pages. lens int32 [n]: the places of each sequence that are in use. All
 * of table and lens may hold any values: a place without a page (behind the
 * table, or its page outside [0, n_pages)) is not there, for reading and for
 * writing. Page offsets are 64-bit.
 */
#ifndef LA_SERVE_H
#define LA_SERVE_H

#include "la_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * la_cache_append -- new tokens into the cache: token i of the m new ones of
 * sequence s goes to place p = lens[s] - m + i (lens counts them already: it is
 * what la_paged_attn reads), its key turned like la_rotary's, its value as it
 * is; and the queries, turned, to q_out.
 *
 *   q       [total][H][d] or NULL (then q_out is NULL), k, v [total][Hk][d],
 *           token-major, token strides ldq, ldk, ldv
 *   q_out   [total][H][d], dense; may be q if that is dense
 *   cu_seqlens  int32 [n_seq + 1], device, as la_packed_fwd's: the new tokens of
 *           sequence s are cu_seqlens[s] .. cu_seqlens[s+1] - 1 (none: nothing
 *           happens to it); rows of tokens in no sequence are not written.
 *           NULL: one token for each sequence; then total = n_seq.
 *   table, lens, k_cache, v_cache  as above; a token whose place is negative or
 *           has no page is not written to the cache. Two tokens with one place
 *           in the same page: either may be kept.
 *   n_axes, s0, s1, s2, freq  as la_rotary's, freq float64 [P]; n_axes = 0: no
 *           rotation (freq NULL, s0 = s1 = s2 = 0)
 *   pos     int32 [total][n_axes], or NULL: the place p is the position
 *           (n_axes = 1)
 *   flags   LA_F32 (float32 q, k, v, caches; else bfloat16) | LA_ROT_INTERLEAVED
 *
 * 1 <= d <= 512; H, Hk <= 65535; page_size >= 1; n_seq, total >= 0. Tensors need the alignment
 * of their elements; 16-byte aligned ones with rows of multiples of 16 bytes
 * are moved 16 bytes at a time.
 */
int la_cache_append(const void *q, const void *k, const void *v, void *q_out, void *k_cache, void *v_cache,
                    const int *table, const int *lens, const int *cu_seqlens, const int *pos, const double *freq,
                    int n_axes, int s0, int s1, int s2, int n_seq, int total, int H, int Hk, int d, int page_size,
                    int n_pages, int max_pages, long long ld_table, long long ldq, long long ldk, long long ldv,
                    long long ld_page, int flags, la_stream_t stream);

/*
 * la_paged_attn -- attention of one new token of each of n sequences over the
 * cache: for query head h, with key/value head h / (H / Hk),
 *
 *     o_h = sum_p softmax_p(scale q_h . k_p) v_p
 *
 * over the places p of max(0, L - window) .. L - 1, L = lens[s] (at most
 * max_pages*page_size, and 2^31 - 2^16; window = 0: all of them), without those that have no
 * page. A sequence with no place (L <= 0) gives o = 0, and lse = -infinity.
 *
 *   q       [n][H][d], token stride ldq
 *   o       [n][H][d], dense
 *   lse     float32 [n][H], log sum_p exp(scale q_h . k_p), or NULL
 *   H a multiple of Hk; d 64, 128 or 256; scale finite
 *   max_len an upper bound of lens, 0: unknown. Only the split of the work
 *           goes by it, never the result's meaning.
 *   flags   LA_F32 (float32 q, o, caches) or 0 (bfloat16)
 *   q, o, k_cache, v_cache 16-byte aligned; ldq, ld_page multiples of 16 bytes
 *
 * n*Hk*ceil(H/Hk / R)*max_pages*page_size is below 2^36 with R = 16 in
 * bfloat16, below 2^35 with R = 8 in float32 (2^34 with d = 256); of
 * max_pages*page_size, 2^31 - 2^16 at most count. Larger tables may be refused.
 * Workspace from the library's pool where the length may be split: up to about
 * 6 MB. What the cache holds behind a sequence's length, or in front of its
 * window, is not used, whatever it is; inside it, inputs are finite.
 */
int la_paged_attn(const void *q, const void *k_cache, const void *v_cache, void *o, float *lse, const int *table,
                  const int *lens, int n, int H, int Hk, int d, int page_size, int n_pages, int max_pages,
                  long long ld_table, int max_len, int window, float scale, long long ldq, long long ld_page,
                  int flags, la_stream_t stream);

/*
 * la_beam_select -- beam search's step: of the W beams of each of B requests,
 * with scores (sums of log probabilities so far) and the logits of their next
 * token, the K best continuations, best first:
 *
 *     c(w, v) = scores[w] + logits[w][v] - log sum_u exp logits[w][u]
 *
 *   logits  [B*W][V], row stride ld, bfloat16 or float32 (LA_F32); -infinity: a
 *           token that is not allowed
 *   scores  float32 [B][W]
 *   done    uint8 [B][W] or NULL: a beam that has ended (non-zero) has the one
 *           continuation eos, at scores[w]; its logits are not read
 *   scores_out float32 [B][K], parent int32 [B][K] (the beam, 0..W-1), token
 *           int32 [B][K]: outputs, not the inputs
 *   1 <= W <= 32, 1 <= K <= 32, K <= W*V, W*V < 2^31 - 2^16, 0 <= eos < V (with done)
 *
 * Equal candidates are taken in the order of w*V + v. Candidates without a
 * value (a token not allowed, a beam with no token allowed, whose score is not
 * finite, or with a NaN or +infinity among its logits; NaN) count as -infinity and
 * are taken, in that order, where there are fewer than K others. Candidates are
 * compared in 64 bits, behind sums whose terms are float32: each is off by up to
 * 2^-22 and, at a distance a below the row's largest logit, by a 2^-23. Where
 * these do not average out (many equal logits) the log of the sum may be off by
 * 3e-6, by 6e-6 at V = 2^18; measured it is 1e-7 mostly, and below 3e-7.
 * Two beams' candidates closer than twice that may change places; those of
 * beams with the same logits do not, nor do those of one beam.
 * Workspace from the library's pool: 8*K + 16 bytes for each 256 logits of a row
 * at most.
 */
int la_beam_select(const void *logits, const float *scores, const unsigned char *done, float *scores_out, int *parent,
                   int *token, int B, int W, int V, int K, long long ld, int eos, int flags, la_stream_t stream);

/*
 * la_beam_states -- the states of the chosen beams: for every layer and request,
 * row slots[b*W + w] of the pool becomes what row slots[b*W + parent[b][w]] was,
 * for all w at once, in place.
 *
 *   pool    layers x n_slots rows of row_bytes bytes: row r of layer l at byte
 *           l*ld_layer + r*ld_row; any type (la_packed_step's states are
 *           H*dk*dv*4 bytes). Rows do not overlap.
 *   parent  int32 [B][W]; outside [0, W): the row stays as it is
 *   slots   int32 [B*W], device, or NULL (row b*W + w). Outside [0, n_slots):
 *           neither read nor written (nor is a row written whose parent has
 *           such a slot). Slots of different beams are different rows.
 *   1 <= W <= 32; row_bytes, ld_row, ld_layer multiples of 4 and pool 4-byte
 *   aligned (16 moves faster)
 */
int la_beam_states(void *pool, const int *slots, const int *parent, int B, int W, int n_slots, int layers,
                   long long row_bytes, long long ld_row, long long ld_layer, la_stream_t stream);

/*
 * la_beam_cache -- the same for a paged cache. Every beam has pages of its own
 * in its row of the table up to the one that its next token goes to. Pages that
 * are full are shared from then on: beam w's entries in front of its open page
 * become its parent's. The tokens in the open page are copied from the parent's
 * open page into beam w's own, for all w at once. Pages are thus never written
 * once full, and a beam's own page of a place is never another's open page:
 * no counts of references are needed.
 *
 *   k_cache, v_cache  layers x n_pages pages of page_size tokens of token_bytes
 *           bytes: page i of layer l at byte l*ld_layer + i*ld_page of both;
 *           layers = 0: the table alone changes, the caches are not used
 *   table   int32 [B*W][max_pages], row stride ld_table: the same for all
 *           layers; changed in place
 *   lens    int32 [B*W]: the tokens in the cache; the beams of a request have
 *           one length, the first one's counts
 *   parent  as la_beam_states'. With every parent 0 the call forks a request's
 *           prompt into W beams.
 *   1 <= W <= 32; token_bytes, ld_page, ld_layer multiples of 4, caches 4-byte
 *   aligned (16 moves faster)
 */
int la_beam_cache(void *k_cache, void *v_cache, int *table, const int *lens, const int *parent, int B, int W,
                  int page_size, int n_pages, int max_pages, long long ld_table, int layers, long long token_bytes,
                  long long ld_page, long long ld_layer, la_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* LA_SERVE_H */
