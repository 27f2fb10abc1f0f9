// Host side of include/la_serve.h: argument checks.
#include <climits>
#include <cmath>

#include "la_check.h"
#include "la_serve_internal.h"

using namespace la;

namespace {

int unsupported(const char *fn, const char *what, int got) {
  set_error("%s: %s (got %d)", fn, what, got);
  return LA_ERR_UNSUPPORTED;
}

// Page table, lengths and page strides of a cache with `token` elements a token.
int check_cache(const char *fn, const PagedCache &c, long long token) {
  if (c.page_size < 1 || c.n_pages < 0 || c.max_pages < 0) return bad(fn, "page_size must be >= 1, n_pages and max_pages >= 0");
  if (c.ld_table < c.max_pages) return bad(fn, "ld_table must be >= max_pages");
  if (c.ld_page < c.page_size * token) return bad(fn, "ld_page must cover a page");
  if (!at(c.table, 4) || !at(c.lens, 4)) return bad(fn, "table and lens must be 4-byte aligned");
  return LA_OK;
}

}  // namespace

extern "C" {

int la_cache_append(const void *q, const void *k, const void *v, void *q_out, void *k_cache, void *v_cache,
                    const int *table, const int *lens, const int *cu_seqlens, const int *pos, const double *freq,
                    int n_axes, int s0, int s1, int s2, int n_seq, int total, int H, int Hk, int d, int page_size,
                    int n_pages, int max_pages, long long ld_table, long long ldq, long long ldk, long long ldv,
                    long long ld_page, int flags, la_stream_t stream) {
  NvtxRange nvtx_range("la_cache_append");
  const char *fn = "la_cache_append";
  set_error("%s", "");
  if (flags & ~(LA_F32 | LA_ROT_INTERLEAVED)) return bad(fn, "unknown flag");
  if ((q != nullptr) != (q_out != nullptr)) return bad(fn, "q and q_out go together");
  if (n_seq < 0 || total < 0 || (!cu_seqlens && n_seq != total))
    return bad(fn, "n_seq and total must be >= 0, and equal without cu_seqlens");
  if ((q && H < 1) || Hk < 1 || H > 65535 || Hk > 65535) return bad(fn, "H and Hk must be 1..65535");
  if (d < 1 || d > 512) return unsupported(fn, "d must be 1..512", d);
  if (n_axes < 0 || n_axes > 3 || s0 < 0 || s1 < 0 || s2 < 0 || (n_axes < 1 && s0) || (n_axes < 2 && s1) ||
      (n_axes < 3 && s2))
    return bad(fn, "n_axes must be 0..3, with s_a = 0 for the axes that are not there");
  const long long P = (long long)s0 + s1 + s2;
  if ((n_axes > 0 && P < 1) || 2 * P > d) return bad(fn, "s0 + s1 + s2 pairs must be at least one and fit d");
  if ((n_axes > 0) != (freq != nullptr)) return bad(fn, "freq goes with n_axes > 0, and only with it");
  if (pos ? n_axes == 0 : n_axes > 1) return bad(fn, "pos goes with n_axes > 0, and is required for more than one axis");
  const PagedCache c = {table, lens, ld_table, ld_page, page_size, n_pages, max_pages};
  const int rc = check_cache(fn, c, (long long)Hk * d);
  if (rc) return rc;
  if ((q && ldq < (long long)H * d) || ldk < (long long)Hk * d || ldv < (long long)Hk * d)
    return bad(fn, "token strides must cover a token's heads");
  if (total == 0 || n_seq == 0) return LA_OK;
  if (!k || !v || !lens) return bad(fn, "k, v and lens are required");
  if (max_pages > 0 && (!table || (n_pages > 0 && (!k_cache || !v_cache)))) return bad(fn, "table and caches are required");
  const size_t el = (flags & LA_F32) ? 4 : 2;
  const void *all[] = {q, k, v, q_out, k_cache, v_cache};
  for (const void *t : all)
    if (!at(t, el)) return bad(fn, "pointers must be aligned to their elements");
  if (!at(cu_seqlens, 4) || !at(pos, 4) || !at(freq, 8)) return bad(fn, "pointers must be aligned to their elements");
  if (same({q_out, k_cache, v_cache}, {k, v}) || same({k_cache, v_cache}, {q}))
    return bad(fn, "outputs must not be inputs, nor one another; q_out may be q");
  if (q && q == q_out && ldq != (long long)H * d) return bad(fn, "q_out may be q only if that is dense");
  const AppendParams p = {q, k, v, q_out, k_cache, v_cache, c, cu_seqlens, pos, freq, n_axes, s0, s1, s2, n_seq, total,
                          q ? H : 0, Hk, d, ldq, ldk, ldv, (flags & LA_ROT_INTERLEAVED) ? 1 : 0, (flags & LA_F32) ? 1 : 0};
  return launch_cache_append(p, reinterpret_cast<cudaStream_t>(stream));
}

int la_paged_attn(const void *q, const void *k_cache, const void *v_cache, void *o, float *lse, const int *table,
                  const int *lens, int n, int H, int Hk, int d, int page_size, int n_pages, int max_pages,
                  long long ld_table, int max_len, int window, float scale, long long ldq, long long ld_page,
                  int flags, la_stream_t stream) {
  NvtxRange nvtx_range("la_paged_attn");
  const char *fn = "la_paged_attn";
  set_error("%s", "");
  if (flags & ~LA_F32) return bad(fn, "unknown flag");
  if (n < 0 || max_len < 0 || window < 0) return bad(fn, "n, max_len and window must be >= 0");
  if (H < 1 || Hk < 1 || H % Hk != 0 || H > 65535) return bad(fn, "H must be a multiple of Hk, 1 <= H <= 65535");
  if (d != 64 && d != 128 && d != 256) return unsupported(fn, "d must be 64, 128 or 256", d);
  if (!std::isfinite(scale)) return bad(fn, "scale must be finite");
  const PagedCache c = {table, lens, ld_table, ld_page, page_size, n_pages, max_pages};
  const int rc = check_cache(fn, c, (long long)Hk * d);
  if (rc) return rc;
  const int unit = (flags & LA_F32) ? 4 : 8;
  if (ldq < (long long)H * d || ldq % unit || ld_page % unit)
    return bad(fn, "ldq must cover a token's heads, ldq and ld_page be multiples of 16 bytes");
  if ((long long)n * H > INT_MAX / 2) return bad(fn, "n*H too large");
  if (n == 0) return LA_OK;
  if (!q || !o || !lens) return bad(fn, "q, o and lens are required");
  if (max_pages > 0 && (!table || (n_pages > 0 && (!k_cache || !v_cache)))) return bad(fn, "table and caches are required");
  if (!at(q, 16) || !at(o, 16) || !at(k_cache, 16) || !at(v_cache, 16) || !at(lse, 4))
    return bad(fn, "tensors must be 16-byte aligned, lse 4-byte aligned");
  if (same({o, lse}, {q, k_cache, v_cache})) return bad(fn, "outputs must not be inputs, nor one another");
  const PagedAttn p = {q, k_cache, v_cache, o, lse, c, n, H, Hk, d, max_len, window, scale, ldq, (flags & LA_F32) ? 1 : 0};
  return launch_paged_attn(p, reinterpret_cast<cudaStream_t>(stream));
}

int la_beam_select(const void *logits, const float *scores, const unsigned char *done, float *scores_out, int *parent,
                   int *token, int B, int W, int V, int K, long long ld, int eos, int flags, la_stream_t stream) {
  NvtxRange nvtx_range("la_beam_select");
  const char *fn = "la_beam_select";
  set_error("%s", "");
  if (flags & ~LA_F32) return bad(fn, "unknown flag");
  if (B < 0 || V < 1) return bad(fn, "B must be >= 0, V >= 1");
  if (W < 1 || W > kMaxBeams) return unsupported(fn, "W must be 1..32", W);
  if (K < 1 || K > kMaxBeams) return unsupported(fn, "K must be 1..32", K);
  if ((long long)W * V > INT_MAX - 65535 || K > W * V) return bad(fn, "K must be <= W*V, W*V below 2^31 - 2^16");
  if (((long long)V / 128 + 1) * W * B > INT_MAX / 2) return bad(fn, "B*W*V too large");
  if (ld < V) return bad(fn, "ld must be >= V");
  if (done && (eos < 0 || eos >= V)) return bad(fn, "eos must be in 0..V-1");
  if (B == 0) return LA_OK;
  if (!logits || !scores || !scores_out || !parent || !token)
    return bad(fn, "logits, scores, scores_out, parent and token are required");
  if (!at(logits, (flags & LA_F32) ? 4 : 2) || !at(scores, 4) || !at(scores_out, 4) || !at(parent, 4) || !at(token, 4))
    return bad(fn, "pointers must be aligned to their elements");
  if (same({scores_out, parent, token}, {logits, scores, done}))
    return bad(fn, "outputs must not be inputs, nor one another");
  const BeamSelect p = {logits, scores, done, scores_out, parent, token, B, W, V, K, eos, (flags & LA_F32) ? 1 : 0, ld};
  return launch_beam_select(p, reinterpret_cast<cudaStream_t>(stream));
}

int la_beam_states(void *pool, const int *slots, const int *parent, int B, int W, int n_slots, int layers,
                   long long row_bytes, long long ld_row, long long ld_layer, la_stream_t stream) {
  NvtxRange nvtx_range("la_beam_states");
  const char *fn = "la_beam_states";
  set_error("%s", "");
  if (B < 0 || layers < 0 || n_slots < 0 || row_bytes < 0) return bad(fn, "B, layers, n_slots and row_bytes must be >= 0");
  if (W < 1 || W > kMaxBeams) return unsupported(fn, "W must be 1..32", W);
  if (!slots && (long long)B * W > n_slots) return bad(fn, "n_slots must be >= B*W without slots");
  if ((long long)B * layers > (1 << 27) || (long long)B * W > INT_MAX) return bad(fn, "B*layers too large");
  if ((row_bytes | ld_row | ld_layer) & 3) return bad(fn, "row_bytes, ld_row and ld_layer must be multiples of 4");
  if (ld_row < row_bytes || ld_layer < 0) return bad(fn, "ld_row must cover a row");
  if (row_bytes >> 34) return bad(fn, "row_bytes must be below 2^34");
  if (B == 0 || layers == 0 || row_bytes == 0 || n_slots == 0) return LA_OK;
  if (!pool || !parent) return bad(fn, "pool and parent are required");
  if (!at(pool, 4) || !at(parent, 4) || !at(slots, 4)) return bad(fn, "pointers must be 4-byte aligned");
  if (same({pool}, {slots, parent})) return bad(fn, "pool must not be another argument");
  const BeamStates p = {pool, slots, parent, B, W, n_slots, layers, row_bytes, ld_row, ld_layer};
  return launch_beam_states(p, reinterpret_cast<cudaStream_t>(stream));
}

int la_beam_cache(void *k_cache, void *v_cache, int *table, const int *lens, const int *parent, int B, int W,
                  int page_size, int n_pages, int max_pages, long long ld_table, int layers, long long token_bytes,
                  long long ld_page, long long ld_layer, la_stream_t stream) {
  NvtxRange nvtx_range("la_beam_cache");
  const char *fn = "la_beam_cache";
  set_error("%s", "");
  if (B < 0 || layers < 0 || token_bytes < 0) return bad(fn, "B, layers and token_bytes must be >= 0");
  if (W < 1 || W > kMaxBeams) return unsupported(fn, "W must be 1..32", W);
  const PagedCache c = {table, lens, ld_table, ld_page, page_size, n_pages, max_pages};
  const int rc = check_cache(fn, c, token_bytes);
  if (rc) return rc;
  if ((long long)B * (layers + 1) > (1 << 26) || (long long)B * W > INT_MAX) return bad(fn, "B*layers too large");
  if ((token_bytes | ld_page | ld_layer) & 3) return bad(fn, "token_bytes, ld_page and ld_layer must be multiples of 4");
  if (ld_layer < 0) return bad(fn, "ld_layer must be >= 0");
  if (page_size * token_bytes >> 34) return bad(fn, "a page must be below 2^34 bytes");
  if (B == 0 || max_pages == 0) return LA_OK;
  if (!table || !lens || !parent) return bad(fn, "table, lens and parent are required");
  if (layers > 0 && n_pages > 0 && (!k_cache || !v_cache)) return bad(fn, "k_cache and v_cache are required");
  if (!at(k_cache, 4) || !at(v_cache, 4) || !at(parent, 4)) return bad(fn, "pointers must be 4-byte aligned");
  if (same({k_cache, v_cache, table}, {lens, parent})) return bad(fn, "caches and table must not be another argument");
  const BeamCache p = {k_cache, v_cache, table, lens, parent, B, W, page_size, n_pages, max_pages, layers, ld_table,
                       token_bytes, ld_page, ld_layer};
  return launch_beam_cache(p, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
