// Internal declarations of the serving operators (include/la_serve.h): paged
// cache, attention over it, beam selection and reordering.
#pragma once

#include "../../include/la_serve.h"
#include "la_layer_internal.h"

namespace la {

// Where the tokens of a paged cache are.
struct PagedCache {
  const int *table, *lens;
  long long ld_table, ld_page;  // entries, elements
  int page_size, n_pages, max_pages;
};

struct AppendParams {
  const void *q, *k, *v;
  void *q_out, *k_cache, *v_cache;
  PagedCache at;
  const int *cu, *pos;
  const double *freq;
  int n_axes, s0, s1, s2;
  int n_seq, total, H, Hk, d;  // H = 0: no queries
  long long ldq, ldk, ldv;
  int interleaved, f32;
};
int launch_cache_append(const AppendParams &p, cudaStream_t stream);

struct PagedAttn {
  const void *q, *k_cache, *v_cache;
  void *o;
  float *lse;
  PagedCache at;
  int n, H, Hk, d, max_len, window;
  float scale;
  long long ldq;
  int f32;
};
int launch_paged_attn(const PagedAttn &p, cudaStream_t stream);

struct BeamSelect {
  const void *logits;
  const float *scores;
  const unsigned char *done;
  float *scores_out;
  int *parent, *token;
  int B, W, V, K, eos, f32;
  long long ld;
};
int launch_beam_select(const BeamSelect &p, cudaStream_t stream);

// Rows of pools that take another row's place: for request b and beam w, row w's
// bytes become those of row parent[b][w], for all w at once.
struct BeamStates {
  void *pool;
  const int *slots, *parent;
  int B, W, n_slots, layers;
  long long row_bytes, ld_row, ld_layer;
};
int launch_beam_states(const BeamStates &p, cudaStream_t stream);

struct BeamCache {
  void *k_cache, *v_cache;
  int *table;
  const int *lens, *parent;
  int B, W, page_size, n_pages, max_pages, layers;
  long long ld_table, token_bytes, ld_page, ld_layer;
};
int launch_beam_cache(const BeamCache &p, cudaStream_t stream);

constexpr int kMaxBeams = 32;   // beams of a request, and candidates that a selection keeps

}  // namespace la
