// Internal declarations of the serving operators (include/la_serve.h): paged
// cache, attention over it, beam selection and reordering.
#pragma once

#include "../../include/la_serve.h"
#include "la_layer_internal.h"

namespace la {

// The kernels of a decoding step are short and follow one another: each is launched
// programmatically, so that it may be set up while what stands in front of it in
// the stream still runs, and waits for that (wait_for_stream) before it touches
// memory, by loads that are not of the read-only kind (a kernel in front may be
// writing in this one's lifetime). Kernels behind it are let through at the same point.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                         const Args &...args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}
__device__ __forceinline__ void wait_for_stream() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

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

// The units [first, end) of `total` numbered ones that are a CTA's, `share` to each.
struct UnitRun {
  int first, end;
};
__host__ __device__ inline int share_of(int total, unsigned ctas) {
  const unsigned share = (static_cast<unsigned>(total) + ctas - 1) / ctas;
  return share > 0 ? static_cast<int>(share) : 1;
}
__host__ __device__ inline UnitRun run_of(unsigned cta, int share, int total) {
  const long long first = (long long)cta * share, end = first + share;  // (an int may hold total only)
  return {static_cast<int>(first < total ? first : total), static_cast<int>(end < total ? end : total)};
}

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
