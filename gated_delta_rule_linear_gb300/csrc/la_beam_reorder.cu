// The chosen beams' states and pages: row w of a request's W rows becomes what
// row parent[w] was, for all w at once and in place.
//
// Bound by HBM traffic: a row is read once if it is the parent of another one,
// and written if its parent is another one; rows that stay are not touched.
// A thread takes a column of all W rows: it reads the parents' values into
// registers before it writes any, so no row needs a second place. Registers are
// indexed by the parent, an unrolled loop, and a parent's value goes to its
// children's rows one after the other (a bit mask), so that nothing is indexed
// by what is only known at run time.
#include <algorithm>

#include "la_serve_internal.h"

namespace la {
namespace {

constexpr int kThreads = 256;

// What a request's rows do: kids[p] are the rows that become row p, source the rows with such kids.
struct Moves {
  unsigned kids[kMaxBeams];
  char *row[kMaxBeams];
  unsigned source;
};

// Filled by the block's first warp; row: this lane's row, or null if it has none.
__device__ __forceinline__ void read_moves(Moves &m, const int *parent, int W, char *row) {
  const int w = threadIdx.x;
  if (w < 32) {
    const int from = w < W && row ? __ldg(parent + w) : -1;
    const unsigned there = __ballot_sync(~0u, row != nullptr);
    const bool moves = from >= 0 && from < W && from != w && ((there >> from) & 1);
    unsigned source = 0;
    for (int p = 0; p < W; ++p) {
      const unsigned kids = __ballot_sync(~0u, moves && from == p);
      if (w == p) m.kids[p] = kids;
      if (kids) source |= 1u << p;
    }
    m.row[w] = row;
    if (w == 0) m.source = source;
  }
  __syncthreads();
}

// Columns first, first + stride, .. below n of type U.
template <typename U, int WMAX>
__device__ __forceinline__ void move_columns(const Moves &m, long long first, long long n, long long stride) {
  const unsigned source = m.source;
  if (!source) return;
  for (long long c = first; c < n; c += stride) {
    U val[WMAX];
#pragma unroll
    for (int p = 0; p < WMAX; ++p)
      if (source >> p & 1) val[p] = reinterpret_cast<const U *>(m.row[p])[c];
#pragma unroll
    for (int p = 0; p < WMAX; ++p)
      if (source >> p & 1)
        for (unsigned k = m.kids[p]; k; k &= k - 1) reinterpret_cast<U *>(m.row[__ffs(k) - 1])[c] = val[p];
  }
}

template <typename U, int WMAX>
__global__ void __launch_bounds__(kThreads) states_kernel(const BeamStates p, int chunks) {
  __shared__ Moves m;
  const unsigned i = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int l = i % p.layers, b = i / p.layers, w = threadIdx.x;
  char *row = nullptr;
  if (w < p.W) {
    const int at = b * p.W + w, slot = p.slots ? __ldg(p.slots + at) : at;
    if (slot >= 0 && slot < p.n_slots) row = static_cast<char *>(p.pool) + l * p.ld_layer + slot * p.ld_row;
  }
  read_moves(m, p.parent + (size_t)b * p.W, p.W, row);
  move_columns<U, WMAX>(m, (long long)chunk * kThreads + threadIdx.x, p.row_bytes / (long long)sizeof(U),
                        (long long)chunks * kThreads);
}

template <typename U, int WMAX>
__global__ void __launch_bounds__(kThreads) cache_kernel(const BeamCache p, const FastDiv by_page, int chunks) {
  __shared__ Moves m;
  const unsigned jobs = 2 * p.layers * chunks + 1, b = blockIdx.x / jobs, w = threadIdx.x;
  unsigned job = blockIdx.x % jobs;
  const int len = min((long long)max(__ldg(p.lens + (size_t)b * p.W), 0), (long long)p.max_pages * p.page_size);
  uint32_t open, fill;
  by_page.split(len, open, fill);
  int *entries = p.table + ((size_t)b * p.W + w) * p.ld_table;
  const int *parent = p.parent + (size_t)b * p.W;
  if (job == 0) {  // the table
    read_moves(m, parent, p.W, (int)w < p.W ? reinterpret_cast<char *>(entries) : nullptr);
    move_columns<int, WMAX>(m, threadIdx.x, open, kThreads);
    return;
  }
  if (fill == 0) return;  // (open < max_pages otherwise)
  --job;
  const int chunk = job % chunks, l = job / chunks % p.layers, which = job / chunks / p.layers;
  char *row = nullptr;
  if ((int)w < p.W) {
    const int page = __ldg(entries + open);  // behind the entries that are moved
    if (page >= 0 && page < p.n_pages) row = static_cast<char *>(which ? p.v_cache : p.k_cache) + l * p.ld_layer + page * p.ld_page;
  }
  read_moves(m, parent, p.W, row);
  move_columns<U, WMAX>(m, (long long)chunk * kThreads + threadIdx.x, fill * p.token_bytes / (long long)sizeof(U),
                        (long long)chunks * kThreads);
}

// Blocks of a row's columns: one column a thread, up to `most` blocks in all.
int chunks_of(long long columns, long long rows, long long most) {
  const long long c = (columns + kThreads - 1) / kThreads;
  return static_cast<int>(std::max(1ll, std::min(c, most / std::max(rows, 1ll))));
}

long long most_blocks() { return 64ll * std::max(sm_count(), 1); }

template <typename U>
cudaError_t states(const BeamStates &p, cudaStream_t stream) {
  const long long rows = (long long)p.B * p.layers;
  const int chunks = chunks_of(p.row_bytes / (long long)sizeof(U), rows, most_blocks());
  const unsigned grid = static_cast<unsigned>(rows * chunks);  // the caller keeps B * layers below 2^27
  if (p.W <= 4) states_kernel<U, 4><<<grid, kThreads, 0, stream>>>(p, chunks);
  else if (p.W <= 8) states_kernel<U, 8><<<grid, kThreads, 0, stream>>>(p, chunks);
  else if (p.W <= 16) states_kernel<U, 16><<<grid, kThreads, 0, stream>>>(p, chunks);
  else states_kernel<U, 32><<<grid, kThreads, 0, stream>>>(p, chunks);
  return cudaGetLastError();
}

template <typename U>
cudaError_t cache(const BeamCache &p, cudaStream_t stream) {
  const long long rows = 2ll * p.B * p.layers;
  const int chunks = chunks_of(p.page_size * p.token_bytes / (long long)sizeof(U), rows, most_blocks());
  const unsigned grid = static_cast<unsigned>(rows * chunks + p.B);
  const FastDiv by(p.page_size);
  if (p.W <= 4) cache_kernel<U, 4><<<grid, kThreads, 0, stream>>>(p, by, chunks);
  else if (p.W <= 8) cache_kernel<U, 8><<<grid, kThreads, 0, stream>>>(p, by, chunks);
  else if (p.W <= 16) cache_kernel<U, 16><<<grid, kThreads, 0, stream>>>(p, by, chunks);
  else cache_kernel<U, 32><<<grid, kThreads, 0, stream>>>(p, by, chunks);
  return cudaGetLastError();
}

// Whether an address and its strides allow 16 bytes at a time.
bool wide(const void *p, long long a, long long b, long long c) {
  return ((reinterpret_cast<uintptr_t>(p) | a | b | c) & 15) == 0;
}

int done(const char *fn, cudaError_t e) {
  if (e == cudaSuccess) return LA_OK;
  set_error("%s: launch failed: %s", fn, cudaGetErrorString(e));
  return LA_ERR_CUDA;
}

}  // namespace

int launch_beam_states(const BeamStates &p, cudaStream_t stream) {
  return done("la_beam_states", wide(p.pool, p.row_bytes, p.ld_row, p.ld_layer) ? states<uint4>(p, stream)
                                                                                 : states<unsigned>(p, stream));
}

int launch_beam_cache(const BeamCache &p, cudaStream_t stream) {
  const bool w = wide(p.k_cache, p.token_bytes, p.ld_page, p.ld_layer) && wide(p.v_cache, 0, 0, 0);
  return done("la_beam_cache", w ? cache<uint4>(p, stream) : cache<unsigned>(p, stream));
}

}  // namespace la
