// The chosen beams' states and pages: row w of a request's W rows becomes what
// row parent[w] was, for all w at once and in place.
//
// Bound by HBM traffic: a row is read once if it is the parent of another one,
// and written if its parent is another one; rows that stay are not touched.
// A thread takes a column of all W rows: it reads what each row becomes into
// registers before it writes any, so no row needs a second place. A parent of
// several is asked for several times, and comes from memory once.
//
// 8 requests of 4 beams, 2 layers of 16 x 128 x 128 states (69 MB read and
// written): 13.6 us, 5.1 TB/s. Pages of 16 requests of 8 beams, 4 layers (18 MB):
// 9.7 us, the chain lengths -> table -> pages -> store; one block a layer and pool
// instead of all of a request's columns in a row: 9 us of three times the blocks.
#include <algorithm>

#include "la_serve_internal.h"

namespace la {
namespace {

constexpr int kThreads = 256;

// Which rows of a request move, where they start and where their parents do.
struct Moves {
  longlong2 at[kMaxBeams];  // byte of the parent's row, byte of the row
  unsigned rows;
};

// Filled by the block's first warp: lane w's parent is `from`, its row starts at byte `at` (-1: it has none).
__device__ __forceinline__ void set_moves(Moves &m, int W, int from, long long at) {
  const int w = threadIdx.x;
  if (w < 32) {
    const unsigned there = __ballot_sync(~0u, w < W && at >= 0);
    const bool moves = (there >> w & 1) && from >= 0 && from < W && from != w && (there >> from & 1);
    const long long theirs = __shfl_sync(~0u, at, from & 31);
    m.at[w] = make_longlong2(theirs, at);
    const unsigned rows = __ballot_sync(~0u, moves);
    if (w == 0) m.rows = rows;
  }
  __syncthreads();
}

// The rows of `pools` pools (one at least), pool(l) their bases, each of n columns of type U; this thread is number
// `thread` of `threads`.
template <typename U, int WMAX, typename Pool>
__device__ __forceinline__ void move_columns(const Moves &m, Pool pool, unsigned pools, unsigned n, unsigned thread,
                                             unsigned threads) {
  const unsigned rows = m.rows;
  unsigned l = 0;
  for (unsigned long long c = thread;; c += threads) {
    while (c >= n) {
      c -= n;
      if (++l >= pools) return;
    }
    asm volatile("" ::: "memory");  // the rows' places stay in shared memory: held, they would take the registers
    char *at = pool(l) + c * sizeof(U);
    U val[WMAX];
#pragma unroll
    for (int i = 0; i < WMAX; ++i)
      if (rows >> i & 1) val[i] = *reinterpret_cast<const U *>(at + m.at[i].x);
#pragma unroll
    for (int i = 0; i < WMAX; ++i)
      if (rows >> i & 1) *reinterpret_cast<U *>(at + m.at[i].y) = val[i];
  }
}

// Block (request, chunk of the columns): all layers.
template <typename U, int WMAX>
__global__ void __launch_bounds__(kThreads) states_kernel(const BeamStates p, int chunks) {
  __shared__ Moves m;
  const int chunk = blockIdx.x % chunks, b = blockIdx.x / chunks, w = threadIdx.x;
  wait_for_stream();
  int from = -1;
  long long at = -1;
  if (w < p.W) {
    const int i = b * p.W + w, slot = p.slots ? p.slots[i] : i;
    from = p.parent[i];
    if (slot >= 0 && slot < p.n_slots) at = slot * p.ld_row;
  }
  set_moves(m, p.W, from, at);
  if (!m.rows) return;
  move_columns<U, WMAX>(m, [&](unsigned l) { return static_cast<char *>(p.pool) + l * p.ld_layer; }, p.layers,
                        static_cast<unsigned>(p.row_bytes / sizeof(U)), chunk * kThreads + w, chunks * kThreads);
}

// Block (request, chunk): chunk 0 the table, the others the open pages of all layers' keys and values.
template <typename U, int WMAX>
__global__ void __launch_bounds__(kThreads) cache_kernel(const BeamCache p, const FastDiv by_page, int chunks) {
  __shared__ Moves m;
  const int b = blockIdx.x / (chunks + 1), chunk = static_cast<int>(blockIdx.x % (chunks + 1)) - 1, w = threadIdx.x;
  wait_for_stream();
  int from = -1;
  if (w < p.W) from = p.parent[b * p.W + w];
  const int len = min((long long)max(p.lens[(size_t)b * p.W], 0), (long long)p.max_pages * p.page_size);
  uint32_t open, fill;
  by_page.split(len, open, fill);
  int *table = p.table + (long long)b * p.W * p.ld_table;
  if (chunk < 0) {
    set_moves(m, p.W, from, w < p.W ? w * p.ld_table * 4 : -1);
    if (m.rows && open) move_columns<int, WMAX>(m, [&](unsigned) { return reinterpret_cast<char *>(table); }, 1, open, w, kThreads);
    return;
  }
  if (fill == 0) return;  // (open < max_pages otherwise)
  long long at = -1;
  if (w < p.W) {
    const int page = table[w * p.ld_table + open];  // behind the entries that chunk 0 moves
    if (page >= 0 && page < p.n_pages) at = page * p.ld_page;
  }
  set_moves(m, p.W, from, at);
  if (!m.rows) return;
  move_columns<U, WMAX>(m, [&](unsigned l) {
    return static_cast<char *>(l & 1 ? p.v_cache : p.k_cache) + (l >> 1) * p.ld_layer;
  }, 2 * p.layers, static_cast<unsigned>(fill * p.token_bytes / sizeof(U)), chunk * kThreads + w, chunks * kThreads);
}

// Blocks of a request: a column a thread, up to those that are on the SMs together.
int chunks_of(long long columns, int requests) {
  const long long c = (columns + kThreads - 1) / kThreads, most = 8ll * std::max(sm_count(), 1) / requests;
  return static_cast<int>(std::max(1ll, std::min(c, most)));
}

template <typename U>
cudaError_t states(const BeamStates &p, cudaStream_t stream) {
  const int chunks = chunks_of(p.layers * (p.row_bytes / (long long)sizeof(U)), p.B);
  const unsigned grid = static_cast<unsigned>(p.B) * chunks;  // (B of one chunk, or a few for each SM)
  if (p.W <= 4) return launch_early(states_kernel<U, 4>, dim3(grid), kThreads, 0, stream, p, chunks);
  if (p.W <= 8) return launch_early(states_kernel<U, 8>, dim3(grid), kThreads, 0, stream, p, chunks);
  if (p.W <= 16) return launch_early(states_kernel<U, 16>, dim3(grid), kThreads, 0, stream, p, chunks);
  return launch_early(states_kernel<U, 32>, dim3(grid), kThreads, 0, stream, p, chunks);
}

template <typename U>
cudaError_t cache(const BeamCache &p, cudaStream_t stream) {
  // (no layers, or tokens of no bytes: the table alone, as a block of the others would take the first pool for its own)
  const long long columns = 2 * p.layers * (p.page_size * p.token_bytes / (long long)sizeof(U));
  const int chunks = columns > 0 ? chunks_of(columns, p.B) : 0;
  const unsigned grid = static_cast<unsigned>(p.B) * (chunks + 1);
  const FastDiv by(p.page_size);
  if (p.W <= 4) return launch_early(cache_kernel<U, 4>, dim3(grid), kThreads, 0, stream, p, by, chunks);
  if (p.W <= 8) return launch_early(cache_kernel<U, 8>, dim3(grid), kThreads, 0, stream, p, by, chunks);
  if (p.W <= 16) return launch_early(cache_kernel<U, 16>, dim3(grid), kThreads, 0, stream, p, by, chunks);
  return launch_early(cache_kernel<U, 32>, dim3(grid), kThreads, 0, stream, p, by, chunks);
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
