// Packed retention on tcgen05 + TMEM + TMA, bf16 inputs, float32 state: the
// passes of la_packed_fwd and la_packed_bwd (PackedPass).
//
// Chunks of 128 tokens, rows i, j of a chunk of n rows ("Talk Linear Attention"
// sections 3.2 and 5.2), with the state S (da x 64 value columns) that enters
// the chunk:
//
//   P   = (X Y^T) . gamma^(i-j), j <= i     out = gamma^(i+1) (X S) + P Z
//   S  <- gamma^n S + dS,                   dS  = Y^T Z',  Z' = gamma^(n-1-j) Z
//
// and for reversed passes gamma^(j-i) over j >= i, gamma^(n-1-i) for the row and
// gamma^(j+1) for Z, chunks from the last to the first. The decay of a head is
// one number, so every power comes from a table of gamma^0 .. gamma^128.
//
// Work. A unit is one segment (up to seg tokens) of one sequence; an item of
// work is a unit, a head and 64 value columns. One CTA a SM takes items from a
// queue, the longest first, and the roles below go from one item's last chunk to
// the next one's first without draining. Sequences longer than the segment first
// go through the same kernel with STATE set, which only forms each segment's own
// contribution to the state (the last one's is not asked for), and a scan over
// the segments. Their states lie in a workspace, a row for each segment of a
// split sequence: a sequence of n > 1 segments is longer than n - 1 of them, so
// that there are at most total / seg segments but the last ones, and at most
// twice as many in all, however many sequences the call has.
//
// The state stays in registers: every chunk's dS is formed in a TMEM tile of
// its own and added by float32 FMAs, gamma^n - 1 carrying the decay. Adding in
// TMEM instead would cut every product's sum at the accumulator's last bit, and
// thousands of tokens of that show in a float32 state. For the same reason Z'
// goes to the tensor cores as a bf16 high and low part (2^-16), side by side as
// one operand of twice the width: one part alone would leave the state with
// bf16's error. P and the state's copy for X S are rounded to bf16 once; their
// errors are of the order of the output's own rounding.
//
// Out-of-sequence rows: a tile may reach into the next sequence or behind the
// last token. The foreign rows of Z, and of Y once its scores are formed, are
// cleared in shared memory, and the foreign columns of the scores dropped by
// selection, so that whatever they hold (NaN included) stays out; foreign rows
// of X reach only output rows that are not written.
//
// Roles, 896 threads. Every group works on its own part of a chunk and hands it
// on through mbarriers, up to two chunks apart; a group of its own for each
// step, because the steps are bound by their instructions' latency:
//   warp 0        the queue, tables of powers, TMA loads of X, Y, Z, two stages
//   warps 1-3     MMAs: dS and X S; scores (and TMEM); P Z
//   warps 4-7     state: S <- gamma^n S + dS, its bf16 copy
//   warps 8-11    output: gamma^(i+1) X S + P Z, to memory by TMA
//   warps 12-19   Z' high and low
//   warps 20-27   P, in TMEM over its scores
// Measured on GB300, 16 heads of 128, bf16: forward of 4 x 16384 tokens 0.247 ms
// (1.08 GB, 4.4 TB/s), one CTA for each of 128 heads and value tiles at about
// 3450 cycles a chunk. What sets that period (clock64 traces, ncu): the way of a
// chunk through the roles, about 6900 cycles with two chunks in flight (shared
// memory and TMEM hold no third): 8 tensor instructions of a product take 700 to
// 1100 cycles to issue (the pipe itself is busy 1500 of 3450), P 1100, the output
// 600, loads 1400. A change of item costs about 2 periods more, most of it cold
// code: the steady state already fills the instruction cache.
// Every wait is bounded; on expiry the CTA raises the status word, all roles
// leave, copies and MMAs in flight are drained and TMEM is released.
#include <algorithm>
#include <atomic>
#include <climits>

#include "la_f32x2.cuh"
#include "la_layer_internal.h"
#include "la_tc_common.cuh"

namespace la {
namespace {

using namespace sm100;
using namespace tc;
using f32x2::add2;
using f32x2::fma2;
using f32x2::mul2;
using f32x2::pair;

constexpr int kThreads = 896, kN = 128;  // tokens of a chunk
constexpr uint32_t kSpin = 1u << 22;     // polls before a wait gives up (tens of milliseconds at least)
// Registers a thread of each group of four warps, together at most what the block was
// launched with, 7 * 72: issue, state, output, twice Z', twice P.
constexpr int kRegsIssue = 56, kRegsState = 104, kRegsOut = 88, kRegsP = 72, kRegsZ = 56;
static_assert(kRegsIssue + kRegsState + kRegsOut + 2 * kRegsP + 2 * kRegsZ <= 7 * 72, "register split");

// A unit as the plan writes it: tokens [t0, t1), its row of the segments' states (of split
// sequences only), and 4 * state row + 2 * (it is all of its sequence) + (the state behind it is its
// sequence's last); state row -1: none.
struct Unit {
  int t0, t1, u, row;
};

// A sequence of more than one unit: tokens [a, b), its first row of the segments' states, its state row or -1.
struct Split {
  int a, b, u, row;
};

struct Segments {
  int tokens;        // of a segment; 0: every sequence is one unit
  int units;         // at most this many; STATE: segments with a state to form
  const Unit *plan;  // units with something to do, the longest first (STATE: those segments, in any order), or null:
                     // unit u is sequence u, one item a CTA
  const int *count;  // how many of them
  unsigned *queue;   // next item for a CTA that is done, from zero
  const float *in;   // [row][H][dk][dv] entering states of split sequences' segments; the others': S_in by row
  float *out;        // STATE: the segments' own contributions
};

// One item of work: a unit, a head and 64 value columns. chunks < 0: no more items.
struct Item {
  int t0, t1, chunks, h, v0, u, slot, leaves, whole;
};

__device__ __forceinline__ int chunks_of(int tokens) { return (tokens + kN - 1) / kN; }

// Where a long walk is left for the end the other SMs wait for it: the plan
// lists the units from the longest down (a counting sort over their chunks; the
// order of equal ones is arbitrary, and no result goes by it). Split sequences
// and those of their segments whose state the others start from stand in lists
// of their own, so that the passes over them do not go by the number of
// sequences. One CTA a pass; clears the queues on the way.
constexpr int kPlanThreads = 1024, kBuckets = 1024;
// Words of `head`: queue and count of the state kernel, queue and count of the main one, split sequences.
constexpr int kStateQueue = 0, kMainQueue = 1, kUnitCount = 2, kSegmentCount = 3, kSplitCount = 4;
struct PlanJob {
  PackedPass p;
  int seg, units, most;  // most: segments with a state to form, no more than total / seg
  unsigned *head;
  int *owner;
  Unit *plan, *segments;
  Split *splits;
};
struct PlanJobs {
  PlanJob job[3];
};
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanJobs jobs) {
  const PackedPass &p = jobs.job[blockIdx.x].p;
  const int seg = jobs.job[blockIdx.x].seg, units = jobs.job[blockIdx.x].units;
  unsigned *head = jobs.job[blockIdx.x].head;
  int *owner = jobs.job[blockIdx.x].owner;
  const int most = jobs.job[blockIdx.x].most;
  Unit *plan = jobs.job[blockIdx.x].plan, *segments = jobs.job[blockIdx.x].segments;
  Split *splits = jobs.job[blockIdx.x].splits;
  __shared__ int first[kBuckets];
  __shared__ int warp_sum[32];
  __shared__ unsigned long long taken;  // segments given out
  __shared__ int split, given, end;     // split sequences, rows of theirs; where there was no more room
  const int tid = threadIdx.x;
  if (tid < 2) head[tid] = 0;
  if (tid == 0) taken = split = given = 0, end = most;
  first[tid] = 0;
  const bool rows = p.S_in || p.S_out;
  if (rows && p.slots) {  // of sequences that name the same row the first one has it
    for (int i = tid; i < p.n_seq; i += kPlanThreads) {
      const int slot = __ldg(p.slots + i);
      if (slot >= 0 && slot < p.n_slots) owner[slot] = INT_MAX;
    }
    __syncthreads();
    for (int i = tid; i < p.n_seq; i += kPlanThreads) {
      const int slot = __ldg(p.slots + i);
      if (slot >= 0 && slot < p.n_slots) atomicMin(owner + slot, i);
    }
  }
  __syncthreads();
  for (int pass = 0; pass < 2; ++pass) {
    for (int i = tid; i < p.n_seq; i += kPlanThreads) {
      int a, b;
      packed_range(p.cu, i, p.total, &a, &b);
      const int n = seg ? max(1, (b - a + seg - 1) / seg) : 1;
      int row = -1;
      if (rows) {
        row = p.slots ? __ldg(p.slots + i) : i;
        if (row < 0 || row >= p.n_slots || (p.slots && *const_cast<volatile int *>(owner + row) != i)) row = -1;
      }
      if (b == a && !(p.S_out && row >= 0)) continue;  // nothing to do
      bool room = true;                                // (none only where sequences overlap, as they should not)
      int formed = 0, u0 = 0;                          // first of its segments with a state to form, first row of all
      if (pass && n > 1) {
        const unsigned long long at = atomicAdd(&taken, n - 1ull);
        room = at + (n - 1) <= most;
        formed = static_cast<int>(min(at, static_cast<unsigned long long>(most)));
        if (room) {
          u0 = atomicAdd(&given, n);
          splits[atomicAdd(&split, 1)] = {a, b, u0, row};
        } else {
          atomicMin(&end, formed);
        }
      }
      for (int k = 0; k < n; ++k) {
        const int t0 = a + k * seg, t1 = seg ? min(b, t0 + seg) : b;
        const int bucket = kBuckets - 1 - min(chunks_of(t1 - t0), kBuckets - 1);
        const int at = atomicAdd(first + bucket, 1);
        const bool leaves = p.reverse ? k == 0 : k == n - 1;
        if (!pass) continue;
        if (!leaves && room) segments[formed++] = {t0, t1, u0 + k, 0};
        if (static_cast<unsigned>(at) < static_cast<unsigned>(units)) {
          if (room) plan[at] = {t0, t1, u0 + k, 4 * row + 2 * (n == 1) + leaves};
          else plan[at] = {a, a, 0, -1};  // no tokens, no state
        }
      }
    }
    __syncthreads();
    if (pass) {
      if (tid == 0) head[kSegmentCount] = min(taken, static_cast<unsigned long long>(end)), head[kSplitCount] = split;
      break;
    }
    // exclusive prefix sums of the buckets
    int v = first[tid], x = v;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if ((tid & 31) >= o) x += y;
    }
    if ((tid & 31) == 31) warp_sum[tid >> 5] = x;
    __syncthreads();
    if (tid < 32) {
      int y = warp_sum[tid];
      for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (tid >= o) y += z;
      }
      warp_sum[tid] = y;
    }
    __syncthreads();
    x += tid >= 32 ? warp_sum[(tid >> 5) - 1] : 0;
    first[tid] = x - v;
    if (tid == kPlanThreads - 1) head[kUnitCount] = min(x, units);
    __syncthreads();
  }
}

// Shared memory, in 16 KB tiles (128 rows of 64 bf16, 128-byte swizzle).
constexpr uint32_t kTile = 16384;
constexpr uint32_t kSmX = 0, kSmY = kSmX + 4 * kTile, kSmZ = kSmY + 4 * kTile, kSmW = kSmZ + 2 * kTile,
                   kSmS = kSmW + 2 * kTile, kSmO = kSmS + kTile, kSmMisc = kSmO + kTile,
                   kSmBytes = kSmMisc + 3 * 1024;
constexpr int kRing = 4;  // items known ahead
// TMEM columns: two buffers of scores, over which go P (columns 0..63) and P Z (64..127),
// two of X S, and dS of Z' high and low.
constexpr uint32_t kColSc = 0, kColPZ = 64, kColXS = 256, kColD = 384;

// 32 lanes x 32 bits, 8 consecutive columns per thread.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float *v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// Descriptors as desc_sw128's, from the operand's address: the strides are constants, so
// the upper word is one too and only the lower word has to be moved to the issue unit.
__device__ __forceinline__ uint64_t desc(uint32_t saddr, uint32_t lbo) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"((saddr >> 4) | (lbo >> 4) << 16), "n"(1024 >> 4 | 1 << 14 | 2 << 29));
  return d;
}

// An infinity as the largest float of its sign.
__device__ __forceinline__ float finite(float a) {
  float r;
  asm("min.NaN.xorsign.abs.f32 %0, %1, 0f7F7FFFFF;" : "=f"(r) : "f"(a));
  return r;
}

template <int R> __device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R> __device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

template <int DA, bool STATE, bool OF32>
__global__ void __launch_bounds__(kThreads, 1)
packed_tc_kernel(const PackedPass p, const Segments sg, const __grid_constant__ CUtensorMap tm_x,
                 const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ CUtensorMap tm_z,
                 const __grid_constant__ CUtensorMap tm_o) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wq = warp & 3, group = warp >> 2;
  if ((smem_u32(sm) & 1023u) != 0) {  // the tiles' swizzle goes by the address: not met, as there is no static part
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    return;
  }
  const int db = p.db;
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + kSmMisc);
  uint64_t *xy_full = bars, *xy_free = bars + 2, *z_full = bars + 4, *z_free = bars + 6, *sc_full = bars + 8,
           *p_ready = bars + 10, *w_ready = bars + 12, *o_full = bars + 14, *o_free = bars + 16, *t_full = bars + 18,
           *t_free = bars + 20, *d_full = bars + 22, *d_free = bars + 23, *s_ready = bars + 24, *xs_full = bars + 25,
           *drain = bars + 26, *e_full = bars + 29, *e_free = bars + 29 + kRing;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 29 + 2 * kRing);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  Item *ring = reinterpret_cast<Item *>(sm + kSmMisc + 384);
  // Two tables of powers of gamma, of two items' heads: [127 + e] is gamma^e, [0 .. 126] zero
  // (reversed: [127 - e], and zeros behind), [255] is gamma^128. At [127 + i - j] stands the
  // factor of a score, zero where j is not seen from i.
  float *tables = reinterpret_cast<float *>(sm + kSmMisc + 1024);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // see launch_packed_tc
  if (warp == 2) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&xy_full[i], 1);
      mbar_init(&xy_free[i], STATE ? 1 : 2);  // dS and X S, scores
      mbar_init(&z_full[i], 1);
      mbar_init(&z_free[i], STATE ? 1 : 2);   // dS (behind it Z'), P Z
      mbar_init(&sc_full[i], 1);
      mbar_init(&p_ready[i], 8);
      mbar_init(&w_ready[i], 8);
      mbar_init(&o_full[i], 2);  // X S, P Z
      mbar_init(&o_free[i], 4);
      mbar_init(&t_full[i], 1);
      mbar_init(&t_free[i], STATE ? 8 : 20);  // Z' (output, P)
    }
    mbar_init(d_full, 1);
    mbar_init(d_free, 4);
    mbar_init(s_ready, 4);
    mbar_init(xs_full, 1);
    for (int i = 0; i < 3; ++i) mbar_init(&drain[i], 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&e_full[i], 1);
      mbar_init(&e_free[i], STATE ? 13 : 27);  // dS, state, Z' (scores, P Z, output, P)
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (DA == 64) {  // channels 64..127 of Y: zero rows of dS
    for (int i = tid; i < 2 * 1024; i += kThreads)
      reinterpret_cast<uint4 *>(sm + kSmY + (2 * (i >> 10) + 1) * kTile)[i & 1023] = make_uint4(0, 0, 0, 0);
    fence_proxy_async();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const uint32_t tl = tbase + (static_cast<uint32_t>(wq * 32) << 16);
  // The loop is as short as it can be: the code that all roles run for a chunk has to stay in the
  // SM's instruction cache together. With the waits, products and conversions unrolled in place
  // it did not, and a chunk took three times as long. A role whose wait runs out leaves, and the
  // others run out after it.
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    uint32_t left;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmov.u32 %0, %3;\n\t"
        "LA_POLL:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra LA_DONE;\n\t"
        "sub.u32 %0, %0, 1;\n\t"
        "setp.ne.u32 p, %0, 0;\n\t"
        "@p bra LA_POLL;\n\t"
        "LA_DONE:\n\t}"
        : "=&r"(left)
        : "r"(smem_u32(bar)), "r"(parity & 1), "n"(kSpin)
        : "memory");
    if (left == 0) *abort_flag = 1;
    return left != 0;
  };
  // A group of four warps waits: one lane polls, the others sleep on the group's barrier.
  // With a polling lane in each of 24 warps the polls took more issue slots than the work.
  auto wait_group = [&](uint64_t *bar, uint32_t parity) {
    bool ok = true;
    if (wq == (group & 2) && lane == 0) ok = wait(bar, parity);  // not on the schedulers of warps 1 and 3
    return group_all(ok, group);
  };
  // Item k of this CTA, in its ring place; the chunk of its j-th turn.
  auto item_at = [&](int k) { return ring[k & (kRing - 1)]; };
  auto chunk_at = [&](const Item &it, int j) { return p.reverse ? it.chunks - 1 - j : j; };
  auto item_done = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&e_free[k & (kRing - 1)]);
  };
#define LA_ITEM_FULL(k) &e_full[(k) & (kRing - 1)], (k) / kRing

  // In every role: k counts items, n chunks of all items; a chunk's buffers and phases go by n.
  if (warp < 4) {
    regs_down<kRegsIssue>();
    if (warp == 0) {
      // ------------------------------------------- items, and their TMA loads
      if (lane == 0) {
        prefetch_tmap(&tm_y);
        prefetch_tmap(&tm_z);
        if (!STATE) prefetch_tmap(&tm_x);
      }
      const int vtiles = db / 64, per = vtiles * p.H;
      const int items = sg.plan ? *sg.count * per : gridDim.x;
      int n = 0, m = 0;
      bool ok = true;
      int w = blockIdx.x;
      Unit un = {};
      if (sg.plan && w < items) un = sg.plan[w / per];
      auto advance = [&] {  // the item after this one, by lane 0
        w = INT_MAX;
        if (sg.plan) {
          w = gridDim.x + static_cast<int>(atomicAdd(sg.queue, 1u));
          if (w < items) un = sg.plan[w / per];
        }
      };
      auto share = [&] {
        w = __shfl_sync(0xffffffffu, w, 0);
        un.t0 = __shfl_sync(0xffffffffu, un.t0, 0);
        un.t1 = __shfl_sync(0xffffffffu, un.t1, 0);
        un.u = __shfl_sync(0xffffffffu, un.u, 0);
        un.row = __shfl_sync(0xffffffffu, un.row, 0);
      };
      for (int k = 0; ok; ++k) {
        Item it;
        bool found = w < items;
        if (found) {
          if (!sg.plan) {  // the only item of this CTA
            const int u = w / per;
            packed_range(p.cu, u, p.total, &un.t0, &un.t1);
            int slot = -1;
            if (p.S_in || p.S_out) {
              slot = p.slots ? __ldg(p.slots + u) : u;
              if (slot < 0 || slot >= p.n_slots) slot = -1;
              int taken = 0;
              if (p.slots && slot >= 0)
                for (int j = lane; j < u; j += 32) taken |= __ldg(p.slots + j) == slot;
              if (__any_sync(0xffffffffu, taken)) slot = -1;
            }
            un.u = u;
            un.row = 4 * slot + 3;
          }
          it.t0 = un.t0;
          it.t1 = un.t1;
          it.chunks = chunks_of(un.t1 - un.t0);
          it.v0 = w % vtiles * 64;
          it.h = w / vtiles % p.H;
          it.u = un.u;
          it.slot = un.row >> 2;
          it.whole = un.row >> 1 & 1;
          it.leaves = un.row & 1;
        }
        if (!found) it.chunks = -1;
        int go = 1;
        if (lane == 0) {
          // the state that the item starts from, into L2: its reader comes to it between two items
          if (found && !STATE && (!it.whole || (p.S_in && it.slot >= 0)) && it.v0 == 0)
            bulk_prefetch_l2((!it.whole ? sg.in + (size_t)it.u * p.H * p.sized : p.S_in + (size_t)it.slot * p.H * p.sized) +
                                 (size_t)it.h * p.sized, p.sized * 4);
          go = wait(&e_free[k & (kRing - 1)], k / kRing ^ 1);
          if (go) {
            ring[k & (kRing - 1)] = it;
            mbar_arrive(&e_full[k & (kRing - 1)]);
          }
        }
        ok = __shfl_sync(0xffffffffu, go, 0) && found;
        if (ok && it.chunks > 0) {  // the table of the item's head
          if (lane == 0) go = wait(&t_free[m & 1], (m >> 1) ^ 1);
          ok = __shfl_sync(0xffffffffu, go, 0);
          if (!ok) break;
          const float g = p.g ? __ldg(p.g + it.h) : 0.f;
#pragma unroll 4
          for (int at = lane; at < 256; at += 32) {
            const int e = at == 255 ? kN : p.reverse ? 127 - at : at - 127;
            tables[256 * (m & 1) + at] = e >= 0 ? decay_power(g, e) : 0.f;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&t_full[m & 1]);
          ++m;
        }
        if (lane == 0 && ok) {
          const int xh = it.h / p.rx, yh = it.h / p.ry, zh = it.h / p.rz, first = n;
          for (; n < first + it.chunks; ++n) {
            const int j = n - first, t = it.t0 + chunk_at(it, j) * kN, st = n & 1;
            const uint32_t again = (n >> 1) ^ 1;
            // Z first: it is the first to be free (behind P Z) and the first to be used (Z')
            if (!wait(&z_free[st], again)) break;
            mbar_arrive_expect_tx(&z_full[st], kTile);
            tma_load_3d(sm + kSmZ + st * kTile, &tm_z, &z_full[st], it.v0, zh, t);
            if (!wait(&xy_free[st], again)) {
              ++n;  // Z of this chunk is on its way
              break;
            }
            mbar_arrive_expect_tx(&xy_full[st], DA / 64 * kTile * (STATE ? 1 : 2));
#pragma unroll
            for (int c = 0; c < DA / 64; ++c) {
              tma_load_3d(sm + kSmY + (2 * st + c) * kTile, &tm_y, &xy_full[st], 64 * c, yh, t);
              if (!STATE) tma_load_3d(sm + kSmX + (2 * st + c) * kTile, &tm_x, &xy_full[st], 64 * c, xh, t);
            }
            if (j == 0) advance();  // under the first chunk's loads
            // the chunk after the next into L2; its loads wait for this chunk's products. X and Y
            // are read by both CTAs of a head of 128 value columns: one of them asks for each
            if (j + 2 < it.chunks) {
              const int t2 = it.t0 + chunk_at(it, j + 2) * kN;
              tma_prefetch_3d(&tm_z, it.v0, zh, t2);
#pragma unroll
              for (int c = 0; c < DA / 64; ++c) {
                if (vtiles == 1 || it.v0 == 0) tma_prefetch_3d(&tm_y, 64 * c, yh, t2);
                if (!STATE && (vtiles == 1 || it.v0 != 0)) tma_prefetch_3d(&tm_x, 64 * c, xh, t2);
              }
            }
          }
        }
        if (lane == 0 && ok && it.chunks == 0) advance();
        share();
      }
      // given up: copies still in flight must land before the CTA's memory is released
      // (a barrier that was never armed in its last phase just runs out its wait)
      if (lane == 0 && *abort_flag)
        for (int i = n; i >= 0 && i >= n - 2; --i) {
          (void)mbar_wait_bounded(&xy_full[i & 1], (i >> 1) & 1, 1u << 16);
          (void)mbar_wait_bounded(&z_full[i & 1], (i >> 1) & 1, 1u << 16);
        }
    } else if (!STATE && warp == 2 && lane == 0) {
      // -------------------------------------------------------- MMAs: scores
      constexpr uint32_t id_sc = idesc_bf16_f32(128, 128, false, false);
      const uint32_t dx = smem_u32(sm + kSmX), dy = smem_u32(sm + kSmY);
      bool ok = true;
      for (int k = 0, n = 0; ok && wait(LA_ITEM_FULL(k)); ++k) {
        const int chunks = item_at(k).chunks;
        if (chunks < 0) break;
        for (int j = 0; j < chunks; ++j, ++n) {
          const int st = n & 1;
          const uint32_t stage = 2 * st * kTile;
          ok = wait(&xy_full[st], n >> 1) && wait(&o_free[st], (n >> 1) ^ 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 4
          for (int c = 0; c < DA / 16; ++c) {
            const uint32_t off = stage + (c >> 2) * kTile + (c & 3) * 32;
            mma_bf16(tbase + kColSc + 128 * st, desc(dx + off, 16), desc(dy + off, 16), id_sc, c > 0);
          }
          mma_commit(&sc_full[st]);
          mma_commit(&xy_free[st]);
        }
        mbar_arrive(&e_free[k & (kRing - 1)]);
      }
      mma_commit(&drain[2]);
      (void)mbar_wait_bounded(&drain[2], 0, kSpin);
    } else if (warp == 1 && lane == 0) {
      // ------------------------------------------------------- MMAs: dS, X S
      constexpr uint32_t id_d = idesc_bf16_f32(128, 128, true, true), id_o = idesc_bf16_f32(128, 64, false, true);
      const uint32_t dx = smem_u32(sm + kSmX), dyt = smem_u32(sm + kSmY), dw = smem_u32(sm + kSmW);
      const uint32_t ds = smem_u32(sm + kSmS);
      bool ok = true;
      for (int k = 0, n = 0; ok && wait(LA_ITEM_FULL(k)); ++k) {
        const int chunks = item_at(k).chunks;
        if (chunks < 0) break;
        for (int j = 0; j < chunks; ++j, ++n) {
          const int st = n & 1;
          ok = wait(&xy_full[st], n >> 1) && wait(d_free, n ^ 1) && wait(&w_ready[st], n >> 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 4
          for (int c = 0; c < kN / 16; ++c)
            mma_bf16(tbase + kColD, desc(dyt + 2 * st * kTile + c * 2048, kTile), desc(dw + c * 2048, kTile), id_d,
                     c > 0);
          mma_commit(d_full);
          mma_commit(&z_free[st]);
          if (!STATE) {  // in the time that the next Z' takes
            ok = wait(&o_free[st], (n >> 1) ^ 1) && wait(s_ready, n);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 4
            for (int c = 0; c < DA / 16; ++c)
              mma_bf16(tbase + kColXS + 64 * st, desc(dx + 2 * st * kTile + (c >> 2) * kTile + (c & 3) * 32, 16),
                       desc(ds + c * 2048, kTile), id_o, c > 0);
            mma_commit(xs_full);
            mma_commit(&o_full[st]);
          }
          mma_commit(&xy_free[st]);
        }
        mbar_arrive(&e_free[k & (kRing - 1)]);
      }
      mma_commit(&drain[0]);
      (void)mbar_wait_bounded(&drain[0], 0, kSpin);
    } else if (!STATE && warp == 3 && lane == 0) {
      // ----------------------------------------------------------- MMAs: P Z
      constexpr uint32_t id_o = idesc_bf16_f32(128, 64, false, true);
      const uint32_t dz = smem_u32(sm + kSmZ);
      bool ok = true;
      for (int k = 0, n = 0; ok && wait(LA_ITEM_FULL(k)); ++k) {
        const int chunks = item_at(k).chunks;
        if (chunks < 0) break;
        for (int j = 0; j < chunks; ++j, ++n) {
          const int st = n & 1;
          // (behind Z', Z is there and its foreign rows are clear)
          ok = wait(&w_ready[st], n >> 1) && wait(&p_ready[st], n >> 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 4
          for (int c = 0; c < kN / 16; ++c)  // blocks of 32 tokens of P in the order 0, 3, 1, 2
            mma_bf16_ts(tbase + kColSc + 128 * st + kColPZ,
                        tbase + kColSc + 128 * st + (0x1320u >> (c & 6) * 2 & 0xf) * 16 + (c & 1) * 8,
                        desc(dz + st * kTile + c * 2048, kTile), id_o, c > 0);
          mma_commit(&o_full[st]);
          mma_commit(&z_free[st]);
        }
        mbar_arrive(&e_free[k & (kRing - 1)]);
      }
      mma_commit(&drain[1]);
      (void)mbar_wait_bounded(&drain[1], 0, kSpin);
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------- the state
    regs_up<kRegsState>();
    const int c = wq * 32 + lane;  // key channel: row of S
    bool ok = true;
    for (int k = 0, n = 0; ok && wait_group(LA_ITEM_FULL(k)); ++k) {
      const Item it = item_at(k);
      if (it.chunks < 0) break;
      const size_t by_unit = ((size_t)it.u * p.H + it.h) * p.sized, by_slot = ((size_t)it.slot * p.H + it.h) * p.sized;
      const float *src = nullptr;
      float *dst = nullptr;
      if (STATE) {
        dst = sg.out + by_unit;
      } else {
        if (!it.whole) src = sg.in + by_unit;
        else if (p.S_in && it.slot >= 0) src = p.S_in + by_slot;
        if (p.S_out && it.leaves && it.slot >= 0) dst = p.S_out + by_slot;
      }
      float S[64];
      if (src && c < DA) {
        if (p.in_t && it.whole) {  // (the segments' states lie as this pass wants them)
#pragma unroll
          for (int e = 0; e < 64; ++e) S[e] = src[(size_t)(it.v0 + e) * DA + c];
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float4 t = reinterpret_cast<const float4 *>(src + (size_t)c * db + it.v0)[e];
            S[4 * e] = t.x; S[4 * e + 1] = t.y; S[4 * e + 2] = t.z; S[4 * e + 3] = t.w;
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 64; ++e) S[e] = 0.f;
      }
      const float g = p.g ? __ldg(p.g + it.h) : 0.f;
      const Decay whole(g, kN), part(g, it.t1 - it.t0 - (it.chunks - 1) * kN);
      for (int j = 0; j < it.chunks; ++j, ++n) {
        if (!STATE) {  // row c of the bf16 copy, once X S of the chunk before is done with it
          ok = n == 0 || wait_group(xs_full, n - 1);
          if (!ok) break;
          if (c < DA) {
#pragma unroll
            for (int q = 0; q < 8; ++q) *reinterpret_cast<uint4 *>(sm + kSmS + sw128_off(c, 8 * q)) = pack8(S + 8 * q);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_ready);
        }
        ok = wait_group(d_full, n);
        if (!ok) break;
        tc_fence_after();
        const Decay decay = chunk_at(it, j) == it.chunks - 1 ? part : whole;
        // S m (+ S): see Decay
        const uint64_t small = pair(decay.m, decay.m), one = decay.near ? pair(1.f, 1.f) : 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          float d[8], lo[8];
          tmem_ld8(tl + kColD + 8 * q, d);
          tmem_ld8(tl + kColD + 64 + 8 * q, lo);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            add2(d + e, d + e, lo + e);
            fma2(d + e, S + 8 * q + e, small, d + e);
            fma2(S + 8 * q + e, S + 8 * q + e, one, d + e);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_free);
      }
      if (ok && dst && c < DA) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          reinterpret_cast<float4 *>(dst + (size_t)c * db + it.v0)[e] =
              make_float4(S[4 * e], S[4 * e + 1], S[4 * e + 2], S[4 * e + 3]);
      }
      item_done(k);
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ the output
    regs_up<kRegsOut>();
    const int i = wq * 32 + lane;
    uint8_t *ot = sm + kSmO;
    bool ok = !STATE;
    for (int k = 0, n = 0, m = 0; ok && wait_group(LA_ITEM_FULL(k)); ++k) {
      const Item it = item_at(k);
      if (it.chunks < 0) break;
      const float *tab = tables + 256 * (m & 1);
      if (it.chunks > 0 && !wait_group(&t_full[m & 1], m >> 1)) break;
      for (int j = 0; j < it.chunks; ++j, ++n) {
        const int cc = chunk_at(it, j), st = n & 1, rows = min(kN, it.t1 - it.t0 - cc * kN), t = it.t0 + cc * kN + i;
        // gamma^(i+1), reversed gamma^(rows-1-i)
        const float r = tab[p.reverse ? 127 - max(rows - 1 - i, 0) : 128 + i];
        const uint64_t rr = pair(r, r);
        const bool staged = wq * 32 + 32 <= rows;  // all of the warp's rows: through TMA
        const size_t at = (size_t)t * p.ldo + (size_t)it.h * db + it.v0;
        if (n > 0 && lane == 0) bulk_wait_read<0>();  // the staging rows have been read
        ok = wait_group(&o_full[st], n >> 1);
        if (!ok) break;
        tc_fence_after();
        uint4 o[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float xs[16], pz[16];
          tmem_ld16(tl + kColXS + 64 * st + 16 * q, xs);
          tmem_ld16(tl + kColSc + 128 * st + kColPZ + 16 * q, pz);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e += 2) fma2(xs + e, xs + e, rr, pz + e);
          if constexpr (OF32) {  // 32 columns at a time: a row of the staging tile
            uint8_t *to = staged ? ot : reinterpret_cast<uint8_t *>(static_cast<float *>(p.out) + at + 32 * (q >> 1));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int c = 4 * (q & 1) + e;  // 16 bytes of the row
              if (i < rows)
                *reinterpret_cast<float4 *>(to + (staged ? sw128_off(i, 8 * c) : 16u * c)) =
                    make_float4(xs[4 * e], xs[4 * e + 1], xs[4 * e + 2], xs[4 * e + 3]);
            }
            if (q & 1) {
              if (staged) fence_proxy_async();
              __syncwarp();
              if (staged && lane == 0) {
                tma_store_3d(&tm_o, ot + wq * 32 * 128, it.v0 + 16 * (q - 1), it.h, t);
                bulk_commit();
                if (q == 1) bulk_wait_read<0>();
              }
              __syncwarp();
            }
          } else {
            o[2 * q] = pack8(xs);
            o[2 * q + 1] = pack8(xs + 8);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[st]);
        if constexpr (!OF32) {
          // the staging tile, or straight to memory
          uint8_t *to = staged ? ot : reinterpret_cast<uint8_t *>(static_cast<__nv_bfloat16 *>(p.out) + at);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (i < rows) *reinterpret_cast<uint4 *>(to + (staged ? sw128_off(i, 8 * q) : 16u * q)) = o[q];
          if (staged) fence_proxy_async();
          __syncwarp();
          if (staged && lane == 0) {
            tma_store_3d(&tm_o, ot + wq * 32 * 128, it.v0, it.h, t);
            bulk_commit();
          }
        }
      }
      if (it.chunks > 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&t_free[m & 1]);
        ++m;
      }
      item_done(k);
    }
    if (!STATE && lane == 0) bulk_wait<0>();
  } else if (warp < 20) {
    // -------------------------------------------------------- Z' high and low
    regs_down<kRegsZ>();
    const int half = (warp - 12) >> 2, i = wq * 32 + lane;  // columns 32*half .. of row i
    bool ok = true;
    for (int k = 0, n = 0, m = 0; ok && wait_group(LA_ITEM_FULL(k)); ++k) {
      const Item it = item_at(k);
      if (it.chunks < 0) break;
      const float *tab = tables + 256 * (m & 1);
      if (it.chunks > 0) {
        if (!wait_group(&t_full[m & 1], m >> 1)) break;
      }
      for (int j = 0; j < it.chunks; ++j, ++n) {
        const int cc = chunk_at(it, j), st = n & 1, rows = min(kN, it.t1 - it.t0 - cc * kN);
        const bool mine = i < rows;
        ok = wait_group(&z_full[st], n >> 1);
        if (!ok) break;
        uint8_t *zt = sm + kSmZ + st * kTile, *wt = sm + kSmW;
        if (!mine)  // foreign rows of Z
#pragma unroll 1
          for (int q = 4 * half; q < 4 * half + 4; ++q)
            *reinterpret_cast<uint4 *>(zt + sw128_off(i, 8 * q)) = make_uint4(0, 0, 0, 0);
        // gamma^(rows-1-j), reversed gamma^(j+1)
        const float w = mine ? tab[p.reverse ? (i == 127 ? 255 : 126 - i) : 126 + rows - i] : 0.f;
        const uint64_t ww = pair(w, w), minus = pair(-1.f, -1.f);
        uint4 hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) hi[e] = *reinterpret_cast<const uint4 *>(zt + sw128_off(i, 8 * (4 * half + e)));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float f[8], f2[8];
          unpack8(hi[e], f);
#pragma unroll
          for (int c = 0; c < 8; c += 2) mul2(f + c, f + c, ww);
          hi[e] = pack8(f);
          unpack8(hi[e], f2);
#pragma unroll
          for (int c = 0; c < 8; c += 2) fma2(f + c, f2 + c, minus, f + c);
          lo[e] = pack8(f);
        }
        // the buffer itself is free once the dS before has been formed
        ok = n == 0 || wait_group(d_full, n - 1);
        if (!ok) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          *reinterpret_cast<uint4 *>(wt + sw128_off(i, 8 * (4 * half + e))) = hi[e];
          *reinterpret_cast<uint4 *>(wt + kTile + sw128_off(i, 8 * (4 * half + e))) = lo[e];
        }
        if (rows < kN) {  // foreign rows of Y, once their scores are formed
          ok = wait_group(&xy_full[st], n >> 1) && (STATE || wait_group(&sc_full[st], n >> 1));
          if (!ok) break;
          if (!mine)
#pragma unroll 1
            for (int q = half; q < DA / 8; q += 2)
              *reinterpret_cast<uint4 *>(sm + kSmY + (2 * st + (q >> 3)) * kTile + sw128_off(i, 8 * (q & 7))) =
                  make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&w_ready[st]);
      }
      if (it.chunks > 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&t_free[m & 1]);
        ++m;
      }
      item_done(k);
    }
  } else {
    // ------------------------------------------------------------------- P
    const int half = (warp - 20) >> 2, i = wq * 32 + lane;
    bool ok = !STATE;
    for (int k = 0, n = 0, m = 0; ok && wait_group(LA_ITEM_FULL(k)); ++k) {
      const Item it = item_at(k);
      const int chunks = it.chunks;
      if (chunks < 0) break;
      const float *tab = tables + 256 * (m & 1) + 127 + i;
      if (chunks > 0 && !wait_group(&t_full[m & 1], m >> 1)) break;
      for (int j = 0; j < chunks; ++j, ++n) {
        const int st = n & 1, rows = it.t1 - it.t0 - chunk_at(it, j) * kN;
        ok = wait_group(&sc_full[st], n >> 1);
        if (!ok) break;
        tc_fence_after();
        // blocks of 32 columns against the warp's 32 rows
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          const int kb = half ? 1 + c : 3 * c, j0 = 32 * kb;  // half 0: the first and the last block
          const uint32_t sc = tl + kColSc + 128 * st + j0, pt = tl + kColSc + 128 * st + 32 * half + 16 * c;
          float f[32];
          if (p.reverse ? kb < wq : kb > wq) {  // nothing of the block is seen
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = 0.f;
          } else {
            tmem_ld32(sc, f);
            tmem_wait_ld();
            // Tokens that do not see each other have the factor zero, and a score that may be infinite
            // where all that is asked for is finite: it must not make a NaN of it. (4 x 16384 tokens:
            // 237 us without, 244 so, 246 by selection, 252 by selection where a NaN came up.)
            if (kb == wq)
#pragma unroll
              for (int e = 0; e < 32; ++e) f[e] = finite(f[e]);
            const float *at = tab - j0;
#pragma unroll
            for (int e = 0; e < 16; ++e) mul2(f + 2 * e, f + 2 * e, pair(at[-2 * e], at[-2 * e - 1]));
            if (j0 + 32 > rows) {  // foreign columns, by selection: their scores may be anything
#pragma unroll
              for (int e = 0; e < 32; ++e) f[e] = j0 + e < rows ? f[e] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              f[e] = __uint_as_float(pack_bf16(f[2 * e], f[2 * e + 1]));
            }
          }
          tmem_st16(pt, f);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[st]);
      }
      if (chunks > 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&t_free[m & 1]);
        ++m;
      }
      item_done(k);
    }
  }
#undef LA_ITEM_FULL
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tbase, 512);
  if (tid == 0) {
    if (*abort_flag) atomicOr(p.status, kStatusTimeout);
    // behind an independent pass that this one may have run beside: not done before it is
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
}

// The entering state of every segment from the segments' own contributions, in
// place: a running sum per element, the loads of a few segments ahead in flight.
__global__ void __launch_bounds__(256) segment_scan_kernel(const PackedPass p, int seg, const Split *splits,
                                                           const int *count, float *ws) {
  const int h = blockIdx.y, e = (blockIdx.x * 256 + threadIdx.x) * 4;
  const int split = *count;
  const Split sp = splits[blockIdx.z];  // (the grid is within the list's room)
  if (static_cast<int>(blockIdx.z) >= split || e >= p.sized) return;
  const int a = sp.a, b = sp.b, slot = sp.row, n = (b - a + seg - 1) / seg, u0 = sp.u;
  const float g = p.g ? __ldg(p.g + h) : 0.f;
  float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.S_in && slot >= 0) {
    const float *in = p.S_in + ((size_t)slot * p.H + h) * p.sized;
    const int c = e / p.db, v = e % p.db;
    if (p.in_t) S = make_float4(in[(size_t)v * p.da + c], in[(size_t)(v + 1) * p.da + c], in[(size_t)(v + 2) * p.da + c],
                                in[(size_t)(v + 3) * p.da + c]);
    else S = *reinterpret_cast<const float4 *>(in + e);
  }
  auto at = [&](int k) {
    return reinterpret_cast<float4 *>(ws + ((size_t)(u0 + (p.reverse ? n - 1 - k : k)) * p.H + h) * p.sized + e);
  };
  const Decay whole(g, seg), part(g, b - a - (n - 1) * seg);
  constexpr int kAhead = 4;
  for (int k0 = 0; k0 < n; k0 += kAhead) {
    float4 U[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (k0 + i < n - 1) U[i] = *at(k0 + i);  // nothing reads behind the last segment
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = k0 + i;
      if (k >= n) break;
      *at(k) = S;
      if (k == n - 1) break;
      const bool tail = (p.reverse ? n - 1 - k : k) == n - 1;
      S.x = (tail ? part(S.x) : whole(S.x)) + U[i].x;
      S.y = (tail ? part(S.y) : whole(S.y)) + U[i].y;
      S.z = (tail ? part(S.z) : whole(S.z)) + U[i].z;
      S.w = (tail ? part(S.w) : whole(S.w)) + U[i].w;
    }
  }
}

// [tokens][heads][d] with a token stride, boxes of 128 bytes of channels x 1 head x rows.
bool make_token_map(CUtensorMap *m, const void *base, bool f32, int d, int heads, int tokens, long long ld, int rows) {
  const cuuint64_t e = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d * e, (cuuint64_t)ld * e};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / e), 1, (cuuint32_t)rows}, es[3] = {1, 1, 1};
  return g_encode(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                  const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
  CUtensorMap x, y, z, o;
};

template <int DA, bool STATE, bool OF32>
cudaError_t launch_as(const PackedPass &p, const Segments &sg, const Maps &m, bool beside, cudaStream_t stream) {
  auto kernel = packed_tc_kernel<DA, STATE, OF32>;
  // once for each device
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) done[dev].store(true, std::memory_order_release);
  }
  const long long items = (long long)sg.units * p.H * (p.db / 64);
  const int grid = static_cast<int>(std::min<long long>(items, std::max(1, sm_count())));
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmBytes;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = beside ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p, sg, m.x, m.y, m.z, m.o);
}

template <bool STATE>
cudaError_t launch(const PackedPass &p, const Segments &sg, const Maps &m, bool beside, cudaStream_t stream) {
  if constexpr (!STATE)
    if (p.out_f32)
      return p.da == 64 ? launch_as<64, false, true>(p, sg, m, beside, stream) : launch_as<128, false, true>(p, sg, m, beside, stream);
  return p.da == 64 ? launch_as<64, STATE, false>(p, sg, m, beside, stream) : launch_as<128, STATE, false>(p, sg, m, beside, stream);
}

// What a split costs: a factor on the pass, and for each pass its further launches, in tokens of a
// walk. Measured (microseconds, unsplit / split, one sequence of T tokens, 8 heads of 128): forward
// T = 2048 36 / 40, 3000 50 / 42, 4096 62 / 46, 8192 115 / 57; 2 x 4096 tokens of 16 heads 69 / 88.
// Backward T = 4096 65 / 106, 8192 122 / 135: its passes overlap, and fill the GPU without a split.
constexpr double kSplitCost = 1.6;
constexpr int kSplitTokens = 16 * kN;

int fail(const char *what, cudaError_t e) {
  set_error("packed retention: %s: %s", what, cudaGetErrorString(e));
  return LA_ERR_CUDA;
}

// One pass with what it is launched with.
struct Ready {
  Maps m;
  Segments sg;
  int most;                     // segments with a state to form
  size_t owners, plan, lists, states;  // bytes of its workspace behind 256 of counters; plan 0: none
};

// Maps, split and workspace of a pass, of passes with `share` tokens for each SM
// together; an LA_ERR_* code where it cannot run.
int make_ready(const PackedPass &p, int passes, long long share, Ready *r) {
  if (!make_token_map(&r->m.x, p.x, false, p.da, p.H / p.rx, p.total, p.ldx, kN) ||
      !make_token_map(&r->m.y, p.y, false, p.da, p.H / p.ry, p.total, p.ldy, kN) ||
      !make_token_map(&r->m.z, p.z, false, p.db, p.H / p.rz, p.total, p.ldz, kN)) {
    set_error("packed retention: tensor map encoding failed");
    return LA_ERR_CUDA;
  }
  if (!make_token_map(&r->m.o, p.out, p.out_f32, p.db, p.H, p.total, p.ldo, 32)) {
    set_error("packed retention: tensor map encoding failed");
    return LA_ERR_CUDA;
  }
  // Sequences are split into segments where whole ones would leave the GPU to a
  // few long walks. Unsplit the passes take as long as the longest sequence or
  // their share of the whole; split they take that share, and on top the second
  // reading of Y and Z, the states' way through memory and two more launches.
  const long long sms = std::max(1, sm_count());
  const int longest = p.max_len > 0 ? std::min(p.max_len, p.total) : p.total;
  r->sg = {0, p.n_seq, nullptr, nullptr, nullptr, nullptr, nullptr};
  if (longest > kSplitCost * share + kSplitTokens * passes) {
    const long long own = ((long long)p.total * p.H * (p.db / 64) + sms - 1) / sms;
    const long long seg = std::max<long long>((own + kN - 1) / kN * kN, 2 * kN);
    if (seg < longest) {
      r->sg.tokens = static_cast<int>(seg);
      r->sg.units = static_cast<int>(p.total / seg) + p.n_seq;
    }
  }
  const long long items = (long long)r->sg.units * p.H * (p.db / 64);
  if (items > INT_MAX / 2) {
    set_error("packed retention: n_seq * H too large");
    return LA_ERR_INVALID_ARG;
  }
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  r->most = r->sg.tokens ? p.total / r->sg.tokens : 0;
  r->owners = r->plan = r->lists = r->states = 0;
  if (items > sms || r->sg.tokens) {
    r->owners = up(p.slots && (p.S_in || p.S_out) ? (size_t)p.n_slots * 4 : 0);
    r->plan = up((size_t)r->sg.units * sizeof(Unit));
    r->lists = up((size_t)r->most * (sizeof(Unit) + sizeof(Split)));
    r->states = (size_t)2 * r->most * p.H * p.sized * 4;
  }
  return LA_OK;
}

}  // namespace

// The passes do not depend on each other. Each phase of all of them is launched
// back to back, and the tensor-core kernels behind the first may begin before the
// one in front of them is done (programmatic launch): the SMs that its queue has
// no more work for take the next pass's, instead of waiting for its last items.
int launch_packed_tc(const PackedPass *p, int passes, cudaStream_t stream) {
  if (!encode_fn()) {
    set_error("packed retention: cuTensorMapEncodeTiled is unavailable");
    return LA_ERR_CUDA;
  }
  Ready r[3];
  size_t bytes = 0;
  long long share = 0;
  for (int i = 0; i < passes; ++i) share += (long long)p[i].total * p[i].H * (p[i].db / 64);
  share /= std::max(1, sm_count());
  for (int i = 0; i < passes; ++i) {
    const int rc = make_ready(p[i], passes, share, &r[i]);
    if (rc != LA_OK) return rc;
    if (r[i].plan) bytes += 256 + r[i].owners + r[i].plan + r[i].lists + r[i].states;
  }
  uint8_t *ws = nullptr;
  cudaError_t e = cudaSuccess;
  if (bytes) {
    cudaMemPool_t pool = library_pool();
    if (!pool) return fail("could not create the workspace pool", cudaGetLastError());
    e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), bytes, pool, stream);
    if (e != cudaSuccess) return fail("workspace allocation failed", e);
  }
  // counters, owners of the state rows, plan, lists of split sequences and their segments, states of each pass
  uint8_t *at = ws;
  PlanJobs jobs = {};
  Segments state[3];
  const Split *splits[3] = {};
  const int *split_count[3] = {};
  int planned = 0;
  for (int i = 0; i < passes; ++i) {
    if (!r[i].plan) continue;
    unsigned *head = reinterpret_cast<unsigned *>(at);
    uint8_t *behind = at + 256 + r[i].owners;
    Unit *plan = reinterpret_cast<Unit *>(behind), *segments = reinterpret_cast<Unit *>(behind + r[i].plan);
    Split *split = reinterpret_cast<Split *>(segments + r[i].most);
    const int *counts = reinterpret_cast<const int *>(head);
    jobs.job[planned++] = {p[i], r[i].sg.tokens, r[i].sg.units, r[i].most, head, reinterpret_cast<int *>(at + 256),
                           plan, segments, split};
    if (r[i].sg.tokens) {
      float *states = reinterpret_cast<float *>(behind + r[i].plan + r[i].lists);
      state[i] = {r[i].sg.tokens, r[i].most, segments, counts + kSegmentCount, head + kStateQueue, nullptr, states};
      r[i].sg.in = states;
      splits[i] = split;
      split_count[i] = counts + kSplitCount;
    }
    r[i].sg.plan = plan;
    r[i].sg.count = counts + kUnitCount;
    r[i].sg.queue = head + kMainQueue;
    at += 256 + r[i].owners + r[i].plan + r[i].lists + r[i].states;
  }
  if (planned) {
    plan_kernel<<<planned, kPlanThreads, 0, stream>>>(jobs);
    e = cudaGetLastError();
  }
  bool beside = false;
  for (int i = 0; i < passes && e == cudaSuccess; ++i) {
    if (!r[i].sg.tokens) continue;
    e = launch<true>(p[i], state[i], r[i].m, beside, stream);
    beside = true;
  }
  for (int i = 0; i < passes && e == cudaSuccess; ++i) {
    if (!r[i].sg.tokens) continue;
    // (most is below 64 SMs / (H db): a segment is at least a SM's share of all items)
    segment_scan_kernel<<<dim3((p[i].sized / 4 + 255) / 256, p[i].H, std::min(r[i].most, p[i].n_seq)), 256, 0, stream>>>(
        p[i], r[i].sg.tokens, splits[i], split_count[i], state[i].out);
    e = cudaGetLastError();
  }
  for (int i = 0; i < passes && e == cudaSuccess; ++i) e = launch<false>(p[i], r[i].sg, r[i].m, i > 0, stream);
  if (ws) {
    const cudaError_t f = cudaFreeAsync(ws, stream);
    if (e == cudaSuccess) e = f;
  }
  return e == cudaSuccess ? LA_OK : fail("launch failed", e);
}

}  // namespace la
