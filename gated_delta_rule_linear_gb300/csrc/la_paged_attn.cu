// Attention of one new token of each sequence over a paged cache:
// o_h = sum_p softmax_p(scale q_h . k_p) v_p, in one pass over the places with a
// running maximum and sum (Milakov and Gimelshein, 2018).
//
// Bound by reading keys and values once. The heads that share a key/value head
// are the rows of one block of up to 8 or 16 (a `part` of a sequence), so that a
// place is read once for all of a block. More heads than that (16, float32: 8) are
// several blocks, and each reads the places again (32 x 8192, bfloat16, 32/1 heads
// of 128: 48 us, 16/1 31).
//
// Work. The places of a part are cut into units, a block of keys for each of the
// CTA's four warps; the units of all parts, one after the other, are dealt to the
// CTAs in equal runs, however long the sequences are (each CTA adds up the lengths
// for itself: nothing is known on the host). A CTA's run begins and ends inside a
// part: what it has of that goes to a workspace, and join_kernel adds the pieces
// up. Every other part is finished where it was begun.
//
// A warp streams its blocks through two stages of shared memory by 16-byte
// asynchronous copies, across the ends of parts, with no barrier but its own; the
// CTA's warps meet at the end of a part only, two handing their sums to the other
// two.
//
// bfloat16: S = Q K^T and O = P V by 16 x 8 x 16 matrix instructions of a warp.
// With 8 or 16 rows the tensor cores have an eighth of a tile's work (112 of the
// 128 rows of a tcgen05 product would be empty), and the operands come straight from
// the 16-byte rows as they are stored: channels are taken in the order in which a
// thread holds them, for keys and queries alike. P keeps 16 bits as a high and a
// low bfloat16 part; with up to 8 heads the low part is in the tile's other 8 rows
// and costs nothing. float32: CUDA cores, see F32Warp.
//
// 64 sequences of 16384 places, 32/8 heads of 128, bfloat16: 608 to 629 us, 6.8 to
// 7.0 TB/s. Two of 131072, 16/2 heads: 50 us of 40; what is not reading is the
// launch, the way lengths -> table -> first keys (3.7 us) and the pieces' join (3
// us). 16 heads a block: 5.2 TB/s (32/2 heads of 128). Nothing is at its limit there
// (issue 36 %, tensor pipe 21 %): two warps a scheduler do not cover a block's chain
// of S, maximum and P V, whose low part is a second product. 8 heads in float32:
// instructions, 4.6 to 5.8 TB/s.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

#include "la_f32x2.cuh"
#include "la_serve_internal.h"
#include "la_sm100.cuh"

namespace la {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kJoinThreads = 512;

// Sizes of a kernel with d = D and HB rows.
template <typename T, int D, int HB> struct Shape {
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr int kKeys = !kF32 || D == 64 ? 16 : D == 256 && HB == 8 ? 4 : 8;  // places of a warp's block
  static constexpr int kChunks = D * static_cast<int>(sizeof(T)) / 16;    // 16-byte chunks of a row
  static constexpr int kTile = kKeys * kChunks * 16;                      // bytes of a block's keys
  static constexpr int kStage = 2 * kTile;
  // CTAs on a SM, of two stages each: 64 KB on their way are what the memory's latency asks for, and more of these copies
  // stand in the way of the warps' own reads of shared memory. (32 x 16384 places, 16/8 heads of 128: 2 CTAs of two
  // stages 314 us, 6.8 TB/s; of three stages 365, 3 CTAs of two 395. 64 x 8192, 16/8 heads of 64: 4 CTAs of two stages
  // 170 us, 3 181; 2 of three 242.)
  static constexpr int kCtas = D == 64 ? kF32 ? 3 : 4 : D == 128 || (kF32 && HB == 8) ? 2 : 1;  // on a SM
  static constexpr int kStages = 2;
  static constexpr int kUnit = kKeys * kWarps;
  static constexpr int kJoin = kWarps / 2 * HB * D * 4;         // half of the warps' sums, where they meet
  static constexpr int kBytes = kStages * kStage * kWarps + kJoin;
};

// What a part costs besides its units, in units: its queries, and the meeting of the warps at its end.
// (128 ragged sequences: 0 49.8 us, 1 43.4, 2 43.7.)
constexpr int kPartCost = 1;

// What the CTAs of a call share: rows of a part, pieces of parts in the workspace.
struct Split {
  int blocks;      // blocks of HB heads of a key/value head
  int parts;       // parts of a sequence: Hk * blocks
  int lines;       // 128-byte lines of a table row that are asked for ahead
  int whole;       // a CTA takes one whole part: no pieces, no workspace
  float *sums;     // [2 * CTAs][HB][D]
  float2 *ml;      // [2 * CTAs][HB]: maximum (of log2) and sum
  int4 *joins;     // sequence, part, first and last CTA with a piece of it; sequence -1: none
  int by_part;     // joins has an entry for each part of each sequence, else for the first CTA of each
};

constexpr int kMostPlaces = 0x7fff0000;  // a unit behind the last place is still an int

struct Range {
  int first, len;  // places of a sequence: first .. len - 1
  __device__ __forceinline__ int units(int keys, int unit) const {  // from the block of `keys` that holds the first
    return len > first ? (len - first / keys * keys + unit - 1) / unit : 0;
  }
};
__device__ __forceinline__ Range places_of(const PagedAttn &p, int s) {
  const long long most = min((long long)p.at.max_pages * p.at.page_size, (long long)kMostPlaces);
  const int len = static_cast<int>(min((long long)max(p.at.lens[s], 0), most));
  return {p.window > 0 ? max(len - p.window, 0) : 0, len};
}

// A unit in a CTA's run. All parts' units are numbered through, with kPartCost numbers left out in front of each part.
template <int KEYS, int UNIT> struct Cursor {
  int s, part, unit, units;
  Range at;
  int number;

  __device__ __forceinline__ void set(const PagedAttn &p) {
    at = places_of(p, s);
    units = at.units(KEYS, UNIT);
  }
  __device__ __forceinline__ void enter(const PagedAttn &p) {  // the next sequence with a place
    for (; s < p.n; ++s) {
      set(p);
      if (units > 0) return;
    }
  }
  __device__ __forceinline__ void next(const PagedAttn &p, int parts, int end) {
    ++number;
    if (++unit < units) return;
    unit = 0;
    number += kPartCost;
    if (++part < parts) return;
    part = 0;
    ++s;
    if (number < end) enter(p);
  }
};

// Maximum (of log2) and sum of two pieces, and what each is multiplied by.
__device__ __forceinline__ void meet(float &m, float &l, float m2, float l2, float &f, float &f2) {
  const float top = fmaxf(m, m2), base = top == -INFINITY ? 0.f : top;
  f = sm100::ex2(m - base);
  f2 = sm100::ex2(m2 - base);
  l = l * f + l2 * f2;
  m = top;
}
constexpr float kSlack = 8.f;  // log2 that a weight may exceed 1 by before sums are rescaled to a new maximum

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void wait_all_but() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// The 16-byte chunk that chunk c of row r is stored at, so that the reads below hit all banks.
template <bool F32, bool VALUES> __device__ __forceinline__ int stored(int r, int c) {
  if (F32) return c;
  return VALUES ? c ^ ((r >> 1 & 3) << 1) : c ^ ((r & 1) << 2);
}

// A warp's part of the softmax of up to HB heads, bfloat16. Thread (g, t) = (lane / 4, lane % 4) holds rows g and
// g + 8. Channels: the k-th pair of matrix instructions of S takes chunk 4 k + t of every row, thread t's 8 channels of
// it two instructions' fragments; O's tile 8 b + j has channel 64 b + 8 g + j in column g.
template <int D, int HB> struct Bf16Warp {
  static constexpr int R = HB / 8;  // rows of a thread
  uint32_t q[R][D / 32][4];
  float o[D / 8][4], m[R], l[R];
  float scale;

  __device__ __forceinline__ void begin(const PagedAttn &p, int s, int h0, int heads, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const __nv_bfloat16 *row = static_cast<const __nv_bfloat16 *>(p.q) + s * p.ldq + (long long)(h0 + g + 8 * r) * D;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (g + 8 * r < heads) u = reinterpret_cast<const uint4 *>(row)[4 * k + t];
        q[r][k][0] = u.x; q[r][k][1] = u.y; q[r][k][2] = u.z; q[r][k][3] = u.w;
      }
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    scale = p.scale * 1.44269504f;  // exponents of two
  }

  __device__ __forceinline__ void block(uint32_t keys, uint32_t values, uint32_t there, int lane, float *) {
    constexpr int kRow = D * 2;
    const int g = lane >> 2, t = lane & 3;
    float x[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float c[2][4] = {};  // the k steps alternate between two accumulators
      const int row = 8 * i + g;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const uint4 u = lds(keys + row * kRow + stored<false, false>(row, 4 * k + t) * 16);
        mma(c[0], q[0][k][0], q[R - 1][k][0], q[0][k][1], q[R - 1][k][1], u.x, u.y);
        mma(c[1], q[0][k][2], q[R - 1][k][2], q[0][k][3], q[R - 1][k][3], u.z, u.w);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[i][j] = there >> (8 * i + 2 * t + (j & 1)) & 1 ? (c[0][j] + c[1][j]) * scale : -INFINITY;
    }
    uint32_t hi[R][2], lo[R][2];
    float top[R];
    bool moved = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      top[r] = fmaxf(fmaxf(x[0][2 * r], x[0][2 * r + 1]), fmaxf(x[1][2 * r], x[1][2 * r + 1]));
      top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], 2));
      moved |= top[r] > m[r] + kSlack;
    }
    if (__any_sync(~0u, moved)) {
      float keep[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float now = fmaxf(m[r], top[r]);
        keep[r] = now == -INFINITY ? 1.f : sm100::ex2(m[r] - now);
        l[r] *= keep[r];
        m[r] = now;
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= keep[0]; o[i][1] *= keep[0];
        o[i][2] *= keep[R - 1]; o[i][3] *= keep[R - 1];
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float base = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float a = sm100::ex2(x[i][2 * r] - base), b = sm100::ex2(x[i][2 * r + 1] - base);
        l[r] += a + b;
        hi[r][i] = pack(a, b);
        lo[r][i] = pack(a - __uint_as_float(hi[r][i] << 16), b - __uint_as_float(hi[r][i] & 0xffff0000u));
      }
    }
#pragma unroll
    for (int b = 0; b < D / 64; ++b) {
      uint4 u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 2 * t + (i & 1) + 8 * (i >> 1);
        u[i] = lds(values + row * kRow + stored<false, true>(row, 8 * b + g) * 16);
      }
      const uint32_t v[4][4] = {{u[0].x, u[0].y, u[0].z, u[0].w}, {u[1].x, u[1].y, u[1].z, u[1].w},
                                {u[2].x, u[2].y, u[2].z, u[2].w}, {u[3].x, u[3].y, u[3].z, u[3].w}};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t b0 = __byte_perm(v[0][j / 2], v[1][j / 2], j & 1 ? 0x7632 : 0x5410);
        const uint32_t b1 = __byte_perm(v[2][j / 2], v[3][j / 2], j & 1 ? 0x7632 : 0x5410);
        float(&c)[4] = o[8 * b + j];
        if constexpr (R == 1) {
          mma(c, hi[0][0], lo[0][0], hi[0][1], lo[0][1], b0, b1);
        } else {
          mma(c, hi[0][0], hi[1][0], hi[0][1], hi[1][1], b0, b1);
          mma(c, lo[0][0], lo[1][0], lo[0][1], lo[1][1], b0, b1);
        }
      }
    }
  }

  // Rows without a head are left out at a part's end where rows are long (126 x 64 places, 32/32 heads of 256: 82 us with
  // them, 78 without; heads of 64: 25 and 26).
  static constexpr bool kSkip = D == 256;
  // The warp's sums to another warp, as they are held.
  static constexpr int kGiven = R;  // maxima and sums of a lane
  __device__ __forceinline__ void give(float *sums, float2 (*ml)[32], int lane, int heads) {
    if (kSkip && lane >> 2 >= heads) return;
#pragma unroll
    for (int r = 0; r < R; ++r) ml[r][lane] = make_float2(m[r], l[r]);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      if constexpr (R == 1) reinterpret_cast<float2 *>(sums)[i * 32 + lane] = make_float2(o[i][0] + o[i][2], o[i][1] + o[i][3]);
      else reinterpret_cast<float4 *>(sums)[i * 32 + lane] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
    }
  }
  __device__ __forceinline__ void take(const float *sums, const float2 (*ml)[32], int lane, int heads) {
    if (kSkip && lane >> 2 >= heads) return;
    float f[R], f2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) meet(m[r], l[r], ml[r][lane].x, ml[r][lane].y, f[r], f2[r]);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      if constexpr (R == 1) {
        const float2 a = reinterpret_cast<const float2 *>(sums)[i * 32 + lane];
        o[i][0] = fmaf(o[i][0] + o[i][2], f[0], a.x * f2[0]);
        o[i][1] = fmaf(o[i][1] + o[i][3], f[0], a.y * f2[0]);
        o[i][2] = o[i][3] = 0.f;
      } else {
        const float4 a = reinterpret_cast<const float4 *>(sums)[i * 32 + lane];
        o[i][0] = fmaf(o[i][0], f[0], a.x * f2[0]);
        o[i][1] = fmaf(o[i][1], f[0], a.y * f2[0]);
        o[i][2] = fmaf(o[i][2], f[R - 1], a.z * f2[R - 1]);
        o[i][3] = fmaf(o[i][3], f[R - 1], a.w * f2[R - 1]);
      }
    }
  }
  // The warp's sums into [HB][D] and [HB] of shared memory.
  __device__ __forceinline__ void end(float *sums, float2 *ml, int lane, int heads) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l[r] += __shfl_xor_sync(~0u, l[r], 1);
      l[r] += __shfl_xor_sync(~0u, l[r], 2);
      if (kSkip && g + 8 * r >= heads) continue;
      if (t == 0) ml[g + 8 * r] = make_float2(m[r], l[r]);
      float4 *row = reinterpret_cast<float4 *>(sums + (g + 8 * r) * D);
#pragma unroll
      for (int b = 0; b < D / 64; ++b)
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // 16 channels from 64 b + 16 t on: column 2t's 8, then 2t + 1's
          float f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float(&a)[4] = o[8 * b + 4 * (c & 1) + e];
            f[e] = R == 1 ? a[c >> 1] + a[2 + (c >> 1)] : a[2 * r + (c >> 1)];
          }
          row[16 * b + ((4 * t + c) ^ g)] = make_float4(f[0], f[1], f[2], f[3]);
        }
    }
  }
  // Where quad c of row g is in there.
  static __device__ __forceinline__ int quad(int g, int c) { return (c & ~15) + ((c & 15) ^ (g & 7)); }
};

// The same in float32 on the CUDA cores. A lane holds 4 (8) channels of all HB queries; a row of keys is spread over
// 32 lanes (two rows over 16 each), so that a lane has one partial product for each of 32 (16) pairs of key and
// head, and a butterfly that halves the pairs at each step leaves one whole score to each lane: lane % HB is its head.
template <int D, int HB> struct F32Warp {
  static constexpr int kKeys = Shape<float, D, HB>::kKeys;
  static constexpr int kLanes = D / 4 < 32 ? D / 4 : 32, kRows = 32 / kLanes;  // lanes of a row, rows at a time
  static constexpr int kPer = D / 4 / kLanes;                                  // quads of a lane
  static constexpr int kSteps = kLanes / HB, kGroup = kSteps * kRows;          // rows of a butterfly: one after another, all
  static constexpr int kGroups = kKeys / kGroup;
  static_assert(kGroups >= 1 && kGroups * kGroup == kKeys, "");
  float q[HB][kPer][4], o[HB][kPer][4], m, l, scale;

  __device__ __forceinline__ void begin(const PagedAttn &p, int s, int h0, int heads, int lane) {
    const float *src = static_cast<const float *>(p.q) + s * p.ldq + (long long)h0 * D;
#pragma unroll
    for (int h = 0; h < HB; ++h)
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        if (h < heads) a = reinterpret_cast<const float4 *>(src + h * D)[lane % kLanes + 32 * j];
        q[h][j][0] = a.x; q[h][j][1] = a.y; q[h][j][2] = a.z; q[h][j][3] = a.w;
        o[h][j][0] = o[h][j][1] = o[h][j][2] = o[h][j][3] = 0.f;
      }
    m = -INFINITY;
    l = 0.f;
    scale = p.scale * 1.44269504f;  // exponents of two
  }

  static __device__ __forceinline__ void row(uint32_t tile, int r, int lane, float (&v)[kPer][4]) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint4 u = lds(tile + (r * (D / 4) + lane % kLanes + 32 * j) * 16);
      v[j][0] = __uint_as_float(u.x); v[j][1] = __uint_as_float(u.y);
      v[j][2] = __uint_as_float(u.z); v[j][3] = __uint_as_float(u.w);
    }
  }

  __device__ __forceinline__ void block(uint32_t keys, uint32_t values, uint32_t there, int lane, float *weights) {
    const int half = lane / kLanes, step = lane % kLanes / HB, head = lane % HB;
    float x[kGroups], top = -INFINITY;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      float part[kLanes];
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        float v[kPer][4];
        row(keys, g * kGroup + k * kRows + half, lane, v);
#pragma unroll
        for (int h = 0; h < HB; ++h) {
          uint64_t t = f32x2::mul(f32x2::at(v[0]), f32x2::at(q[h][0]));
          t = f32x2::fma(f32x2::at(v[0] + 2), f32x2::at(q[h][0] + 2), t);
#pragma unroll
          for (int j = 1; j < kPer; ++j) {
            t = f32x2::fma(f32x2::at(v[j]), f32x2::at(q[h][j]), t);
            t = f32x2::fma(f32x2::at(v[j] + 2), f32x2::at(q[h][j] + 2), t);
          }
          float two[2];
          f32x2::split(t, two);
          part[k * HB + h] = two[0] + two[1];
        }
      }
#pragma unroll
      for (int d = kLanes / 2; d > 0; d /= 2)
#pragma unroll
        for (int i = 0; i < d; ++i) {
          const bool high = lane & d;
          const float keep = high ? part[i + d] : part[i], give = high ? part[i] : part[i + d];
          part[i] = keep + __shfl_xor_sync(~0u, give, d);
        }
      x[g] = there >> (g * kGroup + step * kRows + half) & 1 ? part[0] * scale : -INFINITY;
      top = fmaxf(top, x[g]);
    }
#pragma unroll
    for (int d = HB; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    if (__any_sync(~0u, top > m + kSlack)) {
      const float now = fmaxf(m, top), keep = now == -INFINITY ? 1.f : sm100::ex2(m - now);
#pragma unroll
      for (int h = 0; h < HB; ++h) {
        const float f = __shfl_sync(~0u, keep, h);
#pragma unroll
        for (int j = 0; j < kPer; ++j) f32x2::vmul(o[h][j], o[h][j], f);
      }
      m = now;
      l *= keep;
    }
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float w = sm100::ex2(x[g] - base);
      l += w;
      weights[(g * kGroup + step * kRows + half) * HB + head] = w;
    }
    __syncwarp();
#pragma unroll 4
    for (int k = 0; k < kKeys / kRows; ++k) {
      const int r = k * kRows + half;
      float w[HB], v[kPer][4];
#pragma unroll
      for (int h = 0; h < HB; h += 4) {
        const float4 a = *reinterpret_cast<const float4 *>(weights + r * HB + h);
        w[h] = a.x; w[h + 1] = a.y; w[h + 2] = a.z; w[h + 3] = a.w;
      }
      row(values, r, lane, v);
#pragma unroll
      for (int h = 0; h < HB; ++h)
#pragma unroll
        for (int j = 0; j < kPer; ++j) f32x2::vfma(o[h][j], v[j], w[h], o[h][j]);
    }
    __syncwarp();
  }

  static constexpr int kGiven = 1;
  __device__ __forceinline__ void halves() {  // the two rows' sums
    if constexpr (kRows == 2)
#pragma unroll
      for (int h = 0; h < HB; ++h)
#pragma unroll
        for (int j = 0; j < kPer; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[h][j][e] += __shfl_xor_sync(~0u, o[h][j][e], 16);
  }
  __device__ __forceinline__ void give(float *sums, float2 (*ml)[32], int lane, int) {
    halves();
    ml[0][lane] = make_float2(m, l);
    if (lane < kLanes)
#pragma unroll
      for (int h = 0; h < HB; ++h)
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          reinterpret_cast<float4 *>(sums)[(h * kPer + j) * kLanes + lane] = make_float4(o[h][j][0], o[h][j][1], o[h][j][2], o[h][j][3]);
  }
  __device__ __forceinline__ void take(const float *sums, const float2 (*ml)[32], int lane, int) {
    halves();
    float mine, theirs;
    meet(m, l, ml[0][lane].x, ml[0][lane].y, mine, theirs);
#pragma unroll
    for (int h = 0; h < HB; ++h) {
      const float f = __shfl_sync(~0u, mine, h), f2 = __shfl_sync(~0u, theirs, h);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const float4 a = reinterpret_cast<const float4 *>(sums)[(h * kPer + j) * kLanes + lane % kLanes];
        o[h][j][0] = fmaf(o[h][j][0], f, a.x * f2);
        o[h][j][1] = fmaf(o[h][j][1], f, a.y * f2);
        o[h][j][2] = fmaf(o[h][j][2], f, a.z * f2);
        o[h][j][3] = fmaf(o[h][j][3], f, a.w * f2);
      }
    }
  }
  // (behind take: the rows' halves are together)
  __device__ __forceinline__ void end(float *sums, float2 *ml, int lane, int) {
#pragma unroll
    for (int d = HB; d < 32; d *= 2) l += __shfl_xor_sync(~0u, l, d);
    if (lane < HB) ml[lane] = make_float2(m, l);
    if (lane < kLanes)
#pragma unroll
      for (int h = 0; h < HB; ++h)
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          reinterpret_cast<float4 *>(sums + h * D)[lane + 32 * j] = make_float4(o[h][j][0], o[h][j][1], o[h][j][2], o[h][j][3]);
  }
  static __device__ __forceinline__ int quad(int, int c) { return c; }
};

template <typename T> __device__ __forceinline__ void store4(T *dst, float4 v) {
  if constexpr (sizeof(T) == 4) *reinterpret_cast<float4 *>(dst) = v;
  else *reinterpret_cast<uint2 *>(dst) = make_uint2(pack(v.x, v.y), pack(v.z, v.w));
}

// A row's result from its sums: maximum m (of log2) and sum l.
template <typename T>
__device__ __forceinline__ void finish(const PagedAttn &p, int s, int h, int D, int quad, float m, float l, float4 v) {
  const float f = l > 0.f ? 1.f / l : 0.f;
  const size_t row = (size_t)s * p.H + h;
  store4(static_cast<T *>(p.o) + row * D + 4 * quad, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
  if (quad == 0 && p.lse) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.693147181f : -INFINITY;
}

template <typename T, int D, int HB>
__global__ void __launch_bounds__(kThreads, Shape<T, D, HB>::kCtas)
attn_kernel(const PagedAttn p, const Split sp, const FastDiv by_page) {
  using S = Shape<T, D, HB>;
  using Warp = std::conditional_t<S::kF32, F32Warp<D, HB>, Bf16Warp<D, HB>>;
  constexpr int kUnit = S::kUnit, kKeys = S::kKeys, kChunks = S::kChunks, kStages = S::kStages;
  constexpr int kHalf = kWarps / 2;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 given[kHalf][Warp::kGiven][32];
  __shared__ float2 ml[kHalf][HB];
  __shared__ uint32_t masks[kWarps][kStages];
  __shared__ int scan[kWarps], start_seq, start_number;
  float *sums = reinterpret_cast<float *>(smem + kStages * S::kStage * kWarps);  // [kHalf][HB][D]
  __shared__ __align__(16) float weights[S::kF32 ? kWarps : 1][S::kF32 ? kKeys * HB : 4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!sp.whole) {  // what the run is found from into L2 while the kernel in front ends
    const int line = blockIdx.x * kThreads + tid;
    if (line * 32ll < p.n) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.at.lens + line * 32ll));
    if (line < p.n * sp.lines)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.at.table + line / sp.lines * p.at.ld_table + line % sp.lines * 32));
  }
  wait_for_stream();

  // the CTA's run: the units with numbers in [t0, t1)
  Cursor<kKeys, kUnit> at = {};
  int t0, t1, part_begin, share = 0;
  if (sp.whole) {
    at.s = blockIdx.x / sp.parts;
    at.part = blockIdx.x % sp.parts;
    at.set(p);
    t0 = part_begin = 0;
    t1 = at.units;
  } else {
    const int per = (p.n + kThreads - 1) / kThreads, a = min(tid * per, p.n), b = min(a + per, p.n);
    auto numbers = [&](int s) {
      const int units = places_of(p, s).units(kKeys, kUnit);
      return units > 0 ? (units + kPartCost) * sp.parts : 0;
    };
    int mine = 0;
    for (int s = a; s < b; ++s) mine += numbers(s);
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int o = __shfl_up_sync(~0u, upto, d);
      if (lane >= d) upto += o;
    }
    if (lane == 31) scan[warp] = upto;
    if (tid == 0 && !sp.by_part) sp.joins[blockIdx.x] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) upto += scan[w];
      total += scan[w];
    }
    // (runs of one unit too: one sequence of 4096 places, 16/4 heads of 128, 10.2 us; of 2 units at least 10.9, 4 12.4)
    share = share_of(total, gridDim.x);
    const UnitRun run = run_of(blockIdx.x, share, total);
    t0 = run.first;
    t1 = run.end;
    if (t0 < t1) {
      int before = upto - mine;
      if (before <= t0 && t0 < upto) {
        for (int s = a; s < b; ++s) {
          const int u = numbers(s);
          if (t0 < before + u) {
            start_seq = s;
            start_number = before;
            break;
          }
          before += u;
        }
      }
      __syncthreads();
      at.s = start_seq;
      at.set(p);
      const unsigned each = at.units + kPartCost, in = t0 - start_number;
      at.part = in / each;
      at.unit = max((int)(in - at.part * each) - kPartCost, 0);
      part_begin = start_number + at.part * each + kPartCost;
      at.number = part_begin + at.unit;
    } else {
      at.number = t1;
    }
  }

  const int share_heads = p.H / p.Hk;
  // the ring
  const uint32_t ring = sm100::smem_u32(smem) + warp * kStages * S::kStage;
  const size_t row_step = (size_t)p.Hk * D;
  Cursor<kKeys, kUnit> to = at;  // where the copies are
  auto load = [&](int stage) {
    // places i0 .. i0 + kKeys - 1; i0 is a multiple of kKeys
    const int i0 = to.at.first / kKeys * kKeys + to.unit * kUnit + warp * kKeys;
    const uint32_t all = (1u << kKeys) - 1;
    uint32_t there = to.at.first > i0 ? all << (to.at.first - i0) & all : all;  // (first is in the first block)
    if (to.at.len - i0 < kKeys) there = to.at.len > i0 ? there & ((1u << (to.at.len - i0)) - 1) : 0;
    const uint32_t keys = ring + stage * S::kStage, values = keys + S::kTile;
    const int head = to.part / sp.blocks;
    const int *table = p.at.table + to.s * p.at.ld_table;
    if (there) {
      uint32_t pg, r0;
      by_page.split(i0, pg, r0);
      if (r0 + kKeys <= (uint32_t)p.at.page_size) {  // all in one page
        const int page = table[pg];
        if (page < 0 || page >= p.at.n_pages) there = 0;
        const size_t e = page * p.at.ld_page + (size_t)r0 * row_step + head * D + lane / kChunks * row_step +
                         lane % kChunks * (16 / (int)sizeof(T));
        const T *k = static_cast<const T *>(p.k_cache) + e, *v = static_cast<const T *>(p.v_cache) + e;
        if (there)
#pragma unroll
          for (int j = 0; j < kKeys * kChunks / 32; ++j) {
            const int c = j * 32 + lane, row = c / kChunks, chunk = c % kChunks;
            const bool on = there >> row & 1;
            copy16(keys + (row * kChunks + stored<S::kF32, false>(row, chunk)) * 16, k, on);
            copy16(values + (row * kChunks + stored<S::kF32, true>(row, chunk)) * 16, v, on);
            // the next one of this lane: 32 / kChunks rows on, or in the same row
            const size_t step = kChunks <= 32 ? 32 / kChunks * row_step
                                : (j + 1) % (kChunks / 32) ? 32 * (16 / sizeof(T))
                                                           : row_step - (kChunks - 32) * (16 / sizeof(T));
            k += step;
            v += step;
          }
      } else {
        const int i = i0 + lane % kKeys;
        long long off = -1;
        if (there >> (lane % kKeys) & 1) {
          uint32_t r;
          by_page.split(i, pg, r);
          const int page = table[pg];
          if (page >= 0 && page < p.at.n_pages) off = page * p.at.ld_page + r * (long long)row_step + head * D;
        }
        there = __ballot_sync(~0u, off >= 0) & all;
        if (there)
#pragma unroll 1
          for (int j = 0; j < kKeys * kChunks / 32; ++j) {
            const int c = j * 32 + lane, row = c / kChunks, chunk = c % kChunks;
            const long long o = __shfl_sync(~0u, off, row);
            const long long e = (o < 0 ? 0 : o) + chunk * (16 / (int)sizeof(T));
            copy16(keys + (row * kChunks + stored<S::kF32, false>(row, chunk)) * 16, static_cast<const T *>(p.k_cache) + e, o >= 0);
            copy16(values + (row * kChunks + stored<S::kF32, true>(row, chunk)) * 16, static_cast<const T *>(p.v_cache) + e, o >= 0);
          }
      }
    }
    if (lane == 0) masks[warp][stage] = there;
    // the queries of a part into L1 while its first keys are on their way
    if (warp == 0 && (to.unit == 0 || to.number == at.number)) {
      const int h0 = head * share_heads + to.part % sp.blocks * HB;
      const char *q = reinterpret_cast<const char *>(static_cast<const T *>(p.q) + to.s * p.ldq + (long long)h0 * D);
      for (int i = lane * 128; i < min(HB, share_heads - to.part % sp.blocks * HB) * D * (int)sizeof(T); i += 32 * 128)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(q + i));
    }
    to.next(p, sp.parts, t1);
  };
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) {
    if (to.number < t1) load(i);
    commit();
  }
  // rows of sequences without a place meanwhile
  if (!sp.whole)
#pragma unroll 1
    for (int s = blockIdx.x; s < p.n; s += gridDim.x) {
      const Range r = places_of(p, s);
      if (r.len > r.first) continue;
      for (int i = tid; i < p.H * (D / 4); i += kThreads)
        finish<T>(p, s, i / (D / 4), D, i % (D / 4), 0.f, 0.f, make_float4(0.f, 0.f, 0.f, 0.f));
      if (sp.by_part)
        for (int i = tid; i < sp.parts; i += kThreads) sp.joins[s * sp.parts + i] = make_int4(-1, 0, 0, 0);
    }
  if (!sp.whole && at.number >= t1) return;

  Warp w;
  int stage = 0;
  bool fresh = true;
  if (at.units == 0) w.begin(p, at.s, 0, 0, lane);  // a whole part without a place
  while (true) {
    const int h0 = at.part / sp.blocks * share_heads + at.part % sp.blocks * HB;
    const int heads = min(HB, share_heads - at.part % sp.blocks * HB);
    bool last = true;
    if (at.units > 0) {
      if (fresh) w.begin(p, at.s, h0, heads, lane);
      wait_all_but<kStages - 2>();
      __syncwarp();
      const int free = stage == 0 ? kStages - 1 : stage - 1;
      const uint32_t there = masks[warp][stage];
      if (to.number < t1) load(free);
      commit();
      if (there) {
        const uint32_t keys = ring + stage * S::kStage;
        w.block(keys, keys + S::kTile, there, lane, weights[S::kF32 ? warp : 0]);
      }
      stage = stage == kStages - 1 ? 0 : stage + 1;
      last = at.unit + 1 == at.units || at.number + 1 == t1;
    }
    fresh = last;
    if (last) {
      // half of the warps hand their sums to the others
      if (warp >= kHalf) w.give(sums + (warp - kHalf) * HB * D, given[warp - kHalf], lane, heads);
      __syncthreads();
      if (warp < kHalf) {
        w.take(sums + warp * HB * D, given[warp], lane, heads);
        __syncwarp();
        w.end(sums + warp * HB * D, ml[warp], lane, heads);
      }
      __syncthreads();
      const int part_end = part_begin + at.units;
      const bool begun = part_begin >= t0, done = part_end <= t1;
      for (int i = tid; i < heads * (D / 4); i += kThreads) {
        const int h = i / (D / 4), c = i % (D / 4);
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int k = 0; k < kHalf; ++k) m = fmaxf(m, ml[k][h].x);
        const float zero = m == -INFINITY ? 0.f : m;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kHalf; ++k) {
          const float f = sm100::ex2(ml[k][h].x - zero);
          const float4 a = reinterpret_cast<const float4 *>(sums + (k * HB + h) * D)[Warp::quad(h, c)];
          l = fmaf(f, ml[k][h].y, l);
          v.x = fmaf(f, a.x, v.x); v.y = fmaf(f, a.y, v.y); v.z = fmaf(f, a.z, v.z); v.w = fmaf(f, a.w, v.w);
        }
        if (begun && done) {
          finish<T>(p, at.s, h0 + h, D, c, m, l, v);
        } else {
          const size_t piece = 2 * (size_t)blockIdx.x + begun;
          reinterpret_cast<float4 *>(sp.sums + (piece * HB + h) * D)[c] = v;
          if (c == 0) sp.ml[piece * HB + h] = make_float2(m, l);
        }
      }
      if (begun && tid == 0 && !sp.whole && (sp.by_part || !done))
        sp.joins[sp.by_part ? at.s * sp.parts + at.part : blockIdx.x] =
            done ? make_int4(-1, 0, 0, 0) : make_int4(at.s, at.part, blockIdx.x, (part_end - 1) / share);
      part_begin = part_end + kPartCost;
    }
    if (at.units == 0) return;
    at.next(p, sp.parts, t1);
    if (at.number >= t1) return;
    if (last) __syncthreads();
  }
}

// The pieces of a part added up: block (entry of joins, some of the heads).
template <typename T, int D, int HB>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const PagedAttn p, const Split sp) {
  constexpr int kQuads = D / 4;
  __shared__ float4 sums[kJoinThreads];
  __shared__ float2 ml[kJoinThreads];
  wait_for_stream();
  const int4 join = sp.joins[blockIdx.x];  // (written by the kernel in front)
  if (join.x < 0) return;
  const int each = HB / gridDim.y, share_heads = p.H / p.Hk, block = join.y % sp.blocks;
  const int heads = min(HB, share_heads - block * HB), h0 = join.y / sp.blocks * share_heads + block * HB;
  const int items = each * kQuads, groups = max(kJoinThreads / items, 1);
  const int pieces = join.w - join.z + 1;
  for (int i0 = 0; i0 < items; i0 += kJoinThreads) {
    const int i = i0 + threadIdx.x % min(items, kJoinThreads), group = threadIdx.x / min(items, kJoinThreads);
    const int h = blockIdx.y * each + i / kQuads, c = i % kQuads;
    float m = -INFINITY, l = 0.f, f, f2;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (h < heads) {
#pragma unroll 4
      for (int k = group; k < pieces; k += groups) {
        const size_t piece = 2 * (size_t)(join.z + k) + (k == 0);
        const float2 b = sp.ml[piece * HB + h];
        const float4 a = reinterpret_cast<const float4 *>(sp.sums + (piece * HB + h) * D)[c];
        meet(m, l, b.x, b.y, f, f2);
        v = make_float4(v.x * f + a.x * f2, v.y * f + a.y * f2, v.z * f + a.z * f2, v.w * f + a.w * f2);
      }
    }
    if (groups > 1) {
      sums[threadIdx.x] = v;
      ml[threadIdx.x] = make_float2(m, l);
      __syncthreads();
      if (group == 0) {
        for (int g = 1; g < groups; ++g) {
          const float2 b = ml[g * items + threadIdx.x];
          const float4 a = sums[g * items + threadIdx.x];
          meet(m, l, b.x, b.y, f, f2);
          v = make_float4(v.x * f + a.x * f2, v.y * f + a.y * f2, v.z * f + a.z * f2, v.w * f + a.w * f2);
        }
      }
    }
    if (group == 0 && h < heads) finish<T>(p, join.x, h0 + h, D, c, m, l, v);
  }
}

int fail(const char *what, cudaError_t e) {
  set_error("la_paged_attn: %s: %s", what, cudaGetErrorString(e));
  return LA_ERR_CUDA;
}

// Units up to which a part is one CTA's, which saves the second kernel; and where there are parts for half of the CTAs
// or more. (16/4 heads of 128, bfloat16, whole and split: 16 x 384 places 9.6 and 12.7 us, 1 x 384 9.1 and 8.9,
// 1 x 512 10.7 and 9.1; 64 x 384 12.2 and 16.8, 64 x 768 21.9 and 26.3.) Where few CTAs of bfloat16 fit on a SM and there
// are several parts for each, a run is better again, as one part's keys come while the one before ends (126 x 200 places,
// 32/32 heads of 128: 94 and 83 us, of 256 220 and 193; 126 x 64 of 256 114 and 82; 126 x 400, 16/8 of 128 46.5 and 44.2;
// heads of 64: 126 x 400 77 and 80; float32, 126 x 200 of 128 128 and 150).
constexpr int kWhole = 6, kWholeOfMany = 16, kManyParts = 3;

template <typename T, int D, int HB>
int launch(const PagedAttn &p, cudaStream_t stream) {
  using S = Shape<T, D, HB>;
  Split sp = {};
  sp.blocks = (p.H / p.Hk + HB - 1) / HB;
  sp.parts = p.Hk * sp.blocks;
  const long long most = std::min((long long)p.at.max_pages * p.at.page_size, (long long)kMostPlaces);
  long long longest = p.max_len > 0 ? std::min<long long>(p.max_len, most) : most;
  if (p.window > 0) longest = std::min<long long>(longest, p.window);
  const long long parts = (long long)p.n * sp.parts;
  // all units of the table, whatever max_len says; where an int does not hold them, short lengths take whole parts
  const bool countable = most / S::kUnit + 2 + kPartCost <= INT_MAX / std::max(parts, 1ll);
  if (!countable && longest > (long long)kWholeOfMany * S::kUnit) {
    set_error("la_paged_attn: n * Hk times max_pages * page_size too large");
    return LA_ERR_INVALID_ARG;
  }
  auto kernel = attn_kernel<T, D, HB>;
  static std::atomic<bool> ready[64];  // once for each device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail("no device", e);
  if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    if (e != cudaSuccess) return fail("shared memory", e);
    if (dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  const long long slots = (long long)S::kCtas * std::max(sm_count(), 1);
  sp.whole = !countable || most == 0 ||
             (longest <= (long long)(2 * parts >= slots ? kWholeOfMany : kWhole) * S::kUnit &&
              (S::kF32 || S::kCtas > 2 || parts < kManyParts * slots));
  const FastDiv by(p.at.page_size);
  if (sp.whole) {
    e = launch_early(kernel, dim3(static_cast<unsigned>(parts)), kThreads, S::kBytes, stream, p, sp, by);
    return e == cudaSuccess ? LA_OK : fail("launch failed", e);
  }
  const long long units = ((longest + S::kUnit - 1) / S::kUnit + kPartCost) * parts;
  const int ctas = static_cast<int>(std::min(slots, units));
  // (of longer rows a part)
  sp.lines = static_cast<int>(std::min<long long>(((longest - 1) / p.at.page_size + 32) / 32, 64));
  if ((long long)sp.lines * p.n > INT_MAX / 2) sp.lines = 0;
  if (p.window > 0) sp.lines = 0;
  const size_t sums = (size_t)2 * ctas * HB * D * 4, ml = (size_t)2 * ctas * HB * sizeof(float2);
  sp.by_part = parts <= ctas;
  const size_t entries = sp.by_part ? parts : ctas;
  cudaMemPool_t pool = library_pool();
  if (!pool) return fail("could not create the workspace pool", cudaGetLastError());
  uint8_t *ws = nullptr;
  e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), sums + ml + entries * sizeof(int4), pool, stream);
  if (e != cudaSuccess) return fail("workspace allocation failed", e);
  sp.sums = reinterpret_cast<float *>(ws);
  sp.ml = reinterpret_cast<float2 *>(ws + sums);
  sp.joins = reinterpret_cast<int4 *>(ws + sums + ml);
  e = launch_early(kernel, dim3(ctas), kThreads, S::kBytes, stream, p, sp, by);
  unsigned apart = 1;  // blocks of a part's heads: up to two for each SM (64 parts of 16 heads, the call: 4 a part 53 us, 16 57)
  while (2 * apart <= HB && 2 * apart * entries <= 2 * (size_t)std::max(sm_count(), 1)) apart *= 2;
  if (e == cudaSuccess)
    e = launch_early(join_kernel<T, D, HB>, dim3(static_cast<unsigned>(entries), apart), kJoinThreads, 0, stream, p, sp);
  const cudaError_t f = cudaFreeAsync(ws, stream);
  if (e == cudaSuccess) e = f;
  return e == cudaSuccess ? LA_OK : fail("launch failed", e);
}

template <int D> int launch_d(const PagedAttn &p, cudaStream_t stream) {
  if (p.f32) return p.H / p.Hk <= 4 ? launch<float, D, 4>(p, stream) : launch<float, D, 8>(p, stream);
  return p.H / p.Hk <= 8 ? launch<__nv_bfloat16, D, 8>(p, stream) : launch<__nv_bfloat16, D, 16>(p, stream);
}

}  // namespace

int launch_paged_attn(const PagedAttn &p, cudaStream_t stream) {
  return p.d == 64 ? launch_d<64>(p, stream) : p.d == 128 ? launch_d<128>(p, stream) : launch_d<256>(p, stream);
}

}  // namespace la
