// Float32 arithmetic on pairs: Blackwell's f32x2 instructions do two lanes'
// worth of FMA, multiply or add in one issue slot (and half the code). The
// array forms take any even length; odd ones go element by element.
#pragma once

#include <cstdint>

namespace la {
namespace f32x2 {

__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(uint64_t p, float *r) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r[0]), "=f"(r[1]) : "l"(p));
}
__device__ __forceinline__ uint64_t fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// On two neighbouring floats.
__device__ __forceinline__ uint64_t at(const float *a) { return pair(a[0], a[1]); }
__device__ __forceinline__ void fma2(float *r, const float *a, uint64_t b, const float *c) { split(fma(at(a), b, at(c)), r); }
__device__ __forceinline__ void add2(float *r, const float *a, const float *b) { split(add(at(a), at(b)), r); }
__device__ __forceinline__ void mul2(float *r, const float *a, uint64_t b) { split(mul(at(a), b), r); }

// On arrays: r = a b, r = a s, r = a b + c, r = a s + c, sum of a b.
template <int E> __device__ __forceinline__ void vmul(float (&r)[E], const float (&a)[E], const float (&b)[E]) {
#pragma unroll
  for (int i = 0; i + 1 < E; i += 2) split(mul(at(a + i), at(b + i)), r + i);
  if constexpr (E % 2) r[E - 1] = a[E - 1] * b[E - 1];
}
template <int E> __device__ __forceinline__ void vmul(float (&r)[E], const float (&a)[E], float s) {
  const uint64_t ss = pair(s, s);
#pragma unroll
  for (int i = 0; i + 1 < E; i += 2) split(mul(at(a + i), ss), r + i);
  if constexpr (E % 2) r[E - 1] = a[E - 1] * s;
}
template <int E>
__device__ __forceinline__ void vfma(float (&r)[E], const float (&a)[E], const float (&b)[E], const float (&c)[E]) {
#pragma unroll
  for (int i = 0; i + 1 < E; i += 2) split(fma(at(a + i), at(b + i), at(c + i)), r + i);
  if constexpr (E % 2) r[E - 1] = fmaf(a[E - 1], b[E - 1], c[E - 1]);
}
template <int E>
__device__ __forceinline__ void vfma(float (&r)[E], const float (&a)[E], float s, const float (&c)[E]) {
  const uint64_t ss = pair(s, s);
#pragma unroll
  for (int i = 0; i + 1 < E; i += 2) split(fma(at(a + i), ss, at(c + i)), r + i);
  if constexpr (E % 2) r[E - 1] = fmaf(a[E - 1], s, c[E - 1]);
}
template <int E> __device__ __forceinline__ float vdot(const float (&a)[E], const float (&b)[E]) {
  uint64_t t = 0;
#pragma unroll
  for (int i = 0; i + 1 < E; i += 2) t = fma(at(a + i), at(b + i), t);
  float s[2];
  split(t, s);
  if constexpr (E % 2) s[0] = fmaf(a[E - 1], b[E - 1], s[0]);
  return s[0] + s[1];
}

}  // namespace f32x2
}  // namespace la
