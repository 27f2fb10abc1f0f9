// What the kernels that turn positions share: the cosine and sine of an angle,
// and rows moved V elements at a time.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace la {

// V elements (16 bytes, or 1) as float32.
template <typename T, int V> struct Vec {
  static __device__ __forceinline__ void load(const T *p, float *f) {
    if constexpr (V == 1) {
      f[0] = static_cast<float>(*p);
    } else {
      const uint4 u = *reinterpret_cast<const uint4 *>(p);
      if constexpr (sizeof(T) == 4) {
        f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
      } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = __uint_as_float(w[i] << 16);
          f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      }
    }
  }
  static __device__ __forceinline__ void store(T *p, const float *f) {
    if constexpr (V == 1) {
      *p = T(f[0]);
    } else if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
      __nv_bfloat162 h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<uint4 *>(h);
    }
  }
};

// Cosine and sine of pos * freq (freq in radians per position).
//
// pos * freq reaches millions of radians, where a float32 product has
// lost the angle and a float64 one is slow here. A frequency is held instead as
// its turns per position modulo one in 64-bit fixed point, F = frac(freq / 2 pi)
// 2^64; the integer product pos * F wraps at whole turns by itself, and its top
// 32 bits, signed, are the angle in [-1/2, 1/2) turns to 2^-32. freq / 2 pi is
// one float64 product: off by 2^-53 of itself, 2^-22 turns at a position of
// 2^31 and a frequency of one radian, far less at any real position.
__device__ __forceinline__ float2 rotary_turn(double freq, int position, bool inverse) {
  const double f = freq * 0.15915494309189535;  // 1 / (2 pi)
  const unsigned long long F = static_cast<unsigned long long>((f - floor(f)) * 18446744073709551616.0);
  const long long pos = position;
  const int t = static_cast<int>((static_cast<unsigned long long>(pos) * F) >> 32);
  float s, co;
  sincospif(static_cast<float>(t) * 4.656612873077393e-10f, &s, &co);  // 2^-31: half turns
  return make_float2(co, inverse ? -s : s);
}

}  // namespace la
