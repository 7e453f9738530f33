// e4m3 conversions and the cache's power-of-two scales.
#pragma once

#include <stdint.h>

namespace kda {

// Two fp32 values to two e4m3 codes (a in the low byte): nearest, ties to even, saturating at
// +-448 (infinities too), NaN to the NaN code.
__device__ __forceinline__ uint32_t e4m3x2_from_f32(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// Two e4m3 codes to two f16 values (exact: every e4m3 value, subnormals and NaN, is one).
__device__ __forceinline__ uint32_t f16x2_from_e4m3(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
  return r;
}
// The four codes of a word: (0, 1) to lo, (2, 3) to hi.
__device__ __forceinline__ void f16x4_from_e4m3(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
__device__ __forceinline__ float2 f32x2_from_f16x2(uint32_t h) {
  float2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\t"
      "cvt.f32.f16 %1, hi;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}

// The bits of |x| if x is finite, else 0 (as unsigned integers they order like the values).
__device__ __forceinline__ uint32_t finite_abs_bits(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
// Exponent of the smallest power of two s with m <= 448 s = 1.75 * 2^8 s, from the bits of m >= 0
// (for m below the normal numbers -135 or -134).
__device__ __forceinline__ int exponent_of(uint32_t mbits) {
  return (int)(mbits >> 23) - 127 - 8 + ((mbits & 0x7fffffu) > 0x600000u ? 1 : 0);
}
// The same of a page's scale: at least -100.
__device__ __forceinline__ int scale_exponent(uint32_t mbits) {
  const int e = exponent_of(mbits);
  return e < -100 ? -100 : e;
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// 16 bytes of a row as fp32 values: 8 bf16 or 4 fp32.
template <class T>
struct Vec16;
template <>
struct Vec16<float> {
  static constexpr int N = 4;
  __device__ static __forceinline__ void unpack(const uint4& r, float* x) {
    x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
  }
  __device__ static __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static __forceinline__ void unpack(const uint4& r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static __forceinline__ uint4 pack(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

}  // namespace kda
