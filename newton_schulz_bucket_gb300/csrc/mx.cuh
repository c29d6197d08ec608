// Microscaled 4-bit numbers: blocks of 32 share a scale 2^(s - 127) (8 bits: s, 255
// is NaN), and each element has a sign, two bits of exponent and one of mantissa:
// 0, 0.5, 1, 1.5, 2, 3, 4 or 6.
#pragma once

#include <cstdint>
#include <type_traits>

#include "common.cuh"

namespace muon {

constexpr int kMxBlock = 32;
constexpr uint32_t kMxNan = 255;

// The scale of a block whose largest magnitude has these bits (fp32 without its
// sign): the power of two at or below it, over 2^2, the largest one at or below 6.
// A block that holds an infinity or a NaN is NaN as a whole (the scale has no
// infinity), whatever its elements are.
__device__ __forceinline__ uint32_t mx_scale(uint32_t top) {
  const uint32_t e = top >> 23;
  return e == 255 ? kMxNan : (e > 2 ? e - 2 : 0);
}
// 1 / scale (any number for NaN).  Both are powers of two, so that dividing by one is
// exact; what is lost below 2^-126 is far below half of the smallest element.
__device__ __forceinline__ float mx_inverse(uint32_t s) { return __uint_as_float((254 - s) << 23 & 0x7f800000u); }
__device__ __forceinline__ float mx_value(uint32_t s) {
  return __uint_as_float(s == kMxNan ? 0x7fc00000u : (s ? s << 23 : 0x00400000u));
}

// Eight numbers rounded to nearest (ties to the even mantissa, 6 at most), the first
// in the low bits.
__device__ __forceinline__ uint32_t mx_pack8(const float* f) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}
// Eight neighbouring numbers of a row.
template <typename T>
struct Eight {
  static constexpr int kWords = 2 * (int)sizeof(T);
  uint32_t w[kWords];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void fetch(const T* p) {  // 16-byte loads; read once
#pragma unroll
    for (int c = 0; c < kWords / 4; ++c)
      *reinterpret_cast<uint4*>(w + 4 * c) = __ldcs(reinterpret_cast<const uint4*>(p) + c);
  }
  __device__ __forceinline__ void fetch_some(const T* p, int64_t n) {  // the first n, zeros behind
    T* h = reinterpret_cast<T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = i < n ? p[i] : from_f32<T>(0.f);
  }
  // The largest magnitude as the type's bits, a NaN above all (they compare as
  // integers).
  __device__ __forceinline__ uint32_t top() const {
    if constexpr (sizeof(T) == 4) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
      return m;
    } else {
      using Pair = typename std::conditional<std::is_same<T, __nv_bfloat16>::value, __nv_bfloat162, __half2>::type;
      const Pair* h = reinterpret_cast<const Pair*>(w);
      const Pair m = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])), __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
      const T one = __hmax_nan(m.x, m.y);
      return *reinterpret_cast<const uint16_t*>(&one);
    }
  }
  // The scale of a block whose largest magnitude has these bits.
  static __device__ __forceinline__ uint32_t scale(uint32_t top) {
    if constexpr (sizeof(T) == 4) return mx_scale(top);
    else if constexpr (std::is_same<T, __nv_bfloat16>::value) return mx_scale(top << 16);
    else return mx_scale(__float_as_uint(__half2float(__ushort_as_half((uint16_t)top))));
  }
  __device__ __forceinline__ uint32_t packed(float inverse) const {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 4) f[i] = __uint_as_float(w[i]);
      else if constexpr (std::is_same<T, __nv_bfloat16>::value) f[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
      else f[i] = __half2float(__ushort_as_half((uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu)));
      f[i] *= inverse;
    }
    return mx_pack8(f);
  }
};

__device__ __forceinline__ void mx_unpack8(uint32_t v, float scale, float* f) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(v));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    f[2 * i] = t.x * scale;
    f[2 * i + 1] = t.y * scale;
  }
}

}  // namespace muon
