// Microscaled 4-bit numbers: blocks of 32 share a scale 2^(s - 127) (8 bits: s, 255
// is NaN), and each element has a sign, two bits of exponent and one of mantissa:
// 0, 0.5, 1, 1.5, 2, 3, 4 or 6.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

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
