// Pieces shared by the tensor-core kernels of a layer's product.
#pragma once

#include "act.cuh"
#include "common.cuh"
#include "mbarrier.cuh"
#include "ops.h"
#include "tcgen05.cuh"

namespace muon {

constexpr int BK = 64;  // steps of the sum in one block of the ring: a 128-byte swizzle row

// Cycles after which a wait for a tile's whole sum gives up: the bound of a short
// wait, and 4096 for each block of each partial product (which takes 400 to 700), so
// that no length the calls accept runs into it.
__device__ __forceinline__ long long sum_wait(int steps, int products) {
  return kWaitCycles + (long long)((steps + BK - 1) / BK) * products * 4096;
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Planes (0 high, 1 middle, 2 low) of the two operands in partial product i,
// smallest products first.
constexpr int kProducts = 6;
__device__ __forceinline__ int plane_m(int i) { return (0x010120 >> (4 * i)) & 3; }
__device__ __forceinline__ int plane_n(int i) { return (0x001102 >> (4 * i)) & 3; }

__device__ __forceinline__ float ld_el(const void* p, int64_t i, int type) {
  if (type == DT_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  if (type == DT_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void st_el(void* p, int64_t i, float v, int type) {
  if (type == DT_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else if (type == DT_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<float*>(p)[i] = v;
}
// 8 values of a 16-bit type.
__device__ __forceinline__ void unpack8(const uint4& u, float* f, int type) {
  if (type == DT_BF16) {
    bf16x8_to_f32(u, f);
  } else {
    const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(h[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
}
__device__ __forceinline__ uint4 pack8(const float* f, int type) {
  if (type == DT_BF16) return f32_to_bf16x8(f);
  uint4 u;
  __half2* h = reinterpret_cast<__half2*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
  return u;
}
// SiLU and the tanh form of GELU of 16-bit tensors, two values at a time: both are z p
// with p = 1 / (1 + e^-v) = 1 / (1 + 2^t), t = -v log2(e), on the hardware's power of two
// and reciprocal (PTX ex2.approx, within 2^-22 of itself, and rcp.approx, 2^-23).  t is
// rounded once and its factor once, which 2^t turns into 1.2 |v| 2^-24 of itself; with the
// sum's and the product's roundings z p is within (1.2 |v| + 8) 2^-24 of itself: 7e-6 at
// v = -87, far below half a step of the 16-bit store (2^-11, 2^-8).  Beyond, 2^t > 2^126,
// p may be flushed to 0: off by 2^-126 |z| at most.  Infinite v give 1 and 0.  Every 16-bit
// number is tested against these bounds.  The epilogue takes issue slots and power from the
// product: 4096 tokens, [4096, 16384] in 4 bits, bias, gelu_tanh 113 us against 121 one
// value at a time, silu 109 against 113.  (Done so for GELU too, that form gains nothing,
// 139, and the others lose it again, 128 and 122.)
__device__ __forceinline__ float2 sigmoid2(float2 v) {
  const float2 t = __fmul2_rn(v, make_float2(-1.4426950408889634f, -1.4426950408889634f));
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  e = __fadd2_rn(e, make_float2(1.f, 1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
  return r;
}
__device__ __forceinline__ float2 silu2(float2 z) { return __fmul2_rn(z, sigmoid2(z)); }
__device__ __forceinline__ float2 gelu_tanh2(float2 z) {
  const float c = kTanhCubic, k = 2.f * kSqrt2OverPi;
  const float2 zz = __fmul2_rn(__fmul2_rn(z, make_float2(c, c)), z);
  return __fmul2_rn(z, sigmoid2(__fmul2_rn(__ffma2_rn(zz, z, z), make_float2(k, k))));
}
template <int N, bool kFast>
__device__ __forceinline__ void activate_n(float* v, int act) {
  switch (act) {  // outside the loop over values
    case ACT_NONE: break;
    case ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate<kFast>(v[i], ACT_RELU);
      break;
    case ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        if constexpr (kFast) {
          const float2 r = silu2(make_float2(v[i], v[i + 1]));
          v[i] = r.x;
          v[i + 1] = r.y;
        } else {
          v[i] = activate<kFast>(v[i], ACT_SILU);
          v[i + 1] = activate<kFast>(v[i + 1], ACT_SILU);
        }
      }
      break;
    case ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate<kFast>(v[i], ACT_GELU);
      break;
    default:
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        if constexpr (kFast) {
          const float2 r = gelu_tanh2(make_float2(v[i], v[i + 1]));
          v[i] = r.x;
          v[i + 1] = r.y;
        } else {
          v[i] = activate<kFast>(v[i], ACT_GELU_TANH);
          v[i + 1] = activate<kFast>(v[i + 1], ACT_GELU_TANH);
        }
      }
  }
}

}  // namespace muon
