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
      for (int i = 0; i < N; ++i) v[i] = activate<kFast>(v[i], ACT_SILU);
      break;
    case ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate<kFast>(v[i], ACT_GELU);
      break;
    default:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate<kFast>(v[i], ACT_GELU_TANH);
  }
}

}  // namespace muon
