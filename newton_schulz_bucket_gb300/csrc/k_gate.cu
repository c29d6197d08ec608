// The gate: softmax over a token's expert logits, its top_k experts and their
// weights; and its gradient.
//
// One warp per token, NV neighbouring experts a lane, so that a row is read in
// pieces of up to 16 bytes a lane.  The choice compares the logits themselves
// (the exponential is monotone, and this way equal logits stay equal), as
// integers in the same order: a round of the choice is one warp reduction and
// one vote, and the first lane that holds the maximum holds the lowest expert.
// Bound by instruction issue, not by HBM: 131072 tokens of 64 experts, 34 MB, take
// 44 us (35 back), 32768 of 512 take 48 (40 back); 16384 of 64 take 7.
#include "common.cuh"
#include "ops.h"

namespace muon {

namespace {

constexpr int kWarps = 8;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float nan_f() { return __int_as_float(0x7fc00000); }

// Larger for larger v, equal for equal (-0 and +0 too), 0 for -inf and NaN.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (!(v > -kInf)) return 0;
  const uint32_t u = __float_as_uint(v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// Experts e0 .. e0 + NV - 1 of a row; -inf past the last one.  vec: rows start
// on 16 bytes.
template <typename T, int NV>
__device__ __forceinline__ void load_experts(const T* row, int e0, int experts, bool vec, float* v) {
  constexpr int kBytes = NV * (int)sizeof(T) < 16 ? NV * (int)sizeof(T) : 16;
  constexpr int kEach = kBytes / (int)sizeof(T);
  if (vec && e0 + NV <= experts) {
#pragma unroll
    for (int c = 0; c < NV / kEach; ++c) {
      alignas(16) T h[kEach];
      if constexpr (kBytes == 16) *reinterpret_cast<uint4*>(h) = *reinterpret_cast<const uint4*>(row + e0 + c * kEach);
      else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(h) = *reinterpret_cast<const uint2*>(row + e0 + c * kEach);
      else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(h) = *reinterpret_cast<const uint32_t*>(row + e0 + c * kEach);
      else h[0] = row[e0];
#pragma unroll
      for (int i = 0; i < kEach; ++i) v[c * kEach + i] = to_f32(h[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = e0 + i < experts ? to_f32(row[e0 + i]) : -kInf;
  }
}

template <typename T, int NV>
__global__ void __launch_bounds__(32 * kWarps) k_gate(GateArgs g, bool vec) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  grid_launch_next();
  grid_wait();
  if (t >= g.tokens) return;
  float v[NV];
  uint32_t key[NV];  // 0: masked, or taken
  load_experts<T, NV>(static_cast<const T*>(g.logits) + t * g.stride, lane * NV, g.experts, vec, v);
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    nan |= v[i] != v[i];
    key[i] = order_key(v[i]);
  }
  nan = __any_sync(kAll, nan);
  float top = 0.f, high = 0.f;  // lane j keeps choice j
  int idx = -1;
  for (int j = 0; j < g.top_k; ++j) {
    uint32_t best = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < NV; ++i)
      if (key[i] > best) { best = key[i]; at = i; }
    const uint32_t m = __reduce_max_sync(kAll, best);
    if (m == 0) break;  // the same for the whole warp: no open expert is left
    const int owner = __ffs(__ballot_sync(kAll, best == m)) - 1;
    float value = v[0];
#pragma unroll
    for (int i = 1; i < NV; ++i)
      if (at == i) value = v[i];
    value = __shfl_sync(kAll, value, owner);
    const int e = owner * NV + __shfl_sync(kAll, at, owner);
    if (j == 0) high = value;
    if (lane == j) { top = value; idx = e; }
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (at == i) key[i] = 0;
    }
  }
  const float p = idx >= 0 ? expf(top - high) : 0.f;
  float total = p;
  if (!g.renormalize) {
    total = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) total += v[i] == -kInf ? 0.f : expf(v[i] - high);
  }
  total = warp_sum(total);
  if (lane < g.top_k) {
    g.indices[t * g.top_k + lane] = idx;
    g.weights[t * g.top_k + lane] = idx < 0 ? 0.f : (nan ? nan_f() : p / total);
  }
}

// dlogits = p * (g - <p, g>), p the softmax over every expert or the chosen ones.
template <typename T, int NV>
__global__ void __launch_bounds__(32 * kWarps) k_gate_backward(GateArgs g, bool vec) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  grid_launch_next();
  grid_wait();
  if (t >= g.tokens) return;
  const int e0 = lane * NV;
  float v[NV], grad[NV] = {};
  load_experts<T, NV>(static_cast<const T*>(g.logits) + t * g.stride, e0, g.experts, vec, v);
  int my_e = -1;
  float my_g = 0.f;
  if (lane < g.top_k) {
    my_e = g.indices[t * g.top_k + lane];
    my_g = g.dweights[t * g.top_k + lane];
    if (my_e >= g.experts) my_e = -1;
  }
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) nan |= v[i] != v[i];
  nan = __any_sync(kAll, nan);
  uint32_t chosen = 0;  // bit i: expert e0 + i
  for (int j = 0; j < g.top_k; ++j) {
    const int at = __shfl_sync(kAll, my_e, j) - e0;
    const float gj = __shfl_sync(kAll, my_g, j);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (at == i) { grad[i] = gj; chosen |= 1u << i; }
  }
  float high = -kInf;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (g.renormalize && !(chosen >> i & 1)) v[i] = -kInf;
    high = fmaxf(high, v[i]);
  }
  high = warp_max(high);
  float total = 0.f, dot = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v[i] = v[i] == -kInf ? 0.f : expf(v[i] - high);
    total += v[i];
    dot = fmaf(v[i], grad[i], dot);
  }
  total = warp_sum(total);
  dot = warp_sum(dot);
  const float inv = nan ? nan_f() : (total > 0.f || total != total ? 1.f / total : 0.f);
  dot *= inv;
  T* out = static_cast<T*>(g.dlogits) + t * g.experts;
  T h[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) h[i] = from_f32<T>(v[i] == 0.f ? 0.f : v[i] * inv * (grad[i] - dot));
  constexpr int kEach = NV * sizeof(T) < 16 ? NV : 16 / (int)sizeof(T);
  if (vec && e0 + NV <= g.experts && kEach * sizeof(T) == 16) {
#pragma unroll
    for (int c = 0; c < NV / kEach; ++c) {
      alignas(16) T piece[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) piece[i] = h[c * kEach + i];
      *reinterpret_cast<uint4*>(out + e0 + c * kEach) = *reinterpret_cast<const uint4*>(piece);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e0 + i < g.experts) out[e0 + i] = h[i];
  }
}

template <typename T, int NV>
cudaError_t run_nv(const GateArgs& g, bool backward, bool vec, cudaStream_t s) {
  const dim3 grid((unsigned)((g.tokens + kWarps - 1) / kWarps)), block(32 * kWarps);
  if (backward) return launch_early(k_gate_backward<T, NV>, grid, block, 0, s, g, vec);
  return launch_early(k_gate<T, NV>, grid, block, 0, s, g, vec);
}

template <typename T>
cudaError_t run(const GateArgs& g, bool backward, cudaStream_t s) {
  const auto ok = [](const void* p, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride * (int64_t)sizeof(T) % 16 == 0;
  };
  const bool vec = ok(g.logits, g.stride) && (!backward || ok(g.dlogits, g.experts));
  if (g.experts <= 32) return run_nv<T, 1>(g, backward, vec, s);
  if (g.experts <= 64) return run_nv<T, 2>(g, backward, vec, s);
  if (g.experts <= 128) return run_nv<T, 4>(g, backward, vec, s);
  if (g.experts <= 256) return run_nv<T, 8>(g, backward, vec, s);
  if (g.experts <= 512) return run_nv<T, 16>(g, backward, vec, s);
  return run_nv<T, 32>(g, backward, vec, s);
}

cudaError_t dispatch(const GateArgs& g, bool backward, cudaStream_t s) {
  switch (g.dtype) {
    case DT_F16: return run<__half>(g, backward, s);
    case DT_BF16: return run<__nv_bfloat16>(g, backward, s);
    default: return run<float>(g, backward, s);
  }
}

}  // namespace

cudaError_t launch_gate(const GateArgs& g, cudaStream_t s) { return dispatch(g, false, s); }
cudaError_t launch_gate_backward(const GateArgs& g, cudaStream_t s) { return dispatch(g, true, s); }

}  // namespace muon
