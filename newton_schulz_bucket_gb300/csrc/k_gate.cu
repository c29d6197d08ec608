// The gate: softmax over a token's expert logits, its top_k experts and their
// weights; and its gradient.
//
// One warp per token, expert e in lane e % 32.  The choice compares the
// logits themselves (the exponential is monotone, and this way equal logits
// stay equal): top_k rounds of a warp maximum over (logit, lower index).
#include "common.cuh"
#include "ops.h"

namespace muon {

namespace {

constexpr int kWarps = 8;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <typename T, int NV>
__global__ void __launch_bounds__(32 * kWarps) k_gate(GateArgs g) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  grid_launch_next();
  grid_wait();
  if (t >= g.tokens) return;
  const T* row = static_cast<const T*>(g.logits) + t * g.stride;
  float v[NV], w[NV];  // logits; logits still to choose from
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    v[i] = e < g.experts ? to_f32(row[e]) : -kInf;
    nan |= v[i] != v[i];
    w[i] = v[i] != v[i] ? -kInf : v[i];
  }
  nan = __any_sync(0xffffffffu, nan);
  float top = 0.f, high = 0.f, total = 0.f;  // lane j keeps choice j
  int idx = -1;
  for (int j = 0; j < g.top_k; ++j) {
    float best = -kInf;
    int at = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (w[i] > best) { best = w[i]; at = lane + 32 * i; }
    const float m = warp_max(best);
    if (m == -kInf) break;  // the same for the whole warp: no open expert is left
    const int e = __reduce_min_sync(0xffffffffu, best == m ? at : 0x7fffffff);
    if (j == 0) high = m;
    if (lane == j) { top = m; idx = e; }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e == lane + 32 * i) w[i] = -kInf;
  }
  const float p = idx >= 0 ? expf(top - high) : 0.f;
  if (g.renormalize) {
    total = warp_sum(p);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) total += v[i] == -kInf ? 0.f : expf(v[i] - high);
    total = warp_sum(total);
  }
  if (lane < g.top_k) {
    g.indices[t * g.top_k + lane] = idx;
    g.weights[t * g.top_k + lane] = idx < 0 ? 0.f : (nan ? __int_as_float(0x7fc00000) : p / total);
  }
}

// dlogits = p * (g - <p, g>), p the softmax over every expert or the chosen ones.
template <typename T, int NV>
__global__ void __launch_bounds__(32 * kWarps) k_gate_backward(GateArgs g) {
  extern __shared__ float smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
  grid_launch_next();
  grid_wait();
  if (t >= g.tokens) return;
  float* grad = smem + warp * 2 * g.experts;      // g per expert
  float* chosen = grad + g.experts;               // 1 where chosen
  for (int e = lane; e < g.experts; e += 32) grad[e] = chosen[e] = 0.f;
  __syncwarp();
  if (lane < g.top_k) {
    const int e = g.indices[t * g.top_k + lane];
    if (e >= 0 && e < g.experts) {
      grad[e] = g.dweights[t * g.top_k + lane];
      chosen[e] = 1.f;
    }
  }
  __syncwarp();
  const T* row = static_cast<const T*>(g.logits) + t * g.stride;
  float v[NV], high = -kInf;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    v[i] = e < g.experts ? to_f32(row[e]) : -kInf;
    nan |= v[i] != v[i];
    if (g.renormalize && e < g.experts && chosen[e] == 0.f) v[i] = -kInf;
    high = fmaxf(high, v[i]);
  }
  nan = __any_sync(0xffffffffu, nan);
  high = warp_max(high);
  float total = 0.f, dot = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    v[i] = v[i] == -kInf ? 0.f : expf(v[i] - high);
    total += v[i];
    if (e < g.experts) dot += v[i] * grad[e];
  }
  total = warp_sum(total);
  dot = warp_sum(dot);
  const float inv = nan ? __int_as_float(0x7fc00000) : (total > 0.f || total != total ? 1.f / total : 0.f);
  dot *= inv;
  T* out = static_cast<T*>(g.dlogits) + t * g.experts;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    if (e < g.experts) out[e] = from_f32<T>(v[i] == 0.f ? 0.f : v[i] * inv * (grad[e] - dot));
  }
}

template <typename T, int NV>
cudaError_t run_nv(const GateArgs& g, bool backward, cudaStream_t s) {
  const unsigned blocks = (unsigned)((g.tokens + kWarps - 1) / kWarps);
  const dim3 grid(blocks), block(32 * kWarps);
  if (backward)
    return launch_early(k_gate_backward<T, NV>, grid, block, sizeof(float) * 2 * kWarps * g.experts, s, g);
  return launch_early(k_gate<T, NV>, grid, block, 0, s, g);
}

template <typename T>
cudaError_t run(const GateArgs& g, bool backward, cudaStream_t s) {
  if (backward && g.experts > 512) {  // beyond the 48 KB of shared memory a launch has by default
    cudaError_t e = cudaFuncSetAttribute(k_gate_backward<T, 32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         sizeof(float) * 2 * kWarps * 1024);
    if (e != cudaSuccess) return e;
  }
  if (g.experts <= 32) return run_nv<T, 1>(g, backward, s);
  if (g.experts <= 64) return run_nv<T, 2>(g, backward, s);
  if (g.experts <= 128) return run_nv<T, 4>(g, backward, s);
  if (g.experts <= 256) return run_nv<T, 8>(g, backward, s);
  if (g.experts <= 512) return run_nv<T, 16>(g, backward, s);
  return run_nv<T, 32>(g, backward, s);
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
