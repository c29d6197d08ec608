// A router's balance loss and the load of its experts.  With p the softmax of a
// token's logits over all experts, f_e the share of all assignments that went to
// expert e, and P_e the mean of p_e over the tokens that have an open expert,
//   loss = coef * experts * sum_e f_e P_e,
//   dlogits = dloss * coef * experts / tokens * p (f - <p, f>)
// (the assignments are counted, not differentiated).
//
// One pass over the logits.  NV neighbouring experts a lane and as few lanes a
// token as hold them, so that the two reductions of a softmax cost few shuffles (64
// experts: eight lanes, four tokens a warp).  A lane keeps the sums of its own
// experts' probabilities over its tokens, in two levels (kRun tokens, then their
// sums), so that long batches keep their digits; lanes, warps and blocks are then
// added in a fixed order, and counts are whole numbers: the same bits every time.
#include "common.cuh"
#include "ops.h"

namespace muon {

namespace {

// Threads of a forward block: its warps' sums have to fit in shared memory.
template <int NV>
constexpr int kForward = NV > 16 ? 256 : 512;
constexpr int kBackward = 256;
constexpr int kRun = 64;     // tokens a lane adds up before they join the sum of sums
constexpr float kInf = __builtin_huge_valf();

// Experts e0 .. e0 + NV - 1 of a row; -inf past the last one.  vec: rows start
// on 16 bytes.
template <typename T, int NV>
__device__ __forceinline__ void load_experts(const T* row, int e0, int experts, bool vec, float* v) {
  constexpr int kPiece = 16 / (int)sizeof(T);
  static_assert(NV % kPiece == 0, "whole pieces");
  if (vec && e0 + NV <= experts) {
#pragma unroll
    for (int c = 0; c < NV / kPiece; ++c) {
      const uint4 u = *reinterpret_cast<const uint4*>(row + e0 + c * kPiece);
      const T* h = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) v[c * kPiece + i] = to_f32(h[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = e0 + i < experts ? to_f32(row[e0 + i]) : -kInf;
  }
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// v becomes exp(v - max), -inf gives 0; returns whether any of the token's logits is
// above -inf (a NaN counts: its token comes out NaN).
template <int NV>
__device__ __forceinline__ bool exponentials(float* v, int lanes, bool* nan) {
  float high = -kInf;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    bad |= v[i] != v[i];
    high = fmaxf(high, v[i]);
  }
  for (int o = lanes >> 1; o > 0; o >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
  const unsigned any = __ballot_sync(0xffffffffu, bad);
  const int first = (threadIdx.x & 31) & ~(lanes - 1);
  *nan = (any >> first) & (lanes == 32 ? 0xffffffffu : (1u << lanes) - 1);
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = v[i] == -kInf ? 0.f : expf(v[i] - high);
  return high > -kInf || *nan;
}

template <typename T, int NV>
__global__ void __launch_bounds__(kForward<NV>) k_balance(BalanceArgs a, int lanes, bool vec) {
  extern __shared__ float fold[];  // [warps][experts] sums, then [experts + 1] counts
  constexpr int kThreads = kForward<NV>, kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = (lane & (lanes - 1)) * NV;
  int* hist = reinterpret_cast<int*>(fold + kWarps * a.experts);
  grid_launch_next();
  for (int i = threadIdx.x; i <= a.experts; i += kThreads) hist[i] = 0;
  __syncthreads();
  grid_wait();
  const int per = 32 / lanes;  // tokens a warp
  const int64_t t0 = a.tokens * blockIdx.x / gridDim.x, t1 = a.tokens * (blockIdx.x + 1) / gridDim.x;
  float sum[NV] = {}, run[NV] = {};
  int live = 0, turn = 0;
  const auto load = [&](int64_t t, float* v) {
    if (t < t1) {
      load_experts<T, NV>(static_cast<const T*>(a.logits) + t * a.stride, e0, a.experts, vec, v);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = -kInf;
    }
  };
  float next[NV];  // on its way while a token is worked on
  load(t0 + warp * per + lane / lanes, next);
  for (int64_t i = t0 * a.top_k + threadIdx.x; i < t1 * a.top_k; i += kThreads) {
    const int e = a.indices[i];
    if (e >= 0 && e < a.experts) atomicAdd(&hist[e], 1);  // whole numbers: the order of the additions does not show
  }
  for (int64_t first = t0 + warp * per; first < t1; first += kWarps * per) {
    float v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = next[i];
    load(first + kWarps * per + lane / lanes, next);
    bool nan;
    const bool open = exponentials<NV>(v, lanes, &nan);
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) total += v[i];
    total = lanes_sum(total, lanes);
    const float inv = nan ? __int_as_float(0x7fc00000) : (open ? 1.f / total : 0.f);
    live += open && e0 == 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) run[i] = fmaf(v[i], inv, run[i]);
    if (++turn == kRun) {
      turn = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) { sum[i] += run[i]; run[i] = 0.f; }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    sum[i] += run[i];
    for (int o = lanes; o < 32; o <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
    if (lane < lanes && e0 + i < a.experts) fold[warp * a.experts + e0 + i] = sum[i];
  }
  if (live) atomicAdd(&hist[a.experts], live);
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += fold[w * a.experts + e];
    a.part[(int64_t)blockIdx.x * a.experts + e] = s;
  }
  for (int e = threadIdx.x; e <= a.experts; e += kThreads)
    a.part_counts[(int64_t)blockIdx.x * (a.experts + 1) + e] = hist[e];
}

// The blocks' sums and counts together: one block.  A warp takes 32 experts
// (one a lane) of a share of the blocks: as many shares as there are warps for.  Expert
// `experts` is the tokens.
__global__ void __launch_bounds__(1024) k_balance_join(BalanceArgs a) {
  __shared__ float sums[32][33];
  __shared__ int counts[32][33];
  __shared__ float dots[32];
  __shared__ long long mades[32];
  __shared__ int tokens;
  grid_launch_next();
  grid_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = a.experts / 32 + 1, shares = groups < 32 ? 32 / groups : 1;
  float dot = 0.f;
  long long made = 0;
  for (int g0 = 0; g0 < groups; g0 += 32 / shares) {
    const int g = g0 + warp / shares, share = warp % shares, e = g * 32 + lane;
    const bool live = warp / shares < 32 / shares && g < groups && e <= a.experts;
    float s = 0.f;
    int c = 0;
    if (live) {
#pragma unroll 8
      for (int b = share; b < a.blocks; b += shares) {
        if (e < a.experts) s += a.part[(int64_t)b * a.experts + e];
        c += a.part_counts[(int64_t)b * (a.experts + 1) + e];
      }
    }
    sums[warp][lane] = s;
    counts[warp][lane] = c;
    __syncthreads();
    if (live && share == 0) {
      for (int w = 1; w < shares; ++w) { s += sums[warp + w][lane]; c += counts[warp + w][lane]; }
      if (e < a.experts) {
        a.counts[e] = c;
        made += c;
        dot = fmaf(s, (float)c, dot);
      } else {
        tokens = c;
      }
    }
    __syncthreads();
  }
  for (int o = 16; o > 0; o >>= 1) {
    dot += __shfl_xor_sync(0xffffffffu, dot, o);
    made += __shfl_xor_sync(0xffffffffu, made, o);
  }
  if (lane == 0) { dots[warp] = dot; mades[warp] = made; }
  __syncthreads();
  if (warp > 0) return;
  dot = warp_sum(dots[lane]);
  made = mades[lane];
  for (int o = 16; o > 0; o >>= 1) made += __shfl_xor_sync(0xffffffffu, made, o);
  if (lane == 0) {
    *a.loss = a.coef * (float)a.experts * (dot / (float)(made > 0 ? made : 1) / (float)(tokens > 0 ? tokens : 1));
    *a.live = tokens;
  }
}

template <typename T, int NV>
__global__ void __launch_bounds__(kBackward) k_balance_backward(BalanceArgs a, int lanes, bool vec) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = (lane & (lanes - 1)) * NV;
  grid_launch_next();
  grid_wait();
  const int per = 32 / lanes, step = (int)(kBackward / 32) * per;
  const T* res = static_cast<const T*>(a.residual);
  float v[NV], r[NV];
  const auto load = [&](int64_t t) {
    if (t < a.tokens) {
      load_experts<T, NV>(static_cast<const T*>(a.logits) + t * a.stride, e0, a.experts, vec, v);
      if (res) load_experts<T, NV>(res + t * a.r_stride, e0, a.experts, vec, r);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = -kInf;
    }
  };
  const int64_t begin = (int64_t)blockIdx.x * step + warp * per;
  load(begin + lane / lanes);
  float share[NV], made = 0.f;
  {
    long long all = 0;
    int c[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      c[i] = e0 + i < a.experts ? a.counts[e0 + i] : 0;
      all += c[i];
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    made = all > 0 ? (float)all : 1.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) share[i] = (float)c[i] / made;
  }
  const int tokens = *a.live;
  const float scale = *a.dloss * a.coef * (float)a.experts / (float)(tokens > 0 ? tokens : 1);
  for (int64_t first = begin; first < a.tokens; first += (int64_t)gridDim.x * step) {
    const int64_t t = first + lane / lanes;
    if (first > begin) load(t);
    bool nan;
    const bool open = exponentials<NV>(v, lanes, &nan);
    float total = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      total += v[i];
      dot = fmaf(v[i], share[i], dot);
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    const float inv = nan ? __int_as_float(0x7fc00000) : (open ? 1.f / total : 0.f);
    dot *= inv;
    if (t >= a.tokens) continue;
    T* out = static_cast<T*>(a.dlogits) + t * a.experts + e0;
    T h[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      // (a masked expert's gradient is 0 whatever the others are)
      const float d = v[i] == 0.f ? 0.f : scale * (v[i] * inv) * (share[i] - dot);
      h[i] = from_f32<T>(res ? d + r[i] : d);
    }
    constexpr int kPiece = 16 / (int)sizeof(T);
    if (vec && e0 + NV <= a.experts) {
#pragma unroll
      for (int c = 0; c < NV / kPiece; ++c) {
        alignas(16) T piece[kPiece];
#pragma unroll
        for (int i = 0; i < kPiece; ++i) piece[i] = h[c * kPiece + i];
        *reinterpret_cast<uint4*>(out + c * kPiece) = *reinterpret_cast<const uint4*>(piece);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (e0 + i < a.experts) out[i] = h[i];
    }
  }
}

template <typename T, int NV>
cudaError_t run_nv(const BalanceArgs& a, bool backward, bool vec, cudaStream_t s) {
  int lanes = 1;
  while (lanes * NV < a.experts) lanes *= 2;
  if (backward) {
    const int64_t step = kBackward / lanes, rounds = (a.tokens + step - 1) / step, most = 8ll * num_sms();
    return launch_early(k_balance_backward<T, NV>, dim3((unsigned)(rounds < most ? rounds : most)), dim3(kBackward), 0,
                        s, a, lanes, vec);
  }
  const size_t smem = sizeof(float) * (kForward<NV> / 32) * a.experts + sizeof(int) * (a.experts + 1);
  return launch_early(k_balance<T, NV>, dim3((unsigned)a.blocks), dim3(kForward<NV>), smem, s, a, lanes, vec);
}

template <typename T>
cudaError_t run(const BalanceArgs& a, bool backward, cudaStream_t s) {
  const auto ok = [](const void* p, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride * (int64_t)sizeof(T) % 16 == 0;
  };
  const bool vec = ok(a.logits, a.stride) && (!backward || (ok(a.dlogits, a.experts) && ok(a.residual, a.r_stride)));
  if (a.experts <= 256) return run_nv<T, 8>(a, backward, vec, s);
  if (a.experts <= 512) return run_nv<T, 16>(a, backward, vec, s);
  return run_nv<T, 32>(a, backward, vec, s);
}

cudaError_t dispatch(const BalanceArgs& a, bool backward, cudaStream_t s) {
  switch (a.dtype) {
    case DT_F16: return run<__half>(a, backward, s);
    case DT_BF16: return run<__nv_bfloat16>(a, backward, s);
    default: return run<float>(a, backward, s);
  }
}

}  // namespace

// Blocks of the forward pass: some tokens each, and at most one an SM (one block
// joins their sums).
int balance_blocks(int64_t tokens, int32_t experts) {
  const int64_t some = (tokens * experts + 4095) / 4096, most = num_sms();
  return (int)(some < 1 ? 1 : (some < most ? some : most));
}

cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s) {
  cudaError_t e = dispatch(a, false, s);
  if (e == cudaSuccess) e = launch_early(k_balance_join, dim3(1), dim3(1024), 0, s, a);
  return e;
}
cudaError_t launch_balance_backward(const BalanceArgs& a, cudaStream_t s) { return dispatch(a, true, s); }

}  // namespace muon
