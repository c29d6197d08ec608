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
// Bound by the latency of its loads: a lane has one token ahead on its way, and none on the
// way back, so that DRAM is at 25% (back 22%) and the SM's busiest unit at 51% (60%) of their
// peaks, and waiting for loads is the largest stall.  131072 tokens of 64 experts, fp32, 34 MB,
// take 21 us (back, 67 MB, 18), 32768 of 512 44 (49); 16384 of 64 9.3 (4.7), where the
// latency of the two launches counts.
#include "common.cuh"
#include "ops.h"
#include "tcgen05.cuh"

namespace muon {

namespace {

// Threads of a forward block: its warps' sums have to fit in shared memory.
template <int NV>
constexpr int kForward = NV > 16 ? 256 : 512;
constexpr int kBackward = 256;
// Up to kClusterSize logits of up to 256 experts are one cluster's, which needs no
// scratch and no second launch (256 tokens of 64 experts 5.7 us; 16384 take 25 that way,
// 9.7 in two launches).
constexpr int kClusterBlocks = 8, kClusterThreads = 1024;
constexpr int64_t kClusterSize = 1 << 18;
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

__device__ __forceinline__ bool masked(float v) { return __float_as_uint(v) == 0x80000000u; }
// v becomes exp(v - max); returns whether any of the token's logits is above -inf (a NaN
// counts: its token comes out NaN).  A logit of -inf gives -0, which tells it from an
// exponential that underflowed (+0) and adds nothing all the same; a mask word beside the
// exponentials took 4% more of the way back.
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
  for (int i = 0; i < NV; ++i) v[i] = v[i] == -kInf ? -0.f : expf(v[i] - high);
  return high > -kInf || *nan;
}

template <typename T>
__device__ __forceinline__ T word_of(const T* p, int rank) {  // of the same place in block `rank`
  return ld_shared_of<T>(saddr(p), (uint32_t)rank);
}

__device__ __forceinline__ void write_loss(const BalanceArgs& a, float dot, long long made, int tokens) {
  *a.loss = a.coef * (float)a.experts * (dot / (float)(made > 0 ? made : 1) / (float)(tokens > 0 ? tokens : 1));
  *a.live = tokens;
}
// From the sums of all experts: dot = <sums of probabilities, counts>, made = the
// assignments, of the threads of a block.
__device__ __forceinline__ void finish(const BalanceArgs& a, float dot, long long made, int tokens, float* dots,
                                       long long* mades) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  dot = warp_sum(dot);
  for (int o = 16; o > 0; o >>= 1) made += __shfl_xor_sync(0xffffffffu, made, o);
  if (lane == 0) { dots[warp] = dot; mades[warp] = made; }
  __syncthreads();
  if (warp > 0) return;
  dot = warp_sum(dots[lane]);
  made = mades[lane];
  for (int o = 16; o > 0; o >>= 1) made += __shfl_xor_sync(0xffffffffu, made, o);
  if (lane == 0) write_loss(a, dot, made, tokens);
}

template <typename T, int NV, bool kCluster>
__global__ void __launch_bounds__(kCluster ? kClusterThreads : kForward<NV>) k_balance(BalanceArgs a, int lanes, bool vec) {
  extern __shared__ float fold[];  // [warps][experts] sums, then [experts + 1] counts
  constexpr int kThreads = kCluster ? kClusterThreads : kForward<NV>, kWarps = kThreads / 32;
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
    if constexpr (kCluster) fold[e] = s;  // (the thread's own column: nobody else reads it)
    else a.part[(int64_t)blockIdx.x * a.experts + e] = s;
  }
  if constexpr (kCluster) {  // the first block joins the eight
    __shared__ float dots[32];
    __shared__ long long mades[32];
    cluster_barrier();
    float dot = 0.f;
    int made = 0, tokens = 0;
    if (blockIdx.x == 0) {
      const int e = threadIdx.x;  // (up to 256 experts: one a thread)
      if (e <= a.experts) {
        float s = 0.f;
        int c = 0;
#pragma unroll
        for (int r = 0; r < kClusterBlocks; ++r) {
          if (e < a.experts) s += word_of(fold + e, r);
          c += word_of(hist + e, r);
        }
        if (e < a.experts) {
          a.counts[e] = c;
          made = c;
          dot = s * (float)c;
        } else {
          hist[a.experts] = c;
        }
      }
    }
    cluster_barrier();  // no block leaves while the first one reads its sums
    if (blockIdx.x > 0) return;
    tokens = hist[a.experts];
    finish(a, dot, made, tokens, dots, mades);
  } else {
    for (int e = threadIdx.x; e <= a.experts; e += kThreads)
      a.part_counts[(int64_t)blockIdx.x * (a.experts + 1) + e] = hist[e];
  }
}

// The blocks' sums and counts together: a cluster of blocks shares out the experts, 32
// at a time (one a lane; expert `experts` is the tokens), and a block's warps the
// blocks of the pass before.
__global__ void __launch_bounds__(1024) k_balance_join(BalanceArgs a) {
  __shared__ float sums[32][33];
  __shared__ int counts[32][33];
  __shared__ float dots[32];
  __shared__ long long mades[32];
  __shared__ uint32_t mine[4];  // dot, made (low, high), tokens
  grid_launch_next();
  grid_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float dot = 0.f;              // warp 0: of the lane's experts
  long long made = 0;
  int tokens = 0;
  for (int e0 = 32 * blockIdx.x; e0 <= a.experts; e0 += 32 * kClusterBlocks) {
    const int e = e0 + lane;
    float s = 0.f;
    int c = 0;
    if (e <= a.experts) {
#pragma unroll 8
      for (int b = warp; b < a.blocks; b += 32) {
        if (e < a.experts) s += a.part[(int64_t)b * a.experts + e];
        c += a.part_counts[(int64_t)b * (a.experts + 1) + e];
      }
    }
    sums[warp][lane] = s;
    counts[warp][lane] = c;
    __syncthreads();
    s = warp_sum(sums[lane][warp]);  // expert e0 + warp
    c = counts[lane][warp];
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    const int own = e0 + warp;
    if (lane == 0) {
      if (own < a.experts) {
        a.counts[own] = c;
        made += c;
        dot = fmaf(s, (float)c, dot);
      } else if (own == a.experts) {
        tokens = c;
      }
    }
    __syncthreads();
  }
  if (lane == 0) { dots[warp] = dot; mades[warp] = made; counts[0][warp] = tokens; }
  __syncthreads();
  if (warp == 0) {
    dot = warp_sum(dots[lane]);
    made = mades[lane];
    tokens = counts[0][lane];
    for (int o = 16; o > 0; o >>= 1) {
      made += __shfl_xor_sync(0xffffffffu, made, o);
      tokens += __shfl_xor_sync(0xffffffffu, tokens, o);
    }
    if (lane == 0) {
      mine[0] = __float_as_uint(dot);
      mine[1] = (uint32_t)made;
      mine[2] = (uint32_t)(made >> 32);
      mine[3] = (uint32_t)tokens;
    }
  }
  cluster_barrier();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    dot = 0.f;
    made = 0;
    tokens = 0;
    for (int r = 0; r < kClusterBlocks; ++r) {
      dot += __uint_as_float(word_of(&mine[0], r));
      made += (long long)((uint64_t)word_of(&mine[2], r) << 32 | word_of(&mine[1], r));
      tokens += (int)word_of(&mine[3], r);
    }
    write_loss(a, dot, made, tokens);
  }
  cluster_barrier();  // no block leaves while the first one reads its sums
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
      // (a masked expert's gradient is 0 whatever the others are; in a token with a NaN or
      // +inf every open one's is NaN, the underflowed ones' too: inv and dot are)
      const float d = masked(v[i]) ? 0.f : scale * (v[i] * inv) * (share[i] - dot);
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
  const auto smem = [&](int threads) { return sizeof(float) * (threads / 32) * a.experts + sizeof(int) * (a.experts + 1); };
  if constexpr (NV == 8) {
    if (a.blocks == 0) {
      return launch_early_cluster(k_balance<T, NV, true>, kClusterBlocks, kClusterThreads, smem(kClusterThreads),
                                  kClusterBlocks, s, a, lanes, vec);
    }
  }
  return launch_early(k_balance<T, NV, false>, dim3((unsigned)a.blocks), dim3(kForward<NV>), smem(kForward<NV>), s, a, lanes,
                      vec);
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

// Blocks of the forward pass: some tokens each, and at most two an SM (one block
// joins their sums); 0: one cluster.
int balance_blocks(int64_t tokens, int32_t experts) {
  if (experts <= 256 && tokens * experts <= kClusterSize) return 0;
  const int64_t some = (tokens * experts + 4095) / 4096, most = 2ll * num_sms();
  return (int)(some < 1 ? 1 : (some < most ? some : most));
}

cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s) {
  cudaError_t e = dispatch(a, false, s);
  if (e == cudaSuccess && a.blocks > 0)
    e = launch_early_cluster(k_balance_join, kClusterBlocks, kClusterThreads, 0, kClusterBlocks, s, a);
  return e;
}
cudaError_t launch_balance_backward(const BalanceArgs& a, cudaStream_t s) { return dispatch(a, true, s); }

}  // namespace muon
