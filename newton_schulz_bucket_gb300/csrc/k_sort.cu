// Token rows into expert order and back, and the gradients of both.
//
// dispatch: a stable counting sort of the assignments by expert.  Blocks of
// kSortChunk assignments count their experts, one block turns the counts into
// first rows (offsets, and per chunk), and the blocks place their assignments
// in order; then each token's row is read once and written to its top_k rows.
// combine and the gradients go token by token the other way: a token's row is
// held in registers while its top_k expert rows stream by, so every byte
// crosses HBM once.  No atomics on results: slots, sums and dot products are
// the same bits every time.
#include "common.cuh"
#include "ops.h"

namespace muon {

namespace {

// ---- the order ----

__device__ __forceinline__ int expert_of(const SortArgs& a, int64_t i) {
  const int64_t v = a.index_bits == 64 ? static_cast<const int64_t*>(a.indices)[i]
                                       : static_cast<const int32_t*>(a.indices)[i];
  return v >= 0 && v < a.experts ? (int)v : -1;
}

__global__ void __launch_bounds__(1024) k_sort_count(SortArgs a, int64_t n) {
  extern __shared__ int hist[];
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int64_t i = (int64_t)blockIdx.x * kSortChunk + threadIdx.x;
  const int e = i < n ? expert_of(a, i) : -1;
  if (e >= 0) atomicAdd(&hist[e], 1);  // whole numbers: the order of the additions does not show
  __syncthreads();
  for (int k = threadIdx.x; k < a.experts; k += blockDim.x)
    a.counts[(int64_t)blockIdx.x * a.experts + k] = hist[k];
}

// counts[c][e] becomes the row of the first assignment of chunk c to e.
__global__ void __launch_bounds__(1024) k_sort_scan(SortArgs a, int chunks) {
  __shared__ int total[1024 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = warp; e < a.experts; e += 32) {
    int sum = 0;
    for (int c0 = 0; c0 < chunks; c0 += 32) {
      const int c = c0 + lane;
      int v = c < chunks ? a.counts[(int64_t)c * a.experts + e] : 0;
      const int own = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (c < chunks) a.counts[(int64_t)c * a.experts + e] = sum + v - own;
      sum += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) total[e] = sum;
  }
  __syncthreads();
  if (warp == 0) {
    int base = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
      const int e = e0 + lane;
      int v = e < a.experts ? total[e] : 0;
      const int own = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (e < a.experts) a.offsets[e] = total[e] = base + v - own;
      base += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) a.offsets[a.experts] = base;
  }
  __syncthreads();
  for (int64_t i = threadIdx.x; i < (int64_t)chunks * a.experts; i += blockDim.x)
    a.counts[i] += total[i % a.experts];
}

__global__ void __launch_bounds__(1024) k_sort_place(SortArgs a, int64_t n) {
  extern __shared__ int next[];
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x)
    next[e] = a.counts[(int64_t)blockIdx.x * a.experts + e];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t i = (int64_t)blockIdx.x * kSortChunk + threadIdx.x;
  const int e = i < n ? expert_of(a, i) : -1;
  const unsigned same = __match_any_sync(0xffffffffu, e);
  const int before = __popc(same & ((1u << lane) - 1));
  __syncthreads();
  for (int w = 0; w < kSortChunk / 32; ++w) {  // warp by warp: the order of the assignments
    if (warp == w) {
      const int first = e >= 0 ? next[e] : 0;
      __syncwarp();
      if (e >= 0 && before == 0) next[e] = first + __popc(same);
      if (i < n) a.slot[i] = e >= 0 ? first + before : -1;
    }
    __syncthreads();
  }
}

// ---- rows ----

// 16 bytes of T as floats, or one element.
template <typename T, bool VEC>
struct Piece {
  static constexpr int N = VEC ? 16 / (int)sizeof(T) : 1;
  float f[N];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      const T* h = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = to_f32(h[i]);
    } else {
      f[0] = to_f32(*p);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC) {
      uint4 u;
      T* h = reinterpret_cast<T*>(&u);
#pragma unroll
      for (int i = 0; i < N; ++i) h[i] = from_f32<T>(f[i]);
      *reinterpret_cast<uint4*>(p) = u;
    } else {
      *p = from_f32<T>(f[0]);
    }
  }
};

constexpr int kRowThreads = 256;
constexpr int kMaxTopK = 32;

template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) k_gather(SortArgs a) {
  constexpr int N = Piece<T, VEC>::N;
  __shared__ int slot[kMaxTopK];
  const int64_t t = blockIdx.x;
  if (threadIdx.x < a.top_k) slot[threadIdx.x] = a.slot[t * a.top_k + threadIdx.x];
  const int64_t owned = a.offsets[a.experts];
  __syncthreads();
  const T* x = static_cast<const T*>(a.x) + t * a.x_stride;
  T* xs = static_cast<T*>(a.xs);
  for (int64_t h = (int64_t)threadIdx.x * N; h < a.hidden; h += kRowThreads * N) {
    Piece<T, VEC> v, zero{};
    v.load(x + h);
    for (int j = 0; j < a.top_k; ++j) {
      if (slot[j] >= 0) v.store(xs + (int64_t)slot[j] * a.hidden + h);
      const int64_t r = t * a.top_k + j;  // this block clears its share of the rows that no expert owns
      if (r >= owned) zero.store(xs + r * a.hidden + h);
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) k_combine(SortArgs a) {
  constexpr int N = Piece<T, VEC>::N;
  __shared__ int slot[kMaxTopK];
  __shared__ float wt[kMaxTopK];
  const int64_t t = blockIdx.x, rows = a.tokens * a.top_k;
  if (threadIdx.x < a.top_k) {
    const int s = a.slot[t * a.top_k + threadIdx.x];
    slot[threadIdx.x] = s < rows ? s : -1;
    wt[threadIdx.x] = a.weights ? a.weights[t * a.top_k + threadIdx.x] : 1.f;
  }
  __syncthreads();
  const T* ys = static_cast<const T*>(a.ys);
  for (int64_t h = (int64_t)threadIdx.x * N; h < a.hidden; h += kRowThreads * N) {
    Piece<T, VEC> sum{}, v;
    for (int j = 0; j < a.top_k; ++j) {
      if (slot[j] < 0) continue;
      v.load(ys + (int64_t)slot[j] * a.ys_stride + h);
#pragma unroll
      for (int i = 0; i < N; ++i) sum.f[i] = fmaf(wt[j], v.f[i], sum.f[i]);
    }
    if (a.residual) {
      v.load(static_cast<const T*>(a.residual) + t * a.r_stride + h);
#pragma unroll
      for (int i = 0; i < N; ++i) sum.f[i] += v.f[i];
    }
    sum.store(static_cast<T*>(a.y) + t * a.hidden + h);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) k_combine_backward(SortArgs a) {
  constexpr int N = Piece<T, VEC>::N;
  __shared__ int slot[kMaxTopK];
  __shared__ float wt[kMaxTopK], scratch[33];
  const int64_t t = blockIdx.x, rows = a.tokens * a.top_k;
  if (threadIdx.x < a.top_k) {
    const int s = a.slot[t * a.top_k + threadIdx.x];
    slot[threadIdx.x] = s < rows ? s : -1;
    wt[threadIdx.x] = a.weights[t * a.top_k + threadIdx.x];
  }
  int64_t owned = a.offsets[a.experts];
  if (owned < 0) owned = 0;
  __syncthreads();
  const T* dy = static_cast<const T*>(a.dy) + t * a.dy_stride;
  const T* ys = static_cast<const T*>(a.ys);
  T* dys = static_cast<T*>(a.dys);
  for (int j = 0; j < a.top_k; ++j) {
    float dot = 0.f;
    const int64_t r = t * a.top_k + j;
    for (int64_t h = (int64_t)threadIdx.x * N; h < a.hidden; h += kRowThreads * N) {
      Piece<T, VEC> d, v, zero{};
      d.load(dy + h);
      if (slot[j] >= 0) {
        v.load(ys + (int64_t)slot[j] * a.ys_stride + h);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          dot = fmaf(v.f[i], d.f[i], dot);
          d.f[i] *= wt[j];
        }
        d.store(dys + (int64_t)slot[j] * a.hidden + h);
      }
      if (r >= owned) zero.store(dys + r * a.hidden + h);
    }
    dot = block_sum(dot, scratch);
    if (threadIdx.x == 0) a.dweights[r] = dot;
  }
}

bool vec_ok(const void* p, int64_t stride, int64_t size) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (stride * size) % 16 == 0;
}

enum RowOp { OP_GATHER, OP_COMBINE, OP_COMBINE_BACKWARD };

template <typename T, bool VEC>
void launch_rows(RowOp op, const SortArgs& a, cudaStream_t s) {
  const unsigned grid = (unsigned)a.tokens;
  if (op == OP_GATHER) k_gather<T, VEC><<<grid, kRowThreads, 0, s>>>(a);
  else if (op == OP_COMBINE) k_combine<T, VEC><<<grid, kRowThreads, 0, s>>>(a);
  else k_combine_backward<T, VEC><<<grid, kRowThreads, 0, s>>>(a);
}

// 16-byte accesses where every row of every tensor starts on 16 bytes and has
// a whole number of pieces; single elements otherwise.
template <typename T>
cudaError_t rows_t(RowOp op, const SortArgs& a, cudaStream_t s) {
  const int64_t b = sizeof(T);
  const bool vec = (a.hidden * b) % 16 == 0 && vec_ok(a.x, a.x_stride, b) && vec_ok(a.xs, a.hidden, b) &&
                   vec_ok(a.ys, a.ys_stride, b) && vec_ok(a.residual, a.r_stride, b) &&
                   vec_ok(a.y, a.hidden, b) && vec_ok(a.dy, a.dy_stride, b) && vec_ok(a.dys, a.hidden, b);
  if (vec) launch_rows<T, true>(op, a, s);
  else launch_rows<T, false>(op, a, s);
  return cudaGetLastError();
}

cudaError_t rows(RowOp op, const SortArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case DT_F16: return rows_t<__half>(op, a, s);
    case DT_BF16: return rows_t<__nv_bfloat16>(op, a, s);
    default: return rows_t<float>(op, a, s);
  }
}

}  // namespace

cudaError_t launch_dispatch(const SortArgs& a, cudaStream_t s) {
  const int64_t n = a.tokens * a.top_k;
  const unsigned chunks = (unsigned)((n + kSortChunk - 1) / kSortChunk);
  const size_t smem = sizeof(int) * a.experts;
  if (chunks) k_sort_count<<<chunks, kSortChunk, smem, s>>>(a, n);
  k_sort_scan<<<1, 1024, 0, s>>>(a, (int)chunks);
  if (chunks) k_sort_place<<<chunks, kSortChunk, smem, s>>>(a, n);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && a.xs && a.tokens) e = rows(OP_GATHER, a, s);
  return e;
}

cudaError_t launch_combine(const SortArgs& a, cudaStream_t s) { return rows(OP_COMBINE, a, s); }

cudaError_t launch_combine_backward(const SortArgs& a, cudaStream_t s) {
  return rows(OP_COMBINE_BACKWARD, a, s);
}

}  // namespace muon
