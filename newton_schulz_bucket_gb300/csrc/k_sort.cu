// Token rows into expert order and back, and the gradients of both.
//
// dispatch: a stable counting sort of the assignments by expert.  Blocks of
// kSortChunk assignments count their experts, a scan turns the counts into
// first rows, and the blocks place their assignments in order; up to kSortCluster
// assignments one cluster of blocks does all that in one launch.  Then each
// token's row is read once and written to its top_k rows.  Up to kSortChunk
// assignments order and rows take one launch together.
// combine and the gradients go token by token the other way: a token's row is
// held in registers while its top_k expert rows stream by, so every byte
// crosses HBM once.  No atomics on results: slots, sums and dot products are
// the same bits every time.  Bound by HBM for many tokens: 8192 tokens to eight
// experts each, hidden 7168 bf16, 175 us there with the order (6.0 TB/s), 156 us
// back (6.8), 299 us for the gradient of the way back (6.7).
#include <mutex>
#include <type_traits>

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
  grid_launch_next();
  grid_wait();
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int64_t i = (int64_t)blockIdx.x * kSortChunk + threadIdx.x;
  const int e = i < n ? expert_of(a, i) : -1;
  if (e >= 0) atomicAdd(&hist[e], 1);  // whole numbers: the order of the additions does not show
  __syncthreads();
  for (int k = threadIdx.x; k < a.experts; k += blockDim.x)
    a.counts[(int64_t)blockIdx.x * a.experts + k] = hist[k];
}

// counts[c][e] becomes the number of e's assignments before chunk c, total[e]
// that of all.  A block takes 32 experts (one a lane, so that loads run along
// the table's rows) and each of its 32 warps a run of chunks.
__global__ void __launch_bounds__(1024) k_sort_scan(SortArgs a, int chunks) {
  grid_launch_next();
  grid_wait();
  __shared__ int sum[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  const bool live = e < a.experts;
  const int c0 = (int)((int64_t)chunks * warp / 32), c1 = (int)((int64_t)chunks * (warp + 1) / 32);
  int* col = a.counts + e;
  int s = 0;
  if (live) {
#pragma unroll 8
    for (int c = c0; c < c1; ++c) s += col[(int64_t)c * a.experts];
  }
  sum[warp][lane] = s;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += sum[w][lane];
  if (!live) return;
  for (int c = c0; c < c1; ++c) {
    const int n = col[(int64_t)c * a.experts];
    col[(int64_t)c * a.experts] = before;
    before += n;
  }
  if (warp == 31) a.total[e] = before;
}

// Exclusive prefix of v over a block of 1024 threads (warp totals in w).
__device__ __forceinline__ int block_prefix(int v, int* w) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) w[warp] = incl;
  __syncthreads();
  int before = 0;
  for (int k = 0; k < warp; ++k) before += w[k];
  return before + incl - v;
}

// Slots of 1024 assignments, i this thread's and e its expert (-1: none), in
// order: next[e] is e's first free row, before and after.  Each warp counts its
// own (equal lanes vote), a prefix over the warps makes the counts stable.
// warp_count: [32][experts].
__device__ __forceinline__ void place_round(const SortArgs& a, int64_t i, int64_t n, int e, int* next,
                                            uint16_t* warp_count) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int k = threadIdx.x; k < 32 * a.experts; k += 1024) warp_count[k] = 0;
  const unsigned same = __match_any_sync(0xffffffffu, e);
  const int before = __popc(same & ((1u << lane) - 1));
  __syncthreads();
  if (e >= 0 && before == 0) warp_count[warp * a.experts + e] = (uint16_t)__popc(same);
  __syncthreads();
  for (int k = threadIdx.x; k < a.experts; k += 1024) {
    int sum = 0;
#pragma unroll 8
    for (int w = 0; w < 32; ++w) {
      const int c = warp_count[w * a.experts + k];
      warp_count[w * a.experts + k] = (uint16_t)sum;  // at most 1024
      sum += c;
    }
    next[k] += sum;  // the round's own first row is next - sum
    warp_count[32 * a.experts + k] = (uint16_t)sum;
  }
  __syncthreads();
  if (i < n)
    a.slot[i] = e >= 0 ? next[e] - warp_count[32 * a.experts + e] + warp_count[warp * a.experts + e] + before : -1;
  __syncthreads();
}
size_t place_smem(int experts) { return sizeof(int) * experts + sizeof(uint16_t) * 33 * experts; }

__global__ void __launch_bounds__(1024) k_sort_place(SortArgs a, int64_t n) {
  extern __shared__ int next[];
  __shared__ int warps[32];
  grid_launch_next();
  const int tid = threadIdx.x;
  grid_wait();
  {
    const int count = tid < a.experts ? a.total[tid] : 0;
    const int first = block_prefix(count, warps);  // the expert's first row
    if (tid < a.experts) {
      next[tid] = first + a.counts[(int64_t)blockIdx.x * a.experts + tid];
      if (blockIdx.x == 0) {
        a.offsets[tid] = first;
        if (tid == a.experts - 1) a.offsets[a.experts] = first + count;
      }
    }
  }
  const int64_t i = (int64_t)blockIdx.x * kSortChunk + tid;
  place_round(a, i, n, i < n ? expert_of(a, i) : -1, next, reinterpret_cast<uint16_t*>(next + a.experts));
}

// The whole order in one launch, for up to kSortCluster assignments: a cluster of
// eight blocks, each with a run of them.  Counts meet in distributed shared
// memory instead of scratch.
constexpr int kClusterBlocks = 8;
__global__ void __launch_bounds__(1024) k_sort_cluster(SortArgs a, int64_t n) {
  extern __shared__ int next[];  // [experts] rows, [experts] counts, then place_round's
  __shared__ int warps[32];
  int* hist = next + a.experts;
  grid_launch_next();
  const int tid = threadIdx.x, rank = blockIdx.x;
  const int64_t per = (n + kClusterBlocks * kSortChunk - 1) / (kClusterBlocks * kSortChunk) * kSortChunk;
  const int64_t i0 = rank * per, i1 = min(i0 + per, n);
  for (int e = tid; e < a.experts; e += 1024) hist[e] = 0;
  __syncthreads();
  grid_wait();
  for (int64_t i = i0 + tid; i < i1; i += 1024) {
    const int e = expert_of(a, i);
    if (e >= 0) atomicAdd(&hist[e], 1);  // whole numbers: the order of the additions does not show
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  int total = 0, before = 0;
  if (tid < a.experts) {
    const uint32_t local = (uint32_t)__cvta_generic_to_shared(hist + tid);
#pragma unroll
    for (int r = 0; r < kClusterBlocks; ++r) {
      uint32_t remote;
      int v;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(r));
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
      before += r < rank ? v : 0;
      total += v;
    }
  }
  // no block leaves, or reuses its counts, while another reads them
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  const int first = block_prefix(total, warps);
  if (tid < a.experts) {
    next[tid] = first + before;
    if (rank == 0) {
      a.offsets[tid] = first;
      if (tid == a.experts - 1) a.offsets[a.experts] = first + total;
    }
  }
  for (int64_t c = i0; c < i0 + per; c += kSortChunk) {  // the same rounds for every thread of the block
    const int64_t i = c + tid;
    place_round(a, i, i1, i < i1 ? expert_of(a, i) : -1, next, reinterpret_cast<uint16_t*>(hist + a.experts));
  }
}

// ---- rows ----

// 16 bytes of T, or one element, as floats.
template <typename T, bool VEC>
struct Piece {
  static constexpr int N = VEC ? 16 / (int)sizeof(T) : 1;
  using Raw = typename std::conditional<VEC, uint4, T>::type;
  float f[N];
  // Rows that are read once are marked so: 8192 tokens' rows of 8 experts, hidden
  // 7168, come back in 159 us this way (98% of the copy rate), else in 193.
  static __device__ __forceinline__ Raw fetch(const T* p) {
    if constexpr (VEC) return __ldcs(reinterpret_cast<const uint4*>(p));
    else return *p;
  }
  __device__ __forceinline__ void open(const Raw& u) {
    const T* h = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f32(h[i]);
  }
  __device__ __forceinline__ void load(const T* p) { open(fetch(p)); }
  // kStream: the top_k times larger outputs, which no cache holds for a reader.
  template <bool kStream = false>
  __device__ __forceinline__ void store(T* p) const {
    Raw u;
    T* h = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = from_f32<T>(f[i]);
    if constexpr (VEC && kStream) __stcs(reinterpret_cast<uint4*>(p), u);
    else *reinterpret_cast<Raw*>(p) = u;
  }
};

constexpr int kMaxTopK = 32;
constexpr int kTogether = 8;  // expert rows a thread has in flight

// A block works on one token's rows, or on one of gridDim.y shares of their
// pieces where the tokens are too few to fill the GPU.
struct Span {
  int64_t h, end, step;
};
template <int N>
__device__ __forceinline__ Span my_span(int64_t hidden) {
  const int64_t pieces = hidden / N, per = (pieces + gridDim.y - 1) / gridDim.y;
  const int64_t p0 = per * blockIdx.y, p1 = min(p0 + per, pieces);
  return {(p0 + threadIdx.x) * N, p1 * N, (int64_t)blockDim.x * N};
}

// x[t] to its rows; the block's share of the rows that no expert owns to zero.
template <typename T, bool VEC>
__device__ __forceinline__ void spread_row(const SortArgs& a, int64_t t, const int* slot, int64_t owned) {
  constexpr int N = Piece<T, VEC>::N;
  const T* x = static_cast<const T*>(a.x) + t * a.x_stride;
  T* xs = static_cast<T*>(a.xs);
  const int64_t r0 = t * a.top_k;
  for (Span s = my_span<N>(a.hidden); s.h < s.end; s.h += s.step) {
    Piece<T, VEC> v, zero{};
    v.load(x + s.h);
    for (int j = 0; j < a.top_k; ++j)
      if (slot[j] >= 0) v.store(xs + (int64_t)slot[j] * a.hidden + s.h);
    for (int j = a.top_k - 1; j >= 0 && r0 + j >= owned; --j) zero.store(xs + (r0 + j) * a.hidden + s.h);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(128) k_gather(SortArgs a) {
  __shared__ int slot[kMaxTopK];
  grid_launch_next();
  grid_wait();
  const int64_t t = blockIdx.x;
  if (threadIdx.x < a.top_k) slot[threadIdx.x] = a.slot[t * a.top_k + threadIdx.x];
  const int64_t owned = a.offsets[a.experts];
  __syncthreads();
  spread_row<T, VEC>(a, t, slot, owned);
}

// dispatch in one launch, for at most kSortChunk assignments: every block looks
// at all of them and counts its token's slots (assignments to lower experts, or
// to the same one earlier) instead of sorting.  Block row `tokens` does the
// offsets.
template <typename T, bool VEC>
__global__ void __launch_bounds__(128) k_dispatch_small(SortArgs a) {
  __shared__ int ex[kSortChunk], hist[1024], slot[kMaxTopK], valid;
  const int n = (int)(a.tokens * a.top_k), tid = threadIdx.x;
  grid_launch_next();
  grid_wait();
  if (tid < kMaxTopK) slot[tid] = 0;
  if (tid == 0) valid = 0;
  for (int i = tid; i < n; i += blockDim.x) ex[i] = expert_of(a, i);
  __syncthreads();
  const int64_t t = blockIdx.x;
  if (t == a.tokens) {
    if (blockIdx.y) return;
    for (int e = tid; e < a.experts; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += blockDim.x)
      if (ex[i] >= 0) atomicAdd(&hist[ex[i]], 1);
    __syncthreads();
    if (tid >= 32) return;
    int base = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
      const int own = e0 + tid < a.experts ? hist[e0 + tid] : 0;
      int incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (tid >= o) incl += u;
      }
      if (e0 + tid < a.experts) a.offsets[e0 + tid] = base + incl - own;
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (tid == 0) a.offsets[a.experts] = base;
    return;
  }
  const int i0 = (int)t * a.top_k;
  int live = 0;
  for (int i = tid; i < n; i += blockDim.x) live += ex[i] >= 0;
  if (live) atomicAdd(&valid, live);  // whole numbers
  for (int j = 0; j < a.top_k; ++j) {
    const int e = ex[i0 + j];
    int c = 0;
    for (int i = tid; i < n; i += blockDim.x) c += ex[i] >= 0 && (ex[i] < e || (ex[i] == e && i < i0 + j));
    if (c) atomicAdd(&slot[j], c);
  }
  __syncthreads();
  if (tid < a.top_k) {
    if (ex[i0 + tid] < 0) slot[tid] = -1;
    if (blockIdx.y == 0) a.slot[i0 + tid] = slot[tid];
  }
  __syncthreads();
  if (a.xs) spread_row<T, VEC>(a, t, slot, valid);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(128) k_combine(SortArgs a) {
  constexpr int N = Piece<T, VEC>::N;
  __shared__ int slot[kMaxTopK];
  __shared__ float wt[kMaxTopK];
  grid_launch_next();
  grid_wait();
  const int64_t t = blockIdx.x, rows = a.tokens * a.top_k;
  if (threadIdx.x < kMaxTopK) {
    const bool in = threadIdx.x < a.top_k;
    const int s = in ? a.slot[t * a.top_k + threadIdx.x] : -1;
    slot[threadIdx.x] = s < rows ? s : -1;
    wt[threadIdx.x] = in ? (a.weights ? a.weights[t * a.top_k + threadIdx.x] : 1.f) : 0.f;
  }
  __syncthreads();
  const T* ys = static_cast<const T*>(a.ys);
  for (Span s = my_span<N>(a.hidden); s.h < s.end; s.h += s.step) {
    Piece<T, VEC> sum{}, r{};
    if (a.residual) r.load(static_cast<const T*>(a.residual) + t * a.r_stride + s.h);
    for (int j0 = 0; j0 < a.top_k; j0 += kTogether) {
      typename Piece<T, VEC>::Raw u[kTogether];
#pragma unroll
      for (int j = 0; j < kTogether; ++j)
        if (slot[j0 + j] >= 0) u[j] = Piece<T, VEC>::fetch(ys + (int64_t)slot[j0 + j] * a.ys_stride + s.h);
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        if (slot[j0 + j] < 0) continue;
        Piece<T, VEC> v;
        v.open(u[j]);
#pragma unroll
        for (int i = 0; i < N; ++i) sum.f[i] = fmaf(wt[j0 + j], v.f[i], sum.f[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) sum.f[i] += r.f[i];
    sum.store(static_cast<T*>(a.y) + t * a.hidden + s.h);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(128) k_combine_backward(SortArgs a) {
  constexpr int N = Piece<T, VEC>::N;
  __shared__ int slot[kMaxTopK];
  __shared__ float wt[kMaxTopK], part[4][kTogether];
  grid_launch_next();
  grid_wait();
  const int64_t t = blockIdx.x, rows = a.tokens * a.top_k, r0 = t * a.top_k;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < kMaxTopK) {
    const bool in = threadIdx.x < a.top_k;
    const int s = in ? a.slot[r0 + threadIdx.x] : -1;
    slot[threadIdx.x] = s < rows ? s : -1;
    wt[threadIdx.x] = in ? a.weights[r0 + threadIdx.x] : 0.f;
  }
  const int64_t owned = max(a.offsets[a.experts], 0);
  __syncthreads();
  const T* dy = static_cast<const T*>(a.dy) + t * a.dy_stride;
  const T* ys = static_cast<const T*>(a.ys);
  T* dys = static_cast<T*>(a.dys);
  for (int j0 = 0; j0 < a.top_k; j0 += kTogether) {
    float dot[kTogether] = {};
    for (int64_t h = (int64_t)threadIdx.x * N; h < a.hidden; h += (int64_t)blockDim.x * N) {
      Piece<T, VEC> d;
      typename Piece<T, VEC>::Raw u[kTogether];
#pragma unroll
      for (int j = 0; j < kTogether; ++j)
        if (slot[j0 + j] >= 0) u[j] = Piece<T, VEC>::fetch(ys + (int64_t)slot[j0 + j] * a.ys_stride + h);
      d.load(dy + h);
#pragma unroll
      for (int j = 0; j < kTogether; ++j) {
        if (slot[j0 + j] < 0) continue;
        Piece<T, VEC> v;
        v.open(u[j]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          dot[j] = fmaf(v.f[i], d.f[i], dot[j]);
          v.f[i] = wt[j0 + j] * d.f[i];
        }
        v.template store<true>(dys + (int64_t)slot[j0 + j] * a.hidden + h);
      }
      for (int64_t r = r0 + a.top_k - 1; j0 == 0 && r >= r0 && r >= owned; --r) {
        Piece<T, VEC> zero{};
        zero.store(dys + r * a.hidden + h);
      }
    }
#pragma unroll
    for (int j = 0; j < kTogether; ++j) {
      const float w = warp_sum(dot[j]);
      if (lane == 0) part[warp][j] = w;
    }
    __syncthreads();
    if (threadIdx.x < kTogether && j0 + threadIdx.x < a.top_k) {
      float s = 0.f;
      for (int w = 0; w < (int)blockDim.x / 32; ++w) s += part[w][threadIdx.x];
      a.dweights[r0 + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

bool vec_ok(const void* p, int64_t stride, int64_t size) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (stride * size) % 16 == 0;
}

enum RowOp { OP_GATHER, OP_DISPATCH_SMALL, OP_COMBINE, OP_COMBINE_BACKWARD };

template <typename T, bool VEC>
cudaError_t launch_rows(RowOp op, const SortArgs& a, cudaStream_t s) {
  constexpr int N = Piece<T, VEC>::N;
  const int64_t pieces = (a.hidden + N - 1) / N;
  // enough blocks to fill the GPU (a token's dot products stay in one block; without
  // tokens there are no rows to share out)
  int64_t y = 1;
  if (op != OP_COMBINE_BACKWARD && a.tokens > 0) {
    while (a.tokens * y < 304 && pieces / (2 * y) >= 32) y *= 2;
  }
  // up to four warps (more blocks an SM, at different points: combine 166 -> 159 us
  // against eight) that divide a block's pieces into even rounds
  const int64_t per = (pieces + y - 1) / y, rounds = (per + 127) / 128;
  unsigned threads = (unsigned)(((per + rounds - 1) / rounds + 31) / 32 * 32);
  if (op == OP_DISPATCH_SMALL) threads = 128;  // they count assignments first
  const dim3 grid((unsigned)(a.tokens + (op == OP_DISPATCH_SMALL)), (unsigned)y), block(threads);
  if (op == OP_GATHER) return launch_early(k_gather<T, VEC>, grid, block, 0, s, a);
  if (op == OP_DISPATCH_SMALL) return launch_early(k_dispatch_small<T, VEC>, grid, block, 0, s, a);
  if (op == OP_COMBINE) return launch_early(k_combine<T, VEC>, grid, block, 0, s, a);
  return launch_early(k_combine_backward<T, VEC>, grid, block, 0, s, a);
}

// 16-byte accesses where every row of every tensor starts on 16 bytes and has
// a whole number of pieces; single elements otherwise.
template <typename T>
cudaError_t rows_t(RowOp op, const SortArgs& a, cudaStream_t s) {
  const int64_t b = sizeof(T);
  const bool vec = (a.hidden * b) % 16 == 0 && vec_ok(a.x, a.x_stride, b) && vec_ok(a.xs, a.hidden, b) &&
                   vec_ok(a.ys, a.ys_stride, b) && vec_ok(a.residual, a.r_stride, b) &&
                   vec_ok(a.y, a.hidden, b) && vec_ok(a.dy, a.dy_stride, b) && vec_ok(a.dys, a.hidden, b);
  return vec ? launch_rows<T, true>(op, a, s) : launch_rows<T, false>(op, a, s);
}

cudaError_t rows(RowOp op, const SortArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case DT_F16: return rows_t<__half>(op, a, s);
    case DT_BF16: return rows_t<__nv_bfloat16>(op, a, s);
    default: return rows_t<float>(op, a, s);
  }
}

}  // namespace

// Shared memory beyond the default for many experts (once per device).
static cudaError_t prepare_sort() {
  static bool ready[64] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 64 && ready[dev]) return cudaSuccess;
  const int most = (int)(place_smem(1024) + sizeof(int) * 1024);
  e = cudaFuncSetAttribute(k_sort_place, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_sort_cluster, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess && dev < 64) ready[dev] = true;
  return e;
}

cudaError_t launch_dispatch(const SortArgs& a, cudaStream_t s) {
  const int64_t n = a.tokens * a.top_k;
  if (n <= kSortChunk) return rows(OP_DISPATCH_SMALL, a, s);
  cudaError_t e = prepare_sort();
  if (e != cudaSuccess) return e;
  SortArgs b = a;
  if (n <= kSortCluster) {
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(kClusterBlocks);
    lc.blockDim = dim3(1024);
    lc.dynamicSmemBytes = place_smem(a.experts) + sizeof(int) * a.experts;
    lc.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kClusterBlocks;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 2;
    e = cudaLaunchKernelEx(&lc, k_sort_cluster, b, n);
  } else {
    const unsigned chunks = (unsigned)((n + kSortChunk - 1) / kSortChunk);
    b.total = a.counts + (int64_t)chunks * a.experts;
    e = launch_early(k_sort_count, dim3(chunks), dim3(kSortChunk), sizeof(int) * a.experts, s, b, n);
    if (e == cudaSuccess)
      e = launch_early(k_sort_scan, dim3((a.experts + 31) / 32), dim3(1024), 0, s, b, (int)chunks);
    if (e == cudaSuccess) e = launch_early(k_sort_place, dim3(chunks), dim3(kSortChunk), place_smem(a.experts), s, b, n);
  }
  if (e == cudaSuccess && a.xs) e = rows(OP_GATHER, b, s);
  return e;
}

cudaError_t launch_combine(const SortArgs& a, cudaStream_t s) { return rows(OP_COMBINE, a, s); }

cudaError_t launch_combine_backward(const SortArgs& a, cudaStream_t s) {
  return rows(OP_COMBINE_BACKWARD, a, s);
}

}  // namespace muon
