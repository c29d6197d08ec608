// What the two products of a layer's gradient start from: dz = dy * act'(z),
// and the bias gradient, the column sums of dz over each expert's rows.
//
// In the 16-bit types dz is rounded to the operand type: the tensor cores take no
// other, and two parts (as fp32 tensors have) would double the products.  The
// rounding is at most 2^-8 (bf16) of an element, of either sign, so that dx and dw, sums
// over hundreds of them, carry about as much from it as from their own store: against
// 64 bits 2.35e-3 of the norm instead of 1.66e-3 ([4096, 4096 -> 16384], gelu_tanh).  In
// fp16 dz below 2^-24 becomes zero, as dy itself does; loss scaling keeps both away
// from there.  db is summed from the unrounded dz.
//
// One pass over dy and z, bound by HBM and, for the exponentials, by issue
// ([4096, 16384] bf16 with dz and db: silu 76 us, 5.3 TB/s; gelu_tanh 81, gelu 93).  A
// block takes kGradChunk rows and 32 pieces of columns (16 bytes each where rows
// allow it; element by element it took 212 us), eight threads to a
// column piece that take every eighth row.  The part of the sum that chunk c
// adds to range e goes to row c + e of `part` (along the rows c and e only
// grow, so no two pairs share a row), and a second kernel adds each range's
// parts in row order: the same bits every time, and no atomics.  Up to
// kGradSingle rows are one chunk, whose sums are the result.
#include "act.cuh"
#include "common.cuh"

namespace muon {

namespace {

constexpr int kLanes = 32, kRowLanes = 8;

__device__ __forceinline__ int64_t off_at(const GradPrep& g, int e) {
  if (g.experts == 0) return e ? g.rows : 0;
  const int64_t v = g.offsets[e];
  return v < 0 ? 0 : (v > g.rows ? g.rows : v);
}

template <typename T, int VEC>
__device__ __forceinline__ void load(const T* p, float* f) {
  if constexpr (VEC == 1) {
    f[0] = to_f32(*p);
  } else {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));  // read once
    const T* h = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = to_f32(h[i]);
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T* p, const float* f) {
  if constexpr (VEC == 1) {
    *p = from_f32<T>(f[0]);
  } else {
    uint4 u;
    T* h = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < VEC; ++i) h[i] = from_f32<T>(f[i]);
    *reinterpret_cast<uint4*>(p) = u;
  }
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kLanes* kRowLanes) k_grad_prep(GradPrep g, int col_blocks) {
  constexpr bool kFast = sizeof(T) == 2;
  __shared__ float red[kRowLanes][kLanes * VEC];
  grid_launch_next();
  grid_wait();
  const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int64_t chunk = blockIdx.x / col_blocks;
  const int64_t col = ((int64_t)(blockIdx.x % col_blocks) * kLanes + lane) * VEC;
  const bool live = col < g.cols;
  const bool single = g.rows <= kGradSingle;
  const int64_t r0 = single ? 0 : chunk * kGradChunk, r1 = single ? g.rows : min(r0 + kGradChunk, g.rows);
  const T* dy = static_cast<const T*>(g.dy) + col;
  const T* z = static_cast<const T*>(g.z) + col;
  T* dz = static_cast<T*>(g.dz);
  const int ranges = g.experts ? g.experts : 1;
  int e = 0;
  if (g.experts) {  // the first range that ends behind r0
    int hi = ranges;
    while (e < hi) {
      const int m = (e + hi) / 2;
      if (off_at(g, m + 1) > r0) hi = m;
      else e = m + 1;
    }
  }
  if (single) e = 0;  // empty ranges too: their sums are stored here
  // the chunk's rows range by range; rows of no expert are left out
  for (int64_t a = max(r0, off_at(g, 0)); e < ranges && (a < r1 || (single && g.db)); ++e) {
    const int64_t b = min(off_at(g, e + 1), r1);
    float sum[VEC] = {};
    if (live) {
#pragma unroll 4
      for (int64_t r = a + rl; r < b; r += kRowLanes) {
        float v[VEC];
        load<T, VEC>(dy + r * g.dy_stride, v);
        if constexpr (ACT != ACT_NONE) {
          float zz[VEC];
          load<T, VEC>(z + r * g.cols, zz);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[i] *= act_slope<kFast>(zz[i], ACT);
          if (dz) store<T, VEC>(dz + r * g.dz_stride + col, v);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] += v[i];
      }
    }
    if (g.db && (b > a || single)) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) red[rl][i * kLanes + lane] = sum[i];
      __syncthreads();
      for (int i = threadIdx.x; i < kLanes * VEC; i += kLanes * kRowLanes) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kRowLanes; ++k) s += red[k][i];
        const int64_t c = ((int64_t)(blockIdx.x % col_blocks) * kLanes + i % kLanes) * VEC + i / kLanes;
        if (c >= g.cols) continue;
        if (single) static_cast<T*>(g.db)[e * g.cols + c] = from_f32<T>(s);
        else g.part[(chunk + e) * g.cols + c] = s;
      }
      __syncthreads();
    }
    if (b > a) a = b;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) k_grad_bias(GradPrep g, int col_blocks) {
  const int64_t col = (int64_t)(blockIdx.x % col_blocks) * 256 + threadIdx.x;
  const int e = blockIdx.x / col_blocks;
  grid_launch_next();
  grid_wait();
  if (col >= g.cols) return;
  const int64_t lo = off_at(g, e), hi = off_at(g, e + 1);
  float sum = 0.f;
  if (hi > lo) {
    const float* part = g.part + e * g.cols + col;
    const int64_t last = (hi - 1) / kGradChunk;
#pragma unroll 8
    for (int64_t c = lo / kGradChunk; c <= last; ++c) sum += part[c * g.cols];
  }
  static_cast<T*>(g.db)[(int64_t)e * g.cols + col] = from_f32<T>(sum);
}

template <typename T, int VEC>
cudaError_t prep(const GradPrep& g, cudaStream_t s) {
  const int cb = (int)((g.cols + kLanes * VEC - 1) / (kLanes * VEC));
  const int64_t chunks = g.rows <= kGradSingle ? 1 : (g.rows + kGradChunk - 1) / kGradChunk;
  const dim3 grid((unsigned)(chunks * cb)), block(kLanes * kRowLanes);
  switch (g.act) {
    case ACT_RELU: return launch_early(k_grad_prep<T, VEC, ACT_RELU>, grid, block, 0, s, g, cb);
    case ACT_SILU: return launch_early(k_grad_prep<T, VEC, ACT_SILU>, grid, block, 0, s, g, cb);
    case ACT_GELU: return launch_early(k_grad_prep<T, VEC, ACT_GELU>, grid, block, 0, s, g, cb);
    case ACT_GELU_TANH: return launch_early(k_grad_prep<T, VEC, ACT_GELU_TANH>, grid, block, 0, s, g, cb);
    default: return launch_early(k_grad_prep<T, VEC, ACT_NONE>, grid, block, 0, s, g, cb);
  }
}

template <typename T>
cudaError_t run(const GradPrep& g, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const auto ok = [](const void* p, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % V == 0;
  };
  // 16-byte pieces where every row of every tensor starts on 16 bytes
  const bool vec = g.cols % V == 0 && ok(g.dy, g.dy_stride) && ok(g.z, g.cols) && ok(g.dz, g.dz_stride);
  cudaError_t e = vec ? prep<T, V>(g, s) : prep<T, 1>(g, s);
  if (e == cudaSuccess && g.db && g.rows > kGradSingle) {
    const int cb = (int)((g.cols + 255) / 256);
    e = launch_early(k_grad_bias<T>, dim3((unsigned)cb * (g.experts ? g.experts : 1)), dim3(256), 0, s, g, cb);
  }
  return e;
}

}  // namespace

cudaError_t launch_grad_prep(const GradPrep& g, cudaStream_t s) {
  switch (g.dtype) {
    case DT_F16: return run<__half>(g, s);
    case DT_BF16: return run<__nv_bfloat16>(g, s);
    default: return run<float>(g, s);
  }
}

}  // namespace muon
