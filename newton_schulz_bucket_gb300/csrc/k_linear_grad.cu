// What the two products of a layer's gradient start from: dz = dy * act'(z),
// and the bias gradient, the column sums of dz over each expert's rows.
//
// One pass over dy and z.  A block takes kGradChunk rows and 256 columns; the
// part of the sum that its chunk c adds to range e goes to row c + e of
// `part` (along the rows c and e only grow, so no two pairs share a row), and
// a second kernel adds each range's parts in row order: the same bits every
// time, and no atomics.
#include "act.cuh"
#include "common.cuh"

namespace muon {

namespace {

__device__ __forceinline__ int64_t off_at(const GradPrep& g, int e) {
  if (g.experts == 0) return e ? g.rows : 0;
  const int64_t v = g.offsets[e];
  return v < 0 ? 0 : (v > g.rows ? g.rows : v);
}

template <typename T>
__global__ void __launch_bounds__(256) k_grad_prep(GradPrep g) {
  constexpr bool kFast = sizeof(T) == 2;
  const int64_t col = (int64_t)blockIdx.y * 256 + threadIdx.x;
  const int64_t r0 = (int64_t)blockIdx.x * kGradChunk;
  const int64_t r1 = r0 + kGradChunk < g.rows ? r0 + kGradChunk : g.rows;
  if (col >= g.cols) return;
  const T* dy = static_cast<const T*>(g.dy);
  const T* z = static_cast<const T*>(g.z);
  T* dz = static_cast<T*>(g.dz);
  const int ranges = g.experts ? g.experts : 1;
  int e = 0;
  while (e < ranges && off_at(g, e + 1) <= r0) ++e;  // the range of row r0
  int64_t end = e < ranges ? off_at(g, e + 1) : g.rows;
  float sum = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    while (r >= end && e < ranges) {
      if (g.part) g.part[((int64_t)blockIdx.x + e) * g.cols + col] = sum;
      sum = 0.f;
      ++e;
      end = e < ranges ? off_at(g, e + 1) : g.rows;
    }
    float v = to_f32(dy[r * g.dy_stride + col]);
    if (g.act != ACT_NONE) {
      v *= act_slope<kFast>(to_f32(z[r * g.cols + col]), g.act);
      if (dz) dz[r * g.dz_stride + col] = from_f32<T>(v);
    }
    sum += v;
  }
  if (g.part && e < ranges) g.part[((int64_t)blockIdx.x + e) * g.cols + col] = sum;
}

template <typename T>
__global__ void __launch_bounds__(256) k_grad_bias(GradPrep g) {
  const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int e = blockIdx.y;
  if (col >= g.cols) return;
  const int64_t lo = off_at(g, e), hi = off_at(g, e + 1);
  float sum = 0.f;
  if (hi > lo)
    for (int64_t c = lo / kGradChunk; c <= (hi - 1) / kGradChunk; ++c) sum += g.part[(c + e) * g.cols + col];
  static_cast<T*>(g.db)[(int64_t)e * g.cols + col] = from_f32<T>(sum);
}

template <typename T>
cudaError_t run(const GradPrep& g, cudaStream_t s) {
  const unsigned cols = (unsigned)((g.cols + 255) / 256);
  const unsigned chunks = (unsigned)((g.rows + kGradChunk - 1) / kGradChunk);
  k_grad_prep<T><<<dim3(chunks, cols), 256, 0, s>>>(g);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && g.db) {
    k_grad_bias<T><<<dim3(cols, g.experts ? g.experts : 1), 256, 0, s>>>(g);
    e = cudaGetLastError();
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
