// Rows into microscaled 4-bit numbers and back (mx.cuh): weights once, activations
// in every product, along the sum.
//
// Numbers stored along the sum: four lanes share a block of 32, eight numbers each,
// so that loads and stores are whole lines.  Weights stored across the sum go through
// a tile of 256 steps of it by 64 columns: a lane takes 32 steps of two neighbouring
// columns, so that it has a block to itself, and the packed rows meet in shared
// memory.  Bound by HBM.
#include "common.cuh"
#include "mx.cuh"
#include "ops.h"

namespace muon {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;         // rows of a thread, in flight together

template <typename T>
__device__ __forceinline__ void fetch8(const T* p, int64_t n, bool vec, float* f) {
  if (vec && n >= 8) {
#pragma unroll
    for (int c = 0; c < (int)sizeof(T) / 2; ++c) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p) + c);  // read once
      const T* h = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int i = 0; i < 16 / (int)sizeof(T); ++i) f[c * (16 / sizeof(T)) + i] = to_f32(h[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}

// Where a thread of the row kernels works: its piece of eight columns, its first row.
struct Spot {
  int64_t piece, row;
  int by;                        // rows between a thread's rows
};
__device__ __forceinline__ Spot spot(const MxRows& q) {
  const int across = 1 << q.log_across, down = kThreads >> q.log_across;
  const int64_t cb = blockIdx.x % q.col_blocks, rb = blockIdx.x / q.col_blocks;
  return {cb * across + (threadIdx.x & (across - 1)), rb * down * kRows + (threadIdx.x >> q.log_across), down};
}

// (rows counts those of all matrices; one row after the other in the outputs)
template <typename T>
__global__ void __launch_bounds__(kThreads) k_mx_quantize_rows(MxRows q) {
  grid_launch_next();
  grid_wait();
  const Spot at = spot(q);
  const int64_t col = at.piece * 8, kb = (q.cols + kMxBlock - 1) / kMxBlock;
  const bool there = at.piece < 4 * kb;
  float f[kRows][8];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t row = at.row + k * at.by;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[k][i] = 0.f;
    if (!there || row >= q.rows) continue;
    const int64_t mat = q.mat_rows == q.rows ? 0 : row / q.mat_rows;
    fetch8(static_cast<const T*>(q.src) + mat * q.batch_stride + (row - mat * q.mat_rows) * q.stride + col, q.cols - col,
           q.vec, f[k]);
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    uint32_t s;
    const uint32_t v = mx_quantize8(f[k], &s);
    const int64_t row = at.row + k * at.by;
    if (!there || row >= q.rows) continue;
    *reinterpret_cast<uint32_t*>(q.values + (row * kb * 4 + at.piece) * 4) = v;
    if ((at.piece & 3) == 0) q.scales[row * q.scale_pitch + at.piece / 4] = (uint8_t)s;
  }
}

// Two neighbouring columns of one row of a matrix stored across the sum.
template <typename T>
struct Two {
  T v[2];
  __device__ __forceinline__ void fetch(const T* p, int n, bool vec) {
    if (vec && n >= 2) {
      if constexpr (sizeof(T) == 4) *reinterpret_cast<uint2*>(v) = __ldcs(reinterpret_cast<const uint2*>(p));
      else *reinterpret_cast<uint32_t*>(v) = __ldcs(reinterpret_cast<const uint32_t*>(p));
    } else {
      v[0] = n > 0 ? p[0] : from_f32<T>(0.f);
      v[1] = n > 1 ? p[1] : from_f32<T>(0.f);
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) k_mx_quantize_across(MxRows q, int in_tiles, int out_tiles) {
  __shared__ uint4 vals[64][8];  // [column][block ^ (column / 2 & 7)]
  __shared__ uint8_t scale[64][8];
  grid_launch_next();
  grid_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t b = blockIdx.x;
  const int64_t o0 = b % out_tiles * 64, kb = (q.cols + kMxBlock - 1) / kMxBlock;
  b /= out_tiles;
  const int64_t b0 = b % in_tiles * 8, mat = b / in_tiles;
  const int64_t i0 = (b0 + warp) * kMxBlock, o = o0 + 2 * lane;
  const int n = (int)max((int64_t)0, min((int64_t)2, q.mat_rows - o));  // the lane's columns
  const int steps = (int)max((int64_t)0, min((int64_t)kMxBlock, q.cols - i0));
  const T* src = static_cast<const T*>(q.src) + mat * q.batch_stride + i0 * q.stride + o;
  Two<T> t[kMxBlock];
#pragma unroll
  for (int i = 0; i < kMxBlock; ++i) t[i].fetch(src + i * q.stride, i < steps ? n : 0, q.vec);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i) top = max(top, __float_as_uint(to_f32(t[i].v[c])) & 0x7fffffffu);
    const uint32_t s = mx_scale(top);
    const float inv = mx_inverse(s);
    uint32_t v[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = s == kMxNan ? 0.f : to_f32(t[w * 8 + i].v[c]) * inv;
      v[w] = mx_pack8(f);
    }
    vals[2 * lane + c][warp ^ (lane & 7)] = make_uint4(v[0], v[1], v[2], v[3]);
    scale[2 * lane + c][warp] = (uint8_t)s;
  }
  __syncthreads();
#pragma unroll
  for (int i = threadIdx.x; i < 64 * 8; i += kThreads) {
    const int col = i >> 3, blk = i & 7;
    if (o0 + col >= q.mat_rows || b0 + blk >= kb) continue;
    const int64_t row = mat * q.mat_rows + o0 + col;
    *reinterpret_cast<uint4*>(q.values + (row * kb + b0 + blk) * 16) = vals[col][blk ^ (col >> 1 & 7)];
    q.scales[row * q.scale_pitch + b0 + blk] = scale[col][blk];
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_mx_dequantize(MxRows q) {
  grid_launch_next();
  grid_wait();
  const Spot at = spot(q);
  const int64_t col = at.piece * 8, kb = (q.cols + kMxBlock - 1) / kMxBlock;
  if (col >= q.cols) return;
  uint32_t v[kRows], s[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t row = at.row + k * at.by;
    if (row >= q.rows) break;
    v[k] = *reinterpret_cast<const uint32_t*>(q.values + (row * kb * 4 + at.piece) * 4);
    s[k] = q.scales[row * q.scale_pitch + at.piece / 4];
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t row = at.row + k * at.by;
    if (row >= q.rows) break;
    float f[8];
    mx_unpack8(v[k], mx_value(s[k]), f);
    T* out = static_cast<T*>(q.dst) + row * q.cols + col;
    if (q.vec) {  // (then cols is a multiple of 8)
      alignas(16) T h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = from_f32<T>(f[i]);
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i)
        reinterpret_cast<uint4*>(out)[i] = reinterpret_cast<const uint4*>(h)[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < q.cols) out[i] = from_f32<T>(f[i]);
    }
  }
}

template <typename T>
cudaError_t run(MxRows q, MxOp op, cudaStream_t s) {
  constexpr int64_t b = sizeof(T);
  if (op == MX_ACROSS) {
    const int64_t ti = ((q.cols + kMxBlock - 1) / kMxBlock + 7) / 8, to = (q.mat_rows + 63) / 64;
    q.vec = reinterpret_cast<uintptr_t>(q.src) % (2 * b) == 0 && q.stride % 2 == 0 && q.batch_stride % 2 == 0;
    return launch_early(k_mx_quantize_across<T>, dim3((unsigned)(ti * to * (q.rows / q.mat_rows))), dim3(kThreads), 0, s,
                        q, (int)ti, (int)to);
  }
  const int64_t pieces = 4 * ((q.cols + kMxBlock - 1) / kMxBlock);
  q.log_across = 2;
  while (q.log_across < 8 && (1 << q.log_across) < pieces) ++q.log_across;
  q.col_blocks = (pieces + (1 << q.log_across) - 1) >> q.log_across;
  const int64_t down = (int64_t)(kThreads >> q.log_across) * kRows;
  const dim3 grid((unsigned)((q.rows + down - 1) / down * q.col_blocks));
  if (op == MX_BACK) {
    q.vec = reinterpret_cast<uintptr_t>(q.dst) % 16 == 0 && q.cols % 8 == 0;
    return launch_early(k_mx_dequantize<T>, grid, dim3(kThreads), 0, s, q);
  }
  q.vec = reinterpret_cast<uintptr_t>(q.src) % 16 == 0 && q.stride * b % 16 == 0 && q.batch_stride * b % 16 == 0;
  return launch_early(k_mx_quantize_rows<T>, grid, dim3(kThreads), 0, s, q);
}

}  // namespace

// Blocks of the largest grid of these kernels.
int64_t mx_blocks(int64_t rows, int64_t mat_rows, int64_t cols) {
  const int64_t kb = (cols + kMxBlock - 1) / kMxBlock;
  const int64_t along = (rows / kRows + 1) * ((kb * 4 + 255) / 256);
  const int64_t across = (kb + 7) / 8 * ((mat_rows + 63) / 64) * (mat_rows ? rows / mat_rows : 0);
  return along > across ? along : across;
}

cudaError_t launch_mx_rows(int32_t dtype, MxOp op, const MxRows& q, cudaStream_t s) {
  switch (dtype) {
    case DT_F16: return run<__half>(q, op, s);
    case DT_BF16: return run<__nv_bfloat16>(q, op, s);
    default: return run<float>(q, op, s);
  }
}

}  // namespace muon
