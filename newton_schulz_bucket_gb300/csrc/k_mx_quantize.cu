// Rows into microscaled 4-bit numbers and back (mx.cuh): weights once, activations
// in every product, along the sum.
//
// Numbers stored along the sum: four lanes share a block of 32, eight numbers each,
// so that loads and stores are whole lines.  Weights stored across the sum go through
// a tile of 256 steps of it by 64 columns: a lane takes 32 steps of two neighbouring
// columns, so that it has a block to itself, and the packed rows meet in shared
// memory.  Bound by HBM.
#include <type_traits>

#include "common.cuh"
#include "linear_tiles.cuh"
#include "mx.cuh"
#include "ops.h"

namespace muon {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;         // rows of a thread, in flight together

// Eight neighbouring numbers of a row.
template <typename T>
struct Eight {
  static constexpr int kWords = 2 * (int)sizeof(T);
  uint32_t w[kWords];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void fetch(const T* p) {  // 16-byte loads; read once
#pragma unroll
    for (int c = 0; c < kWords / 4; ++c)
      *reinterpret_cast<uint4*>(w + 4 * c) = __ldcs(reinterpret_cast<const uint4*>(p) + c);
  }
  __device__ __forceinline__ void fetch_some(const T* p, int64_t n) {  // the first n, zeros behind
    T* h = reinterpret_cast<T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = i < n ? p[i] : from_f32<T>(0.f);
  }
  // The largest magnitude, as bits of fp32 (magnitudes compare as integers, a NaN above
  // all).
  __device__ __forceinline__ uint32_t top() const {
    if constexpr (sizeof(T) == 4) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
      return m;
    } else {
      uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
      for (int i = 1; i < 4; ++i) asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7fff7fffu));
      m = max(m & 0xffffu, m >> 16);
      if constexpr (std::is_same<T, __nv_bfloat16>::value) return m << 16;
      else return __float_as_uint(__half2float(__ushort_as_half((uint16_t)m)));
    }
  }
  __device__ __forceinline__ uint32_t packed(float inverse) const {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 4) f[i] = __uint_as_float(w[i]);
      else if constexpr (std::is_same<T, __nv_bfloat16>::value) f[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
      else f[i] = __half2float(__ushort_as_half((uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu)));
      f[i] *= inverse;
    }
    return mx_pack8(f);
  }
};

// Where a thread of the row kernels works: its piece of eight columns, its first row.
struct Spot {
  int64_t piece, row;
  int by;                        // rows between a thread's rows
};
__device__ __forceinline__ Spot spot(const MxRows& q, int64_t block) {
  const int across = 1 << q.log_across, down = kThreads >> q.log_across;
  const int64_t cb = block % q.col_blocks, rb = block / q.col_blocks;
  return {cb * across + (threadIdx.x & (across - 1)), rb * down * kRows + (threadIdx.x >> q.log_across), down};
}

// Loads and rounds a thread's rows; each row's block of 32 and its scale go to `give`,
// which all lanes of a warp call together.
// (rows counts those of all matrices; one row after the other in the outputs)
template <typename T, typename M, typename F>
__device__ __forceinline__ void quantize_rows(const MxRows& q, int64_t block, M meanwhile, F give) {
  const Spot at = spot(q, block);
  const int64_t col = at.piece * 8, kb = (q.cols + kMxBlock - 1) / kMxBlock;
  const bool there = at.piece < 4 * kb;
  const T* src = static_cast<const T*>(q.src) + at.row * q.stride + col;  // (of one matrix)
  Eight<T> v[kRows];
  const bool whole = q.vec && col + 8 <= q.cols;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t row = at.row + k * at.by;
    v[k].zero();
    if (!there || row >= q.rows) continue;
    const T* p = src + k * at.by * q.stride;
    if (q.mat_rows != q.rows) {
      const int64_t mat = row / q.mat_rows;
      p = static_cast<const T*>(q.src) + mat * q.batch_stride + (row - mat * q.mat_rows) * q.stride + col;
    }
    if (whole) v[k].fetch(p);
    else v[k].fetch_some(p, q.cols - col);
  }
  meanwhile();
  uint32_t* out = reinterpret_cast<uint32_t*>(q.values) + at.row * kb * 4 + at.piece;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {  // four lanes share a block
    uint32_t top = v[k].top();
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t s = mx_scale(top);
    const int64_t row = at.row + k * at.by;
    if (there && row < q.rows) out[k * at.by * kb * 4] = v[k].packed(mx_inverse(s));
    give(row, at.piece / 4, s, row < q.rows);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_mx_quantize_rows(MxRows q) {
  grid_launch_next();
  grid_wait();
  const int64_t kb = (q.cols + kMxBlock - 1) / kMxBlock;
  quantize_rows<T>(q, blockIdx.x, [] {}, [&](int64_t row, int64_t b, uint32_t s, bool there) {
    if (there && b < kb && (threadIdx.x & 3) == 0) q.scales[row * kb + b] = (uint8_t)s;
  });
}

__device__ __forceinline__ int clamped(const MxPrepare& q, int e) {
  const int v = q.offsets[e], rows = (int)q.x.rows;
  return v < 0 ? 0 : (v > rows ? rows : v);
}

// Byte of a token row's first scale: the slot of its tile (as Walk cuts ranges into
// tiles), its row there; -1 for a row of no range.  ends: the ranges' offsets.
__device__ __forceinline__ int64_t token_scales(const MxPrepare& q, const int* ends, int row, int64_t slot_bytes) {
  int e = 0, lo = 0, hi = (int)q.x.rows;
  if (q.experts) {  // the range that holds the row: the first that ends behind it
    int end = q.experts;
    while (e < end) {
      const int m = (e + end) / 2;
      if (ends[m + 1] > row) end = m;
      else e = m + 1;
    }
    if (e == q.experts) return -1;
    lo = ends[e];
    hi = ends[e + 1];
    if (row < lo) return -1;
  }
  const int n = hi - lo, tiles = (n + q.tile_rows - 1) / q.tile_rows;
  const int units = (n + 31) / 32, each = units / tiles, more = units - each * tiles, u = (row - lo) / 32;
  const int tile = u < more * (each + 1) ? u / (each + 1) : more + (u - more * (each + 1)) / each;
  const int r = row - lo - token_start(n, tiles, tile);
  return (int64_t)(mx_token_slot(lo, e, q.tile_rows) + tile) * slot_bytes + (r >> 7) * 512 + mx_scale_byte(r, 0);
}

// What a product starts from, in one launch: the token rows, then the weights' scales
// (of the matrices that any row reaches) through shared memory, 128 rows x 64 words.
constexpr int kWords = 16;
constexpr int kMostRows = kThreads / 4 * kRows;  // of a block
template <typename T>
__global__ void __launch_bounds__(kThreads) k_mx_prepare(MxPrepare q) {
  __shared__ uint32_t words[128][kWords + 1];
  __shared__ int ends[1025];
  __shared__ int64_t place[kMostRows];
  grid_wait();
  // only now: the product reads the weights before it waits for this launch
  grid_launch_next();
  const int64_t kb = (q.x.cols + kMxBlock - 1) / kMxBlock, parts = (kb + 3) / 4;
  if (blockIdx.x < q.x_blocks) {
    const int64_t part_bytes = 512 * mx_token_blocks(q.tile_rows), slot_bytes = parts * part_bytes;
    const int across = 1 << q.x.log_across, rows = (kThreads >> q.x.log_across) * kRows;
    const int64_t row0 = blockIdx.x / q.x.col_blocks * rows;
    const auto find = [&] {  // (while the rows are on their way)
      if (q.experts) {
        for (int i = threadIdx.x; i <= q.experts; i += kThreads) ends[i] = clamped(q, i);
        __syncthreads();
      }
      for (int i = threadIdx.x; i < rows; i += kThreads)
        place[i] = row0 + i < q.x.rows ? token_scales(q, ends, (int)(row0 + i), slot_bytes) : -1;
      __syncthreads();
    };
    quantize_rows<T>(q.x, blockIdx.x, find, [&](int64_t row, int64_t b, uint32_t s, bool there) {
      // the scales of 128 steps in one store where a warp's lanes hold them (zeros behind
      // the row's end)
      const int64_t at = there && b < kb ? place[row - row0] : -1;
      if (across >= 16) {
        uint32_t v = s << (8 * (b & 3));
        v |= __shfl_xor_sync(0xffffffffu, v, 4);
        v |= __shfl_xor_sync(0xffffffffu, v, 8);
        if (at >= 0 && (threadIdx.x & 15) == 0) *reinterpret_cast<uint32_t*>(q.x.scales + at + (b >> 2) * part_bytes) = v;
      } else if (at >= 0 && (threadIdx.x & 3) == 0) {  // one part
        q.x.scales[at + b] = (uint8_t)s;
        if (b + 1 == kb)
          for (int64_t z = b + 1; z < 4; ++z) q.x.scales[at + z] = 0;
      }
    });
    return;
  }
  int64_t j = blockIdx.x - q.x_blocks;
  const int64_t run = j % q.w_parts, tiles = (q.out + 127) / 128;
  j /= q.w_parts;
  const int64_t mat = j / tiles, row0 = j % tiles * 128;
  if (q.experts && clamped(q, (int)mat) >= clamped(q, (int)mat + 1)) return;
  const uint8_t* src = q.w_scales + (mat * q.out + row0) * kb;
  const int rows = (int)min((int64_t)128, q.out - row0);
  const int64_t w0 = run * kWords;
  const int n = (int)min((int64_t)kWords, parts - w0);
  const bool vec = kb % 4 == 0 && (reinterpret_cast<uintptr_t>(q.w_scales) & 3) == 0;
#pragma unroll 8
  for (int i = threadIdx.x; i < 128 * kWords; i += kThreads) {
    const int r = i / kWords, w = i % kWords;
    uint32_t v = 0;
    if (r < rows && w < n) {
      const uint8_t* p = src + r * kb + (w0 + w) * 4;
      if (vec) {
        v = *reinterpret_cast<const uint32_t*>(p);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if ((w0 + w) * 4 + k < kb) v |= (uint32_t)p[k] << (8 * k);
      }
    }
    words[r][w] = v;
  }
  __syncthreads();
  uint4* out = reinterpret_cast<uint4*>(q.w_ordered + ((mat * tiles + row0 / 128) * parts + w0) * 512);
  for (int i = threadIdx.x; i < n * 32; i += kThreads) {
    const int w = i >> 5, lane = i & 31;
    out[i] = make_uint4(words[lane][w], words[32 + lane][w], words[64 + lane][w], words[96 + lane][w]);
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
      for (int i = 0; i < 8; ++i) f[i] = to_f32(t[w * 8 + i].v[c]) * inv;
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
    q.scales[row * kb + b0 + blk] = scale[col][blk];
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_mx_dequantize(MxRows q) {
  grid_launch_next();
  grid_wait();
  const Spot at = spot(q, blockIdx.x);
  const int64_t col = at.piece * 8, kb = (q.cols + kMxBlock - 1) / kMxBlock;
  if (col >= q.cols) return;
  uint32_t v[kRows], s[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t row = at.row + k * at.by;
    if (row >= q.rows) break;
    v[k] = *reinterpret_cast<const uint32_t*>(q.values + (row * kb * 4 + at.piece) * 4);
    s[k] = q.scales[row * kb + at.piece / 4];
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

// How blocks cover rows of pieces of eight columns; their number.
int64_t shape_rows(MxRows* q) {
  const int64_t pieces = 4 * mx_blocks_of(q->cols);
  q->log_across = 2;
  while (q->log_across < 8 && (1 << q->log_across) < pieces) ++q->log_across;
  q->col_blocks = (pieces + (1 << q->log_across) - 1) >> q->log_across;
  const int64_t down = (int64_t)(kThreads >> q->log_across) * kRows;
  return (q->rows + down - 1) / down * q->col_blocks;
}
// 16-byte loads: every row starts on 16 bytes.
template <typename T>
bool vector_rows(const MxRows& q) {
  constexpr int64_t b = sizeof(T);
  return reinterpret_cast<uintptr_t>(q.src) % 16 == 0 && (q.mat_rows == 1 || q.stride * b % 16 == 0) &&
         q.batch_stride * b % 16 == 0;
}

template <typename T>
cudaError_t run(MxRows q, MxOp op, cudaStream_t s) {
  if (op == MX_ACROSS) {
    const int64_t ti = ((q.cols + kMxBlock - 1) / kMxBlock + 7) / 8, to = (q.mat_rows + 63) / 64;
    q.vec = reinterpret_cast<uintptr_t>(q.src) % (2 * sizeof(T)) == 0 && q.stride % 2 == 0 && q.batch_stride % 2 == 0;
    return launch_early(k_mx_quantize_across<T>, dim3((unsigned)(ti * to * (q.rows / q.mat_rows))), dim3(kThreads), 0, s,
                        q, (int)ti, (int)to);
  }
  const dim3 grid((unsigned)shape_rows(&q));
  if (op == MX_BACK) {
    q.vec = reinterpret_cast<uintptr_t>(q.dst) % 16 == 0 && q.cols % 8 == 0;
    return launch_early(k_mx_dequantize<T>, grid, dim3(kThreads), 0, s, q);
  }
  q.vec = vector_rows<T>(q);
  return launch_early(k_mx_quantize_rows<T>, grid, dim3(kThreads), 0, s, q);
}

template <typename T>
cudaError_t run_prepare(MxPrepare q, cudaStream_t s) {
  q.x_blocks = shape_rows(&q.x);
  q.x.vec = vector_rows<T>(q.x);
  q.w_parts = (mx_parts(q.x.cols) + kWords - 1) / kWords;
  const int64_t grid = q.x_blocks + q.w_parts * ((q.out + 127) / 128) * q.mats;
  return launch_early(k_mx_prepare<T>, dim3((unsigned)grid), dim3(kThreads), 0, s, q);
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

int64_t mx_prepare_blocks(int64_t rows, int64_t in, int64_t out, int64_t mats) {
  return mx_blocks(rows, rows, in) + (mx_parts(in) + kWords - 1) / kWords * ((out + 127) / 128) * mats;
}

cudaError_t launch_mx_prepare(int32_t dtype, const MxPrepare& q, cudaStream_t s) {
  switch (dtype) {
    case DT_F16: return run_prepare<__half>(q, s);
    case DT_BF16: return run_prepare<__nv_bfloat16>(q, s);
    default: return run_prepare<float>(q, s);
  }
}

}  // namespace muon
