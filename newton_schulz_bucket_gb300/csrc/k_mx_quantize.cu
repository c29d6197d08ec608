// Rows into microscaled 4-bit numbers and back (mx.cuh): weights once, activations
// in every product, along the sum.
//
// Numbers stored along the sum: four lanes share a block of 32, eight numbers each,
// so that loads and stores are whole lines.  Weights stored across the sum go through
// a tile of 256 steps of it by 64 columns: a lane takes 32 steps of two neighbouring
// columns, so that it has a block to itself, and the packed rows meet in shared
// memory.  Bound by HBM: [4096, 16384] bf16 into 4 bits and back 57.6 us, 340 MB with the
// packed numbers (5.9 TB/s).  In front of a product, 32768 rows of 7168 and the scales of 64
// matrices [7168, 2048] take about 130 us, 646 MB (5 TB/s).
#include "common.cuh"
#include "linear_tiles.cuh"
#include "mx.cuh"
#include "ops.h"

namespace muon {

namespace {

constexpr int kThreads = 256;
// Rows of a thread, in flight together: in front of a product (4096 rows of 4096 before
// [4096, 16384]: 110 us with four, 112 with eight or two; 32 rows over 64 experts 50.6, 54,
// 51.2), and of weights held along the sum (into 4 bits and back, [16384, 4096] bf16 56 us with
// four, 59 with two; [4096, 4096] fp32 31.9 and 31.1, five [777, 1001] 16.8 and 14.2).
constexpr int kRowsOf = 4;
template <typename T>
constexpr int kWeightRows = sizeof(T) == 4 ? 2 : 4;

// Where a thread of the row kernels works: its piece of eight columns, its first row.
struct Spot {
  int64_t row;
  int piece, by;                 // rows between a thread's rows
};
template <int kRows>
__device__ __forceinline__ Spot spot(const MxRows& q, uint32_t block) {
  const int across = 1 << q.log_across, down = kThreads >> q.log_across;
  const uint32_t rb = block / q.col_blocks, cb = block - rb * q.col_blocks;  // (the first of its column blocks)
  return {(int64_t)rb * down * kRows + (threadIdx.x >> q.log_across),
          (int)cb * across + ((int)threadIdx.x & (across - 1)), down};
}

// Loads and rounds a thread's rows; each row's block of 32 and its scale go to `give`,
// which all lanes of a warp call together.  kMats: rows of several matrices (rows counts
// all of them; one row after the other in the outputs).
template <typename T, int kRows, bool kMats, typename M, typename F>
__device__ __forceinline__ void quantize_rows(const MxRows& q, const Spot& at, M meanwhile, F give) {
  const int64_t col = (int64_t)at.piece * 8, kb = (q.cols + kMxBlock - 1) / kMxBlock;
  const bool there = at.piece < 4 * kb;
  const T* src = static_cast<const T*>(q.src) + at.row * q.stride + col;
  const int64_t step = at.by * q.stride;
  const int left = (int)min((int64_t)kRows * at.by, q.rows - at.row);  // rows from the first on
  Eight<T> v[kRows];
  const bool whole = q.vec && col + 8 <= q.cols;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    v[k].zero();
    const T* p = src + k * step;
    if (kMats) {
      const int64_t row = at.row + k * at.by;
      const int64_t mat = row / q.mat_rows;
      p = static_cast<const T*>(q.src) + mat * q.batch_stride + (row - mat * q.mat_rows) * q.stride + col;
    }
    if (there && k * at.by < left) {
      if (whole) v[k].fetch(p);
      else v[k].fetch_some(p, q.cols - col);
    }
  }
  meanwhile();
  uint32_t* out = reinterpret_cast<uint32_t*>(q.values) + at.row * kb * 4 + at.piece;
  const int64_t out_step = at.by * kb * 4;
  uint32_t top[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) top[k] = v[k].top();
  // four lanes share a block; two rows of 16 bits go through the shuffles together
#pragma unroll
  for (int k = 0; k < kRows; k += 2) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = k; j < k + 2; ++j) {
        top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 1));
        top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 2));
      }
    } else {
      uint32_t t = __byte_perm(top[k], top[k + 1], 0x5410);
      asm("max.u16x2 %0, %0, %1;" : "+r"(t) : "r"(__shfl_xor_sync(0xffffffffu, t, 1)));
      asm("max.u16x2 %0, %0, %1;" : "+r"(t) : "r"(__shfl_xor_sync(0xffffffffu, t, 2)));
      top[k] = t & 0xffffu;
      top[k + 1] = t >> 16;
    }
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const uint32_t s = Eight<T>::scale(top[k]);
    const bool live = k * at.by < left;
    if (there && live) out[k * out_step] = v[k].packed(mx_inverse(s));
    give(k, at.piece / 4, s, live);
  }
}

template <typename T, bool kMats>
__global__ void __launch_bounds__(kThreads) k_mx_quantize_rows(MxRows q) {
  grid_launch_next();
  grid_wait();
  const int64_t kb = (q.cols + kMxBlock - 1) / kMxBlock;
  const Spot at = spot<kWeightRows<T>>(q, blockIdx.x);
  quantize_rows<T, kWeightRows<T>, kMats>(q, at, [] {}, [&](int k, int b, uint32_t s, bool live) {
    if (live && b < kb && (threadIdx.x & 3) == 0) q.scales[(at.row + k * at.by) * kb + b] = (uint8_t)s;
  });
}

__device__ __forceinline__ int clamped(const MxPrepare& q, int e) {
  const int v = q.offsets[e], rows = (int)q.x.rows;
  return v < 0 ? 0 : (v > rows ? rows : v);
}

// Where a token row's scales start, in words of 128 steps' (four): the slot of its tile
// (as Walk cuts ranges into tiles), its row there; kNowhere for a row of no range.
constexpr uint32_t kNowhere = 0xffffffffu;
__device__ __forceinline__ uint32_t token_scales(const MxPrepare& q, int row, uint32_t slot_words) {
  int e = 0, lo = 0, hi = (int)q.x.rows;
  if (q.experts) {  // the range that holds the row: the first that ends behind it
    int end = q.experts;
    while (e < end) {
      const int m = (e + end) / 2;
      if (clamped(q, m + 1) > row) end = m;
      else e = m + 1;
    }
    if (e == q.experts) return kNowhere;
    lo = clamped(q, e);
    hi = clamped(q, e + 1);
    if (row < lo) return kNowhere;
  }
  const int n = hi - lo, tiles = (n + q.tile_rows - 1) / q.tile_rows;
  const int units = (n + 31) / 32, each = units / tiles, more = units - each * tiles, u = (row - lo) / 32;
  const int tile = u < more * (each + 1) ? u / (each + 1) : more + (u - more * (each + 1)) / each;
  const int r = row - lo - token_start(n, tiles, tile);
  return (mx_token_slot(lo, e, q.tile_rows) + tile) * slot_words + (r >> 7) * 128 + mx_scale_byte(r, 0) / 4;
}

// What a product starts from, in one launch: the token rows, then the weights' scales
// (of the matrices that any row reaches) through shared memory, 128 rows x 16 words.
constexpr int kWords = 16;
template <typename T>
__global__ void __launch_bounds__(kThreads) k_mx_prepare(MxPrepare q) {
  __shared__ uint32_t words[128][kWords + 1];
  __shared__ uint32_t place[kThreads / 4 * kRowsOf];
  grid_wait();
  // only now: the product reads the weights before it waits for this launch
  grid_launch_next();
  const int64_t kb = (q.x.cols + kMxBlock - 1) / kMxBlock, parts = (kb + 3) / 4;
  if (blockIdx.x < (uint32_t)q.x_blocks) {
    constexpr int kRows = kRowsOf;
    const uint32_t part_words = 128 * mx_token_blocks(q.tile_rows), slot_words = (uint32_t)parts * part_words;
    const Spot at = spot<kRows>(q.x, blockIdx.x);
    // the block's rows' places, while the rows are on their way (each warp for itself took
    // half of the instructions of the whole kernel)
    const int rows = (kThreads >> q.x.log_across) * kRows, across = 1 << q.x.log_across;
    const int64_t row0 = at.row - (threadIdx.x >> q.x.log_across);
    const auto find = [&] {
      for (int i = threadIdx.x; i < rows; i += kThreads)
        place[i] = row0 + i < q.x.rows ? token_scales(q, (int)(row0 + i), slot_words) : kNowhere;
      __syncthreads();
    };
    // four lanes store the scales of 128 steps side by side, zeros behind the row's end
    const int last = across >= 16 ? (int)parts * 4 : (int)kb;
    const uint32_t* mine = place + (at.row - row0);
    const auto give = [&](int k, int b, uint32_t s, bool) {
      const uint32_t to = mine[k * at.by];
      if (to == kNowhere || (threadIdx.x & 3) != 0 || b >= last) return;
      uint8_t* word = q.x.scales + (int64_t)(to + (uint32_t)(b >> 2) * part_words) * 4;
      word[b & 3] = (uint8_t)s;
      if (across < 16 && b + 1 == (int)kb)  // no lanes there
        for (int z = b + 1; z < 4; ++z) word[z] = 0;
    };
    quantize_rows<T, kRows, false>(q.x, at, find, give);
    // (enough rows to fill the GPU: one block takes all columns of its own)
    for (Spot next = at; next.piece + across * (int)q.x.col_blocks < across * q.x.col_total;) {
      next.piece += across * (int)q.x.col_blocks;
      quantize_rows<T, kRows, false>(q.x, next, [] {}, give);
    }
    return;
  }
  const uint32_t j = blockIdx.x - (uint32_t)q.x_blocks, runs = (uint32_t)q.w_parts;
  const uint32_t tiles = (uint32_t)((q.out + 127) / 128), tile = j / runs;
  const int64_t mat = tile / tiles, row0 = (int64_t)(tile - mat * tiles) * 128;
  if (q.experts && clamped(q, (int)mat) >= clamped(q, (int)mat + 1)) return;
  const uint8_t* src = q.w_scales + (mat * q.out + row0) * kb;
  const int rows = (int)min((int64_t)128, q.out - row0);
  const bool vec = kb % 4 == 0 && (reinterpret_cast<uintptr_t>(q.w_scales) & 3) == 0;
  for (int64_t w0 = (int64_t)(j - tile * runs) * kWords; w0 < parts; w0 += runs * kWords) {
    const int n = (int)min((int64_t)kWords, parts - w0);
    __syncthreads();  // the words of the round before are stored
#pragma unroll
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
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_mx_quantize_across(MxRows q, int in_tiles, int out_tiles) {
  __shared__ uint4 vals[64][8];  // [column][block ^ (column / 2 & 7)]
  __shared__ uint8_t scale[64][8];
  struct Two {
    T v[2];
  };
  using Word = typename std::conditional<sizeof(T) == 4, uint2, uint32_t>::type;
  grid_launch_next();
  grid_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t b = blockIdx.x / (uint32_t)out_tiles;
  const int64_t o0 = (int64_t)(blockIdx.x - b * out_tiles) * 64, kb = (q.cols + kMxBlock - 1) / kMxBlock;
  const int64_t mat = b / (uint32_t)in_tiles, b0 = (int64_t)(b - (uint32_t)mat * in_tiles) * 8;
  const int64_t i0 = (b0 + warp) * kMxBlock, o = o0 + 2 * lane;
  const int n = (int)max((int64_t)0, min((int64_t)2, q.mat_rows - o));  // the lane's columns
  const int steps = (int)max((int64_t)0, min((int64_t)kMxBlock, q.cols - i0));
  const T* src = static_cast<const T*>(q.src) + mat * q.batch_stride + i0 * q.stride + o;
  Two t[kMxBlock];
  if (q.vec && n == 2 && steps == kMxBlock) {
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i) {
      const Word u = __ldcs(reinterpret_cast<const Word*>(src + i * q.stride));
      t[i] = *reinterpret_cast<const Two*>(&u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i) {
      t[i].v[0] = i < steps && n > 0 ? src[i * q.stride] : from_f32<T>(0.f);
      t[i].v[1] = i < steps && n > 1 ? src[i * q.stride + 1] : from_f32<T>(0.f);
    }
  }
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

constexpr int kBackRows = 4;
template <typename T>
__global__ void __launch_bounds__(kThreads) k_mx_dequantize(MxRows q) {
  grid_launch_next();
  grid_wait();
  constexpr int kRows = kBackRows;
  const Spot at = spot<kRows>(q, blockIdx.x);
  const int64_t col = (int64_t)at.piece * 8, kb = (q.cols + kMxBlock - 1) / kMxBlock;
  // lanes of a warp that share a row
  const int w = min(1 << q.log_across, 32), own = threadIdx.x & (w - 1);
  uint32_t v[kRows] = {}, s[kRows] = {};
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t row = at.row + k * at.by;
    if (row >= q.rows || col >= q.cols) break;
    v[k] = *reinterpret_cast<const uint32_t*>(q.values + (row * kb * 4 + at.piece) * 4);
    s[k] = q.scales[row * kb + at.piece / 4];
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t row = at.row + k * at.by;
    if (q.vec && (row >= q.rows || col >= q.cols)) break;
    if (q.vec) {  // (then cols is a multiple of 8)
      float f[8];
      mx_unpack8(v[k], mx_value(s[k]), f);
      T* out = static_cast<T*>(q.dst) + row * q.cols + col;
      alignas(16) T h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = from_f32<T>(f[i]);
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i)
        reinterpret_cast<uint4*>(out)[i] = reinterpret_cast<const uint4*>(h)[i];
    } else {  // element by element, neighbouring ones in neighbouring lanes
      T* out = static_cast<T*>(q.dst) + row * q.cols + (col - own * 8);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = j * w + own;  // of the w pieces that these lanes hold
        const uint32_t from = __shfl_sync(0xffffffffu, v[k], i >> 3, w), by = __shfl_sync(0xffffffffu, s[k], i >> 3, w);
        float f[8];
        mx_unpack8(from >> (4 * (i & 7)), mx_value(by), f);
        if (row < q.rows && col - own * 8 + i < q.cols) out[i] = from_f32<T>(f[0]);
      }
    }
  }
}

// How blocks cover rows of pieces of eight columns; their number.
int64_t shape_rows(MxRows* q, int each) {
  const int64_t pieces = 4 * mx_blocks_of(q->cols);
  q->log_across = 2;
  while (q->log_across < 8 && (1 << q->log_across) < pieces) ++q->log_across;
  q->col_blocks = (uint32_t)((pieces + (1 << q->log_across) - 1) >> q->log_across);
  q->col_total = (int32_t)q->col_blocks;
  const int64_t down = (int64_t)(kThreads >> q->log_across) * each;
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
  const dim3 grid((unsigned)shape_rows(&q, op == MX_BACK ? kBackRows : kWeightRows<T>));
  if (op == MX_BACK) {
    q.vec = reinterpret_cast<uintptr_t>(q.dst) % 16 == 0 && q.cols % 8 == 0;
    return launch_early(k_mx_dequantize<T>, grid, dim3(kThreads), 0, s, q);
  }
  q.vec = vector_rows<T>(q);
  return q.mat_rows == q.rows ? launch_early(k_mx_quantize_rows<T, false>, grid, dim3(kThreads), 0, s, q)
                              : launch_early(k_mx_quantize_rows<T, true>, grid, dim3(kThreads), 0, s, q);
}

template <typename T>
cudaError_t run_prepare(MxPrepare q, cudaStream_t s) {
  q.x_blocks = shape_rows(&q.x, kRowsOf);
  q.x.vec = vector_rows<T>(q.x);
  // a block takes all columns of its rows, or all parts of its 128 features, where that
  // leaves blocks enough
  if (q.x_blocks / q.x.col_blocks >= 4 * num_sms()) {
    q.x_blocks /= q.x.col_blocks;
    q.x.col_blocks = 1;
  }
  const int64_t features = (q.out + 127) / 128 * q.mats;
  q.w_parts = features >= 2 * num_sms() ? 1 : (mx_parts(q.x.cols) + kWords - 1) / kWords;
  const int64_t grid = q.x_blocks + q.w_parts * features;
  return launch_early(k_mx_prepare<T>, dim3((unsigned)grid), dim3(kThreads), 0, s, q);
}

}  // namespace

// Blocks of the largest grid of these kernels.
int64_t mx_blocks(int64_t rows, int64_t mat_rows, int64_t cols) {
  const int64_t kb = (cols + kMxBlock - 1) / kMxBlock;
  const int64_t along = (rows / 2 + 1) * ((kb * 4 + 255) / 256);
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
