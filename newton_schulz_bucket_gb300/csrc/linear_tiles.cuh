// The tiles of a product on the tensor cores in CTA pairs, and what both kernels
// that compute them share: the arguments, the walk over the tiles, the stores of
// token rows, and the token operand's maps.
#pragma once

#include <cuda.h>

#include "linear.cuh"

namespace muon {

constexpr int BM = 256;  // features (rows form) or output rows (sum form) of a pair's tile
constexpr int kEpiWarps = 8;

__device__ __forceinline__ void mbar_arrive_release_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

struct TcProduct {
  int mode, experts, splits;
  const int32_t* offsets;
  int rows, K;              // rows form: token rows; the sum's length (GROUP_SUM: all rows)
  int M, N;                 // rows form: features (M); sum form: the output
  int tiles_m, tiles_n;     // sum form; rows form: feature tiles (tiles_m)
  int tile_rows;            // rows form: most token rows of a tile (64, 128 or 256; 4-bit operands 64, 128 or 192)
  int stages;               // rows form: ring depth, more for smaller tiles
  int type, act, vec;       // DType; vec: output rows (and the epilogue's tensors) start on 16 bytes
  void* D;                  // rows form: [rows][M]; sum form: [M][N] per expert
  const void* bias;
  const void* residual;
  int64_t r_m;
  void* preact;
  int first;                // first of the partial products (0 for fp32, 5 for the 16-bit types: one product)
  float* part;              // splits > 1: [splits][output rows][part_pitch] sums
  int64_t part_pitch;
  int* err;
};

__device__ __forceinline__ int range_at(const TcProduct& p, int e, int hi) {
  const int v = p.offsets[e];  // (an earlier launch may have written them while this one was resident)
  return v < 0 ? 0 : (v > hi ? hi : v);
}

// One tile's work.  Rows form: features m0 .., token rows n0 .. n_end - 1 (256
// at most).  Sum form: output rows m0 .., columns n0 ...  Sum over k0 .. k1 - 1.
struct Item {
  int e, m0, n0, n_end, k0, k1, split;
  int tile;                   // rows form: the token tile within its range
};

// Token tiles of a range of n rows: as few as tile_rows allows, in steps of 32
// rows shared out evenly (the first ones take one more).  Tile i of tiles starts
// at token_start(i); none is empty, as tiles - 1 full ones do not hold n.
__host__ __device__ __forceinline__ int token_start(int n, int tiles, int i) {
  const int units = (n + 31) / 32, each = units / tiles;
  return 32 * (i * each + min(i, units - each * tiles));
}
// Columns of a tile's MMA.
__device__ __forceinline__ int mma_cols(const Item& it) { return (it.n_end - it.n0 + 31) / 32 * 32; }

// 8 tile rows share a sweep over the tile columns, so that the tiles in
// flight reuse a compact set of panels through L2.
__device__ __forceinline__ void raster(int r, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int GM = 8;
  const int group = r / (GM * tiles_n), first = group * GM;
  const int gsz = min(tiles_m - first, GM);
  r -= group * GM * tiles_n;
  tm = first + r % gsz;
  tn = r / gsz;
}

// Walks this pair's tiles: every role of both CTAs sees the same sequence.
template <int BN>
struct Walk {
  int r, step;                // item within the current range / part, stride
  int e, lo, hi, after;       // the current range, its rows, the end of the one behind it
  int cnt, tt;                // the range's items and token tiles
  __device__ __forceinline__ Walk(const TcProduct& p)
      : r(blockIdx.x >> 1), step(gridDim.x >> 1), e(-1), lo(0), hi(0), after(0), cnt(0), tt(0) {
    const int most = BN == 0 ? p.rows : p.K;
    if (p.mode == GROUP_NONE) {
      after = most;
    } else {
      hi = range_at(p, 0, most);
      after = range_at(p, 1, most);
    }
  }
  // The next range; the end of its successor is on its way by the time it is
  // needed.
  __device__ __forceinline__ void advance(const TcProduct& p) {
    ++e;
    lo = hi;
    hi = max(lo, after);
    if (p.mode != GROUP_NONE && e + 2 <= p.experts) after = range_at(p, e + 2, BN == 0 ? p.rows : p.K);
  }
  __device__ __forceinline__ void part_of_sum(const TcProduct& p, int split, Item& it) {
    it.split = split;
    it.k0 = 0;
    it.k1 = p.K;
    if (p.splits > 1) {  // splits * blocks of the sum stays below 2^31
      const int kb = (p.K + BK - 1) / BK;
      it.k0 = kb * split / p.splits * BK;
      if (split + 1 < p.splits) it.k1 = kb * (split + 1) / p.splits * BK;
    }
  }
  __device__ __forceinline__ bool next(const TcProduct& p, Item& it) {
    int tm, tn;
    if constexpr (BN == 0) {
      while (r >= cnt) {
        r -= cnt;
        if (e + 1 >= (p.mode == GROUP_ROWS ? p.experts : 1)) { cnt = 0; return false; }
        advance(p);
        tt = (hi - lo + p.tile_rows - 1) / p.tile_rows;
        cnt = tt * p.tiles_m * p.splits;
      }
      int q = r, split = 0;
      if (p.splits > 1) {
        const int per = tt * p.tiles_m;
        split = q / per;
        q -= split * per;
      }
      raster(q, p.tiles_m, tt, tm, tn);
      it.e = e;
      it.m0 = tm * BM;
      it.tile = tn;
      it.n0 = lo + token_start(hi - lo, tt, tn);
      it.n_end = min(hi, lo + token_start(hi - lo, tt, tn + 1));
      part_of_sum(p, split, it);
    } else {
      const int per = p.tiles_m * p.tiles_n;
      while (r >= cnt) {  // range or part e + 1
        r -= cnt;
        if (e + 1 >= (p.mode == GROUP_SUM ? p.experts : p.splits)) { cnt = 0; return false; }
        if (p.mode == GROUP_SUM) advance(p);
        else ++e;
        cnt = per;
      }
      raster(r, p.tiles_m, p.tiles_n, tm, tn);
      it.m0 = tm * BM;
      it.n0 = tn * BN;
      it.n_end = p.N;
      if (p.mode == GROUP_SUM) {
        it.e = e;
        it.split = 0;
        it.k0 = lo;
        it.k1 = hi;
      } else {
        it.e = 0;
        part_of_sum(p, e, it);
      }
    }
    r += step;
    return true;
  }
};

// Rows form, one warp: feature f (this lane's) of tokens t0 .. t0 + n - 1 (n
// <= 32) from 32 accumulator columns.  Each store covers 32 features of one
// token's row.
template <typename T>
__device__ __forceinline__ void write_tokens(const TcProduct& p, float* v, int e, int64_t f, int64_t t0, int n) {
  const int64_t at = t0 * p.M + f;
  if (p.bias) {
    const float b = to_f32(static_cast<const T*>(p.bias)[e * (int64_t)p.M + f]);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] += b;
  }
  if (p.preact) {
    T* z = static_cast<T*>(p.preact) + at;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < n) z[(int64_t)i * p.M] = from_f32<T>(v[i]);
  }
  activate_n<32, sizeof(T) == 2>(v, p.act);
  if (p.residual) {
    const T* r = static_cast<const T*>(p.residual) + t0 * p.r_m + f;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < n) v[i] += to_f32(r[i * p.r_m]);
  }
  T* y = static_cast<T*>(p.D) + at;
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i < n) y[(int64_t)i * p.M] = from_f32<T>(v[i]);
}

// 16-bit units from .. to - 1 to zero, by all epilogue threads of the grid.
__device__ inline void zero_span(void* base, int64_t from, int64_t to, int64_t tid, int64_t n_threads) {
  uint16_t* p = static_cast<uint16_t*>(base);
  while (from < to && (reinterpret_cast<uintptr_t>(p + from) & 15)) {
    if (tid == 0) p[from] = 0;
    ++from;
  }
  const int64_t v = (to - from) / 8;
  for (int64_t i = tid; i < v; i += n_threads) reinterpret_cast<uint4*>(p + from)[i] = make_uint4(0, 0, 0, 0);
  for (int64_t i = from + v * 8 + tid; i < to; i += n_threads) p[i] = 0;
}

// Maps of the N operand.  Rows form: the same rows in boxes of 16, 32, 64, 96 and
// 128, so that a block's tokens come in one copy and drag few others along.
constexpr int kBoxes = 5;
struct NMaps {
  CUtensorMap box[kBoxes];
};
__host__ __device__ constexpr int box_rows(int b) { return b < 2 ? 16 << b : 32 * b; }

}  // namespace muon
