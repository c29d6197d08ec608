// A layer's product on the tensor cores: D(m, n) = act(sum_k A(m, k) B(k, n) +
// bias) + residual in fp16 / bf16 operands with fp32 sums.
//
// fp32 tensors.  Each operand is cut into three bf16 numbers, x = h + m + l, each
// the nearest to what is left (8 significant bits, so the three hold all 24), and
// the product is the sum of the six partial products down to h l, m m and l h.  A
// part is at most 2^-8 (m) and 2^-17 (l) of the operand's power of two, so that what is
// left out, m l + l m + l l, is below 2^-24 of the product and of either sign (cut off
// instead of rounded, the parts would leave out up to 2^-21, always towards zero).  Six
// bf16 products are 4 to 5 times as fast as one in fp32 FMA.
//
// An infinity or a NaN goes into the low part, with h = +-1 and m = 0 beside it: of
// the six products only h l and l h then see it, each time against the other
// operand's h, which is zero only where that operand is (in the high part it would
// meet the zero m and l of every short number, and make NaN of 1 times infinity).
//
// A cluster of two CTAs computes one 256 x N tile (N <= 256) with tcgen05.mma
// cta_group::2, as the Newton-Schulz products do: each CTA stages its 128 rows
// of the M operand and its half of the N operand's rows in a ring of TMA tiles,
// the leader issues the MMAs, and both hold 128 rows of the accumulator in
// TMEM (two accumulators, so that the epilogue of one tile runs under the
// products of the next).  Operands may be stored along the sum or across it, so
// none is ever transposed in memory.
//
// Rows form (y = x W, dx = dz W^T).  The weight matrix is the M operand and
// the token rows are the N operand, i.e. a tile is 256 features x N tokens.  N
// is chosen per tile from the rows there are, in steps of 32: few rows stream the
// weights through 32-column MMAs, and an expert with 257 rows costs two tiles of
// 160 and 128 columns, not two of 256.  An accumulator lane is a feature, so a
// warp's stores run along a token's row for any width and alignment.  Measured:
// [4096 x 4096] x [4096, 16384] with gelu_tanh and its pre-activation 344 us back to
// back (1600 TFLOP/s under the power cap, where cuBLAS alone sustains 1700); 64
// experts [7168, 2048] with 16 rows each 263 us (7.1 TB/s of weights: HBM), with
// 256 rows 315 us (1530 TFLOP/s), with 320 rows 410 us: two tiles an expert, bound
// by neither HBM nor the MMAs alone.
//
// Sum form (dw = x^T dz).  Both operands are stored across the sum (tokens);
// tiles are 256 x 256 or 256 x 128.  With few tokens to an expert the stores set
// the pace: 32 x 64 blocks of rounded outputs are staged swizzled and leave by TMA
// stores (where output rows start on 16 bytes), so that the load/store pipe
// carries each output once, not three times (654 -> 564 us at its first measure).
// 64 experts [2048, 7168] from 64 rows each: 356 us (5.3 TB/s of stores), from 256
// rows 400 us, from 512 rows 618 us, where loads alone would take 474.
//
// Experts.  Row ranges come from a device array, so every role walks the
// ranges itself.  GROUP_ROWS: an expert's rows are tiled from its first row;
// rows past its end are loaded (they are the next expert's), multiplied into
// accumulator columns of their own, and not stored.  GROUP_SUM: the sum over an
// expert's rows ends inside a 64-row block of the ring, whose other rows belong
// to the next expert, and may hold NaN there: a helper warp overwrites them in
// shared memory with zeros, in both operands, before the block is handed to
// the MMAs.
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "linear.cuh"

namespace muon {

namespace {

constexpr int BM = 256;  // features (rows form) or output rows (sum form) of a pair's tile
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (3 + kEpiWarps);  // producer, MMA issuer, epilogue, range-tail helper

__device__ int g_err;       // the operators' error word (one per device)

struct TcProduct {
  int mode, experts, splits;
  const int32_t* offsets;
  int rows, K;              // rows form: token rows; the sum's length (GROUP_SUM: all rows)
  int M, N;                 // rows form: features (M); sum form: the output
  int tiles_m, tiles_n;     // sum form; rows form: feature tiles (tiles_m)
  int tile_rows;            // rows form: most token rows of a tile (64, 128 or 256)
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

// Ring and staging of one CTA.  Rows form (BN = 0): the same bytes hold 7, 9 or
// 11 stages for tiles of up to 256, 128 or 64 tokens, so that a stream of
// weights past few tokens has more of them in flight.
constexpr int kMaxStages = 11;
template <int BN>
struct Smem {
  static constexpr int kStages = BN == 0 ? 7 : (BN == 256 ? 6 : 8);
  static constexpr uint32_t kA = 128 * BK * 2;
  static constexpr uint32_t kB = (BN == 0 ? 128 : BN / 2) * BK * 2;
  static constexpr uint32_t kStage = kA + kB;
  static constexpr uint32_t kEpi = kStages * kStage;  // sum form: 4 KB a warp, 1024-byte aligned for TMA's swizzle
  static constexpr uint32_t kBars = kEpi + (BN == 0 ? 0 : kEpiWarps * 4096);  // full, empty, fix, tfull, tempty,
                                                                               // done; TMEM slot, abort flag
  static constexpr uint32_t kTotal = kBars + 512 + 1024;  // + alignment slack
  static_assert((3 * kMaxStages + 5) * 8 + 8 <= 512 && kTotal <= 227 * 1024, "shared memory layout");
};
__host__ __device__ constexpr uint32_t rows_stage_bytes(int tile_rows) { return (128 + tile_rows / 2) * BK * 2; }
__host__ __device__ constexpr int rows_stages(int tile_rows) { return (int)(Smem<0>::kEpi / rows_stage_bytes(tile_rows)); }
static_assert(rows_stages(256) == 7 && rows_stages(128) == 9 && rows_stages(64) == kMaxStages, "ring depths");

__device__ __forceinline__ void mbar_arrive_release_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ int range_at(const TcProduct& p, int e, int hi) {
  const int v = p.offsets[e];  // (an earlier launch may have written them while this one was resident)
  return v < 0 ? 0 : (v > hi ? hi : v);
}

// One tile's work.  Rows form: features m0 .., token rows n0 .. n_end - 1 (256
// at most).  Sum form: output rows m0 .., columns n0 ...  Sum over k0 .. k1 - 1.
struct Item {
  int e, m0, n0, n_end, k0, k1, split;
};

// Token tiles of a range of n rows: as few as tile_rows allows, in steps of 32
// rows shared out evenly (the first ones take one more).  Tile i of tiles starts
// at token_start(i); none is empty, as tiles - 1 full ones do not hold n.
__device__ __forceinline__ int token_start(int n, int tiles, int i) {
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

// Sum form, a warp's 32 x 32 block from TMEM into its staging block, row =
// lane, the 16-byte pieces of row r at piece index ^ (r & 7): both this write
// and the reads along rows below are free of bank conflicts.
__device__ __forceinline__ void stage_block(uint32_t taddr, float* sw, int lane, bool zero) {
  uint32_t r[32];
  tmem_ld32(taddr, r);
  uint4* row = reinterpret_cast<uint4*>(sw + lane * 32);
#pragma unroll
  for (int q = 0; q < 8; ++q)
    row[q ^ (lane & 7)] = zero ? make_uint4(0, 0, 0, 0)
                               : make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
  __syncwarp();
}

// Rows row0 .. row0 + 31 (those < M) and columns col0 .. col0 + 31 (those < N)
// of an fp32 output from the staging block, one column a lane, for rows that TMA
// cannot store.
__device__ __forceinline__ void write_block(const TcProduct& p, const float* sw, int lane, int row0, int col0,
                                            int64_t d_base) {
  if (col0 + lane < p.N) {
    const int rows = min(32, p.M - row0);
    float* d = static_cast<float*>(p.D) + d_base + (int64_t)row0 * p.N + col0 + lane;
    const float* col = sw + (lane & 3);
#pragma unroll 8
    for (int rr = 0; rr < rows; ++rr) d[(int64_t)rr * p.N] = col[rr * 32 + (((lane >> 2) ^ (rr & 7)) << 2)];
  }
  __syncwarp();  // the block is overwritten next
}

// 32 rows x 64 columns of a 16-bit output from the block that stage_rounded
// wrote, for rows that TMA cannot store: two columns a lane where rows start on 4
// bytes, else one at a time.  (Aligned 16-byte windows put together by shifts,
// with single elements at a row's ends, took 1.3 times as long.)
__device__ __forceinline__ void write_rounded(const TcProduct& p, const uint8_t* sw, int lane, int row0, int col0,
                                              int64_t d_base) {
  const int rows = min(32, p.M - row0), n = p.N - col0;
  uint16_t* d = static_cast<uint16_t*>(p.D) + d_base + (int64_t)row0 * p.N + col0;
  if ((p.N & 1) == 0 && (reinterpret_cast<uintptr_t>(p.D) & 3) == 0) {
    if (2 * lane < n) {
#pragma unroll 8
      for (int rr = 0; rr < rows; ++rr)
        *reinterpret_cast<uint32_t*>(d + (int64_t)rr * p.N + 2 * lane) =
            *reinterpret_cast<const uint32_t*>(sw + rr * 128 + (((lane >> 2) ^ (rr & 7)) << 4) + (lane & 3) * 4);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = h * 32 + lane;
      if (c < n) {
#pragma unroll 8
        for (int rr = 0; rr < rows; ++rr)
          d[(int64_t)rr * p.N + c] =
              *reinterpret_cast<const uint16_t*>(sw + rr * 128 + (((c >> 3) ^ (rr & 7)) << 4) + (c & 7) * 2);
      }
    }
  }
  __syncwarp();  // the block is overwritten next
}

// 32 rows x 64 columns (two TMEM loads of 32) rounded into the staging block in
// the layout of a 128-byte-swizzled TMA box.
__device__ __forceinline__ void stage_rounded(const float* v, uint8_t* sw, int lane, bool zero, int type) {
  uint4* row = reinterpret_cast<uint4*>(sw + lane * 128);
#pragma unroll
  for (int q = 0; q < 8; ++q) row[q ^ (lane & 7)] = zero ? make_uint4(0, 0, 0, 0) : pack8(v + 8 * q, type);
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
               "r"(src), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// The same block of one part of a split sum, in fp32 (pitch a multiple of 32).
__device__ __forceinline__ void write_part(const TcProduct& p, const float* sw, int lane, int row0, int col0,
                                           int split) {
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    const int rr = it * 4 + (lane >> 3), row = row0 + rr, q = lane & 7;
    const uint4 u = reinterpret_cast<const uint4*>(sw + rr * 32)[q ^ (rr & 7)];
    if (row < p.M && col0 < p.part_pitch)
      *reinterpret_cast<uint4*>(p.part + ((int64_t)split * p.M + row) * p.part_pitch + col0 + q * 4) = u;
  }
  __syncwarp();
}

// 16-bit units from .. to - 1 to zero, by all epilogue threads of the grid.
__device__ void zero_span(void* base, int64_t from, int64_t to, int64_t tid, int64_t n_threads) {
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

// BN = 0: rows form (M operand stored across the sum if AMN); else sum form.
template <bool AMN, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_tc(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ NMaps mapsB,
                const __grid_constant__ CUtensorMap mapD, const __grid_constant__ TcProduct p) {
  using L = Smem<BN>;
  const int S = BN == 0 ? p.stages : L::kStages;
  const uint32_t stage_bytes = BN == 0 ? rows_stage_bytes(p.tile_rows) : L::kStage;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * kMaxStages + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  const uint32_t bar0 = saddr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto fix = [&](int s) { return bar0 + 8u * (2 * kMaxStages + s); };
  auto tfull = [&](int a) { return bar0 + 8u * (3 * kMaxStages + a); };
  auto tempty = [&](int a) { return bar0 + 8u * (3 * kMaxStages + 2 + a); };
  const uint32_t done = bar0 + 8u * (3 * kMaxStages + 4);
  constexpr bool kRows = BN == 0;
  constexpr int kAccCols = kRows ? 256 : BN;
  constexpr uint32_t kCols = 2 * kAccCols;  // two accumulators
  const bool group_sum = !kRows && p.mode == GROUP_SUM;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      // GROUP_SUM: a block may be handed over by each CTA's helper, so each CTA arrives
      mbar_init(full(s), group_sum ? 2 : 1);
      mbar_init(empty(s), 1);
      mbar_init(fix(s), 1);
    }
    for (int a = 0; a < 2; ++a) { mbar_init(tfull(a), 1); mbar_init(tempty(a), 2 * kEpiWarps); }
    mbar_init(done, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mapA) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mapsB.box[0]) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_barrier();  // both CTAs' barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_launch_next();
  grid_wait();  // all that runs before this launch is done: its results may be read, its inputs overwritten
  Walk<BN> walk(p);
  Item it;
  bool more = walk.next(p, it);

  // The producer's and the issuer's loops have to stay ahead of the MMAs (about
  // 500 cycles a block).  Whole warps run them, so that their addresses and
  // descriptors stay in uniform registers, and one elected lane issues.
  if (warp == 0) {  // ---- TMA producer (both CTAs) ----
    const uint32_t ring = saddr(smem), full_leader = map_to(full(0), 0);
    int s = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (; ok && more; more = walk.next(p, it)) {
      const int arow = it.m0 + (int)rank * 128;
      // rows form: this CTA's half of the tile's tokens
      const int half = kRows ? mma_cols(it) / 2 : BN / 2;
      const int brow = it.n0 + (int)rank * half;
      int box = 0;
      if (kRows) while (box_rows(box) < half) ++box;
      const CUtensorMap* mapB = &mapsB.box[box];
      const uint32_t bytes = kRows ? L::kA + (uint32_t)box_rows(box) * (BK * 2) : L::kStage;
      for (int i = p.first; ok && i < kProducts; ++i) {
        const int planes = p.first == 0 ? 3 : 1;
        const int ae = (kRows ? it.e * planes : 0) + plane_m(i), be = plane_n(i);
        for (int k = it.k0; k < it.k1; k += BK) {
          if (!(ok = mbar_wait(empty(s), ph, abort_flag, p.err, 1))) break;
          const uint32_t sa = ring + s * stage_bytes, sb = sa + L::kA;
          if (elect_lane()) {
            uint32_t bar = full_leader + 8u * s;  // where this CTA's copies are counted: the leader's ring
            if (group_sum && it.k1 - k < BK) {    // or, for a range's last rows, its own helper
              bar = fix(s);
              mbar_expect_tx(bar, bytes);
            } else if (rank == 0) {
              mbar_expect_tx(full(s), 2 * bytes);
            } else if (group_sum) {
              mbar_arrive_cluster(bar);
            }
            if (AMN) {
              tma_load_3d_pair(sa, &mapA, bar, arow, k, ae);
              tma_load_3d_pair(sa + 64 * BK * 2, &mapA, bar, arow + 64, k, ae);
            } else {
              tma_load_3d_pair(sa, &mapA, bar, k, arow, ae);
            }
            if constexpr (kRows) {
              tma_load_3d_pair(sb, mapB, bar, k, brow, be);
            } else {
#pragma unroll
              for (int c = 0; c < BN / 128; ++c)
                tma_load_3d_pair(sb + c * (64 * BK * 2), mapB, bar, brow + c * 64, k, be);
            }
          }
          __syncwarp();
          if (++s == S) { s = 0; ph ^= 1; }
        }
      }
    }
    if (!ok) {  // gave up: let the copies in flight land before the block leaves
      const long long t0 = clock64();
      while (clock64() - t0 < (1ll << 21)) {}
    }
  } else if (warp == 1) {
    if (rank == 0) {  // ---- MMA issuer (leader only) ----
      // descriptors of stage 0; a stage further is stage_bytes / 16 more in the
      // low word, 16 steps of the sum further kStepA / kStepB more
      const uint64_t da = AMN ? smem_desc(saddr(smem), 64 * BK * 2, 1024) : smem_desc(saddr(smem), 16, 1024);
      const uint64_t db = kRows ? smem_desc(saddr(smem) + L::kA, 16, 1024)
                                : smem_desc(saddr(smem) + L::kA, 64 * BK * 2, 1024);
      constexpr uint64_t kStepA = AMN ? 2048 / 16 : 32 / 16, kStepB = kRows ? 32 / 16 : 2048 / 16;
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 1;
      bool ok = true;
      for (; more; more = walk.next(p, it)) {
        if (!(ok = mbar_wait(tempty(acc), aph, abort_flag, p.err, 2))) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kAccCols);
        const uint32_t idesc = instr_desc(p.type == DT_F16 ? 0u : 1u, BM, kRows ? mma_cols(it) : BN, !kRows, AMN);
        uint32_t add = 0;  // the tile's first MMA overwrites
        for (int i = p.first; ok && i < kProducts; ++i) {
          for (int k = it.k0; k < it.k1; k += BK) {
            if (!(ok = mbar_wait(full(s), ph, abort_flag, p.err, 4))) break;
            if (group_sum && it.k1 - k < BK) mbar_acquire_cluster(full(s), ph);  // both helpers' zeros
            tc_fence_after();
            const uint64_t a = da + s * (stage_bytes >> 4), b = db + s * (stage_bytes >> 4);
            if (elect_lane()) {
              umma_pair(d_tmem, a, b, idesc, add);
              if (it.k1 - k >= BK) {
                umma_pair(d_tmem, a + kStepA, b + kStepB, idesc, 1);
                umma_pair(d_tmem, a + 2 * kStepA, b + 2 * kStepB, idesc, 1);
                umma_pair(d_tmem, a + 3 * kStepA, b + 3 * kStepB, idesc, 1);
              } else {  // behind the sum's end there are only zeros: skipped
                for (int kk = 1; kk * 16 < it.k1 - k; ++kk)
                  umma_pair(d_tmem, a + kk * kStepA, b + kk * kStepB, idesc, 1);
              }
              umma_commit_pair(empty(s), 3);  // frees the stage in both CTAs once these MMAs retire
            }
            __syncwarp();
            add = 1;
            if (++s == S) { s = 0; ph ^= 1; }
          }
        }
        if (!ok) break;
        if (elect_lane()) umma_commit_pair(tfull(acc), 3);
        __syncwarp();
        if (++acc == 2) { acc = 0; aph ^= 1; }
      }
      // every MMA issued has completed before TMEM and shared memory go away
      // (waited for even after an abort, so the wait ignores the abort flag)
      if (elect_lane()) umma_commit_pair(done, 1);
      __syncwarp();
      volatile int keep_waiting = 0;
      mbar_wait(done, 0, &keep_waiting, p.err, 16);
    }
  } else if (warp < 2 + kEpiWarps) {  // ---- epilogue ----
    const int quarter = warp & 3;     // TMEM lanes this warp may read
    const int half = (warp - 2) >> 2; // which half of the tile's columns
    int acc = 0;
    uint32_t aph = 0;
    for (; more; more = walk.next(p, it)) {
      const long long limit = sum_wait(it.k1 - it.k0, kProducts - p.first);
      if (!mbar_wait(tfull(acc), aph, abort_flag, p.err, 8, limit)) break;
      tc_fence_after();
      const uint32_t tacc = tmem_base + (uint32_t)(acc * kAccCols) + ((uint32_t)(quarter * 32) << 16);
      const int row0 = it.m0 + (int)rank * 128 + quarter * 32;
      if constexpr (kRows) {
        // the warps of a quarter take turns at 32 tokens
        for (int c = half * 32; row0 < p.M && it.n0 + c < it.n_end; c += 64) {
          float v[32];
          __syncwarp();  // lanes without a feature skip the rest of the loop
          tmem_ld32(tacc + (uint32_t)c, reinterpret_cast<uint32_t*>(v));
          const int n = min(32, it.n_end - it.n0 - c), f = row0 + lane;
          const int64_t t0 = it.n0 + c;
          if (f >= p.M) continue;
          if (p.splits > 1) {
            float* dst = p.part + ((int64_t)it.split * p.rows + t0) * p.part_pitch + f;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i < n) dst[i * p.part_pitch] = v[i];
          } else if (p.type == DT_BF16) {
            write_tokens<__nv_bfloat16>(p, v, it.e, f, t0, n);
          } else if (p.type == DT_F16) {
            write_tokens<__half>(p, v, it.e, f, t0, n);
          } else {
            write_tokens<float>(p, v, it.e, f, t0, n);
          }
        }
      } else {
        uint8_t* sw = smem + L::kEpi + (warp - 2) * 4096;
        const bool zero = it.k0 >= it.k1;
        const int c0 = half * (BN / 2);  // this warp's columns of the tile
        const int64_t d_base = group_sum ? (int64_t)it.e * p.M * p.N : 0;
        if (p.splits == 1 && p.type != DT_F32) {
#pragma unroll 1
          for (int c = c0; c < c0 + BN / 2; c += 64) {
            if (it.n0 + c >= p.N || row0 >= p.M) break;  // the same for the whole warp
            float v[64];
            tmem_ld32_async(tacc + (uint32_t)c, reinterpret_cast<uint32_t*>(v));
            tmem_ld32_async(tacc + (uint32_t)c + 32, reinterpret_cast<uint32_t*>(v) + 32);
            // the last store has read the block
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
            tmem_wait_ld();
            stage_rounded(v, sw, lane, zero, p.type);
            if (!p.vec) {
              __syncwarp();
              write_rounded(p, sw, lane, row0, it.n0 + c, d_base);
              continue;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) tma_store_3d(&mapD, saddr(sw), it.n0 + c, row0, it.e);
          }
        } else {
#pragma unroll 1
          for (int c = c0; c < c0 + BN / 2; c += 32) {
            if (it.n0 + c >= p.N || row0 >= p.M) break;
            if (p.splits == 1 && p.vec) {  // fp32: a staged block is a TMA box of 32 x 32
              if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
              __syncwarp();
              stage_block(tacc + (uint32_t)c, reinterpret_cast<float*>(sw), lane, zero);
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
              if (lane == 0) tma_store_3d(&mapD, saddr(sw), it.n0 + c, row0, it.e);
              continue;
            }
            stage_block(tacc + (uint32_t)c, reinterpret_cast<float*>(sw), lane, zero);
            if (p.splits > 1) write_part(p, reinterpret_cast<float*>(sw), lane, row0, it.n0 + c, it.split);
            else write_block(p, reinterpret_cast<float*>(sw), lane, row0, it.n0 + c, d_base);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to(tempty(acc), 0));
      if (++acc == 2) { acc = 0; aph ^= 1; }
    }
    if (!kRows && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (p.mode == GROUP_ROWS) {  // rows of no expert: before the first range and behind the last
      const int64_t row = (p.type == DT_F32 ? 2ll : 1ll) * p.M;  // in 16-bit units
      const int64_t head = row * range_at(p, 0, p.rows);
      const int64_t from = max(head, row * range_at(p, p.experts, p.rows)), to = row * p.rows;
      const int64_t tid = (int64_t)blockIdx.x * (32 * kEpiWarps) + threadIdx.x - 64;
      const int64_t n_threads = (int64_t)gridDim.x * (32 * kEpiWarps);
      zero_span(p.D, 0, head, tid, n_threads);
      zero_span(p.D, from, to, tid, n_threads);
      if (p.preact) {
        zero_span(p.preact, 0, head, tid, n_threads);
        zero_span(p.preact, from, to, tid, n_threads);
      }
    }
  } else if (group_sum) {  // ---- helper: zeros behind a range's end ----
    int s = 0;
    uint32_t fph = 0;  // parity of each stage's fix barrier
    bool ok = true;
    for (; ok && more; more = walk.next(p, it)) {
      const int blocks = (it.k1 - it.k0 + BK - 1) / BK, rem = (it.k1 - it.k0) % BK;
      for (int i = p.first; ok && i < kProducts; ++i) {
        if (rem) {
          const int st = (s + blocks - 1) % S;
          // (the sum's last block: it comes when all others have been taken)
          if (!(ok = mbar_wait(fix(st), (fph >> st) & 1, abort_flag, p.err, 32, sum_wait(it.k1 - it.k0, 1)))) break;
          fph ^= 1u << st;
          uint8_t* stage = smem + st * L::kStage;
          for (int box = 0; box < (int)(L::kStage / (64 * BK * 2)); ++box)  // 64 rows of k, 128 bytes each
            for (int i = rem * 8 + lane; i < BK * 8; i += 32)
              reinterpret_cast<uint4*>(stage + box * (64 * BK * 2))[i] = make_uint4(0, 0, 0, 0);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive_release_cluster(map_to(full(st), 0));
        }
        s = (s + blocks) % S;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // neither CTA leaves while the pair's MMAs or copies may touch it
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kCols) : "memory");
  }
}

// Joins the parts of a split sum, in order, and runs the epilogue: output
// [rows][cols], VEC columns a thread: 8 (16-bit types whose rows start on 16
// bytes) or 1.
template <int VEC>
__global__ void __launch_bounds__(256) k_linear_join(const __grid_constant__ TcProduct p, int rows, int cols) {
  grid_launch_next();
  grid_wait();
  const int64_t per_row = cols / VEC;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= per_row * rows) return;
  const int64_t row = i / per_row, c = (i - row * per_row) * VEC;
  const float* part = p.part + row * p.part_pitch + c;
  const int64_t between = (int64_t)rows * p.part_pitch;
  if constexpr (VEC == 1) {
    float z = 0.f;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) z += part[s * between];
    if (p.bias) z += ld_el(p.bias, c, p.type);
    if (p.preact) st_el(p.preact, row * cols + c, z, p.type);
    z = p.type == DT_F32 ? activate<false>(z, p.act) : activate<true>(z, p.act);
    if (p.residual) z += ld_el(p.residual, row * p.r_m + c, p.type);
    st_el(p.D, row * cols + c, z, p.type);
  } else {
    float v[8] = {}, b[8];
    for (int s = 0; s < p.splits; ++s) {
      const uint4* src = reinterpret_cast<const uint4*>(part + s * between);
      float f[8];
      u4_to_f4x2(src[0], src[1], f);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += f[k];
    }
    if (p.bias) {
      unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.bias) + c), b, p.type);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += b[k];
    }
    if (p.preact) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.preact) + row * cols + c) = pack8(v, p.type);
    activate_n<8, true>(v, p.act);
    if (p.residual) {
      unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.residual) + row * p.r_m + c), b, p.type);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += b[k];
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.D) + row * cols + c) = pack8(v, p.type);
  }
}

// Eight 16-bit elements from any address: two aligned 16-byte loads and a shift
// where both lie in begin .. end, else element by element; nothing outside is
// read.  The loads (fetch) are apart from the rest (finish) so that a thread has
// several pieces in flight.
struct Unaligned {
  uintptr_t begin, end;
  struct Piece {
    uint4 v0, v1;
  };
  __device__ __forceinline__ bool inside(const uint16_t* p) const {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15);
    return lo >= begin && lo + 32 <= end;
  }
  __device__ __forceinline__ Piece fetch(const uint16_t* p, bool wanted) const {
    Piece u{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (wanted && inside(p)) {
      const uint4* lo = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15));
      u.v0 = __ldcs(lo);
      u.v1 = __ldcs(lo + 1);
    }
    return u;
  }
  // The elements, those from the n-th on as zeros.
  __device__ __forceinline__ uint4 finish(const Piece& s, const uint16_t* p, int64_t n) const {
    const uint32_t w[8] = {s.v0.x, s.v0.y, s.v0.z, s.v0.w, s.v1.x, s.v1.y, s.v1.z, s.v1.w};
    const int word = (int)(reinterpret_cast<uintptr_t>(p) & 15) >> 2;
    const int bits = (int)(reinterpret_cast<uintptr_t>(p) & 3) * 8;
    uint32_t o[5];
#pragma unroll
    for (int i = 0; i < 5; ++i)  // w[word + i] without an indexed register
      o[i] = word == 0 ? w[i] : word == 1 ? w[i + 1] : word == 2 ? w[i + 2] : w[i + 3];
    const uint4 u = make_uint4(__funnelshift_r(o[0], o[1], bits), __funnelshift_r(o[1], o[2], bits),
                               __funnelshift_r(o[2], o[3], bits), __funnelshift_r(o[3], o[4], bits));
    if (n >= 8 && inside(p)) return u;
    alignas(16) uint16_t h[8];  // a row's end, or the buffer's
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = i < n ? p[i] : (uint16_t)0;
    return *reinterpret_cast<const uint4*>(h);
  }
};

// Operands that TMA cannot read as they are, up to two tensors a launch.  fp32
// rows become three bf16 planes, dst [batch][3][rows][pitch]: each is what is left
// rounded to nearest, whose remainder is exact in fp32, and a non-finite value goes
// into the low plane beside +-1, 0.  16-bit rows are copied, dst [batch][rows][pitch].
// Padding is zero.
// A thread takes a piece of eight elements of kPrepRows rows.
constexpr int kPrepRows = 4;
struct PrepBlocks {
  RowsJob job;
  int64_t blocks;              // of this job
  int64_t row_blocks;
  int col_blocks, per;         // blocks along a row, pieces of each
};

__device__ __forceinline__ void load_piece(const float* s, int64_t n, float* f) {
  if (n >= 8 && (reinterpret_cast<uintptr_t>(s) & 15) == 0) {
    u4_to_f4x2(__ldcs(reinterpret_cast<const uint4*>(s)), __ldcs(reinterpret_cast<const uint4*>(s) + 1), f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? s[i] : 0.f;
  }
}
__device__ __forceinline__ void split_piece(const float* f, uint4* plane) {
  alignas(16) __nv_bfloat16 h[3][8];
  bool plain = true;  // not infinite or NaN, nor carried there by the first rounding
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    plain &= fabsf(f[i]) < __int_as_float(0x7f7f8000);
    h[0][i] = __float2bfloat16_rn(f[i]);
    const float v = f[i] - __bfloat162float(h[0][i]);
    h[1][i] = __float2bfloat16_rn(v);
    h[2][i] = __float2bfloat16_rn(v - __bfloat162float(h[1][i]));
  }
  if (!plain) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (fabsf(f[i]) < __int_as_float(0x7f7f8000)) continue;
      if (fabsf(f[i]) < __int_as_float(0x7f800000)) {  // cut off, not rounded up
        const float top = __uint_as_float(__float_as_uint(f[i]) & 0xffff0000u), v = f[i] - top;
        h[0][i] = __float2bfloat16_rn(top);
        h[1][i] = __float2bfloat16_rn(v);
        h[2][i] = __float2bfloat16_rn(v - __bfloat162float(h[1][i]));
      } else {
        h[0][i] = __float2bfloat16_rn(copysignf(1.f, f[i]));
        h[1][i] = __float2bfloat16_rn(0.f);
        h[2][i] = __float2bfloat16_rn(f[i]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) plane[k] = *reinterpret_cast<const uint4*>(h[k]);
}

template <bool kSplit>
__global__ void __launch_bounds__(256) k_prepare_rows(const __grid_constant__ PrepBlocks first,
                                                      const __grid_constant__ PrepBlocks second) {
  grid_launch_next();
  grid_wait();
  int64_t at = blockIdx.x;
  const bool two = at >= first.blocks;
  if (two) at -= first.blocks;
  const PrepBlocks& q = two ? second : first;
  const RowsJob& j = q.job;
  if ((int)threadIdx.x >= q.per) return;
  const int64_t c = ((at % q.col_blocks) * q.per + threadIdx.x) * 8;
  at /= q.col_blocks;
  const int64_t r0 = at % q.row_blocks * kPrepRows, b = at / q.row_blocks;
  if (c >= j.pitch || (j.offsets && j.offsets[b] >= j.offsets[b + 1])) return;
  if constexpr (kSplit) {
    const float* s = static_cast<const float*>(j.src) + b * j.batch_stride + r0 * j.stride + c;
    float f[kPrepRows][8];  // in flight together
#pragma unroll
    for (int k = 0; k < kPrepRows; ++k)
      if (r0 + k < j.rows) load_piece(s + k * j.stride, j.cols - c, f[k]);
#pragma unroll
    for (int k = 0; k < kPrepRows; ++k) {
      if (r0 + k >= j.rows) break;
      uint4 u[3];
      split_piece(f[k], u);
#pragma unroll
      for (int p = 0; p < 3; ++p)
        *reinterpret_cast<uint4*>(j.dst + ((b * 3 + p) * j.rows + r0 + k) * j.pitch + c) = u[p];
    }
  } else {
    const uint16_t* s = static_cast<const uint16_t*>(j.src) + b * j.batch_stride + r0 * j.stride + c;
    const uintptr_t begin = reinterpret_cast<uintptr_t>(j.src);
    const Unaligned d{begin,
                      begin + (uintptr_t)(((j.batch - 1) * j.batch_stride + (j.rows - 1) * j.stride + j.cols) * 2)};
    Unaligned::Piece u[kPrepRows];
#pragma unroll
    for (int k = 0; k < kPrepRows; ++k) u[k] = d.fetch(s + k * j.stride, r0 + k < j.rows);
#pragma unroll
    for (int k = 0; k < kPrepRows; ++k)
      if (r0 + k < j.rows)
        *reinterpret_cast<uint4*>(j.dst + (b * j.rows + r0 + k) * j.pitch + c) =
            d.finish(u[k], s + k * j.stride, j.cols - c);
  }
}

bool aligned_rows(const void* p, int64_t stride, int type) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % (type == DT_F32 ? 4 : 8) == 0;
}
// Operands are bf16 planes for fp32.
int operand_type(const TcProduct& q) { return q.type == DT_F16 ? NS_F16 : NS_BF16; }
int planes(const TcProduct& q) { return q.type == DT_F32 ? 3 : 1; }

// The kernel with its function attributes set (once per device).
template <bool AMN, int BN>
cudaError_t launch(const CUtensorMap& ma, const NMaps& mb, const CUtensorMap& md, const TcProduct& q,
                   int64_t items, cudaStream_t s) {
  auto fn = k_linear_tc<AMN, BN>;
  static bool ready[64] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !ready[dev]) {
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<BN>::kTotal);
      if (e != cudaSuccess) return e;
      if (dev < 64) ready[dev] = true;
    }
  }
  const int64_t most = num_sms() / 2;
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3((unsigned)(2 * (items < 1 ? 1 : (items < most ? items : most))));
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = Smem<BN>::kTotal;
  lc.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 2;
  return cudaLaunchKernelEx(&lc, fn, ma, mb, md, q);
}

// Rows form of D[p.M rows][p.N features]: M operand p.B (the weights).
cudaError_t run_rows(const Product& p, TcProduct q, cudaStream_t s) {
  const int type = operand_type(q), np = planes(q);
  const int64_t mats = np * (p.mode == GROUP_ROWS ? p.experts : 1);
  const bool across = p.b_k != 1;  // weights stored across the sum
  const int64_t between = mats > 1 ? p.b_e : (across ? p.K * p.b_k : p.N * p.b_n);
  CUtensorMap mw;
  NMaps mx;
  cudaError_t e = across ? tc_encode_map(&mw, p.B, type, p.N, p.K, mats, p.b_k, between, 64, 64)
                         : tc_encode_map(&mw, p.B, type, p.K, p.N, mats, p.b_n, between, 64, 128);
  for (int b = 0; b < kBoxes && e == cudaSuccess; ++b)
    e = tc_encode_map(&mx.box[b], p.A, type, p.K, p.M, np, p.a_m, p.M * p.a_m, 64, (uint32_t)box_rows(b));
  if (e != cudaSuccess) return e;
  int64_t tt = (p.M + q.tile_rows - 1) / q.tile_rows;
  if (p.mode == GROUP_ROWS) tt = p.M / q.tile_rows + (p.M < p.experts ? p.M : p.experts);  // at most
  const int64_t items = tt * q.tiles_m * q.splits;
  return across ? launch<true, 0>(mw, mx, mw, q, items, s) : launch<false, 0>(mw, mx, mw, q, items, s);
}

template <int BN>
cudaError_t run_sum(const Product& p, const TcProduct& q, cudaStream_t s) {
  const int type = operand_type(q), np = planes(q);
  const int64_t mats = p.mode == GROUP_SUM ? p.experts : 1;
  CUtensorMap ma, md;
  NMaps mb{};
  cudaError_t e = tc_encode_map(&ma, p.A, type, p.M, p.K, np, p.a_k, p.K * p.a_k, 64, 64);
  if (e == cudaSuccess) e = tc_encode_map(&mb.box[0], p.B, type, p.N, p.K, np, p.b_k, p.K * p.b_k, 64, 64);
  md = ma;
  if (e == cudaSuccess && q.vec)
    e = tc_encode_map(&md, p.D, q.type == DT_F32 ? NS_F32 : type, p.N, p.M, mats, p.N, p.M * p.N,
                      q.type == DT_F32 ? 32 : 64, 32);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)q.tiles_m * q.tiles_n * (p.mode == GROUP_SUM ? p.experts : q.splits);
  return launch<true, BN>(ma, mb, md, q, items, s);
}

// y and dx sum along the rows of A; dw sums across them.
bool rows_form(const Product& p) { return p.a_k == 1; }

}  // namespace

int num_sms() {
  static int n = [] {
    int dev = 0, v = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    return v > 0 ? v : 152;
  }();
  return n;
}

cudaError_t ops_error_word(int** err) {
  static int* addr[64] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (!addr[dev]) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_err);
    if (e != cudaSuccess) return e;
    addr[dev] = static_cast<int*>(p);
  }
  *err = addr[dev];
  return cudaSuccess;
}

// The tile and the parts of the sum with the least estimated time, in us on one
// GB300.  A pair takes 0.28 us for 64 steps of the sum on 256 columns, in
// proportion for fewer, but no less than 0.2 us (an operand of 256 rows has to
// reach the tensor cores all the same), and about 1 us to start and end a tile.
// All pairs together read weights at 6.2 TB/s.  Parts of the sum cost a launch
// and their traffic.
TilePlan tile_plan(const Product& p) {
  const int64_t pairs = num_sms() / 2;
  const int64_t kb = (p.K + BK - 1) / BK;
  const bool rows = rows_form(p);
  TilePlan best{};
  double best_t = 1e30;
  const auto offer = [&](int bn, int tile_rows, int64_t tiles, double cols, double blocks, double bytes) {
    const double per_kb = (p.dtype == DT_F32 ? 6 : 1) * (0.28 * cols / 256 > 0.2 ? 0.28 * cols / 256 : 0.2);
    for (int s = 1; s <= 16; ++s) {
      if (s > 1 && (p.mode != GROUP_NONE || kb * (p.dtype == DT_F32 ? 4 : 1) / s < 4)) break;
      const double waves = (double)((tiles * s + pairs - 1) / pairs), uneven = waves * pairs / (double)(tiles * s);
      double t = waves * (blocks / s * per_kb + 1.0);
      const double stream = bytes / 6.2e6 * uneven;
      if (t < stream) t = stream;
      if (s > 1) t += 2.5 + (double)p.M * p.N * 8.0 * s / 5e6;
      if (t < best_t * 0.98) { best_t = t; best = {bn, tile_rows, s, 0}; }
    }
  };
  if (rows) {
    const int64_t tm = (p.N + BM - 1) / BM;
    const int64_t ranges = p.mode == GROUP_ROWS ? (p.M < p.experts ? p.M : p.experts) : 1;
    const int64_t each = (p.M + ranges - 1) / ranges;
    const double bytes = (p.dtype == DT_F32 ? 12.0 : 2.0) * ranges * p.N * p.K;
    for (int tr : {256, 128, 64}) {
      const int64_t tt = (each + tr - 1) / tr;
      const int64_t cols = ((each + tt - 1) / tt + 31) / 32 * 32;
      // a range often has more rows than the average: not where that would
      // need another tile.  (The host knows the average only.  A range far above it
      // reads its weights once a tile, mostly from L2: 64 experts [7168, 2048], 2048
      // rows, 270 us spread evenly, 272 with 512 of them in one expert, 288 with 1024.)
      if (p.mode == GROUP_ROWS && tr < 256 && 2 * each > tr) continue;
      offer(0, tr, tm * tt * ranges, (double)cols, (double)kb, bytes);
    }
  } else {
    for (int bn : {256, 128}) {
      int64_t tiles = (p.M + BM - 1) / BM * ((p.N + bn - 1) / bn);
      double blocks = (double)kb;
      if (p.mode == GROUP_SUM) { tiles *= p.experts; blocks = (double)kb / p.experts + 0.5; }
      offer(bn, 0, tiles, bn, blocks, 0.0);
    }
  }
  if (best.splits > 1) best.part_bytes = (int64_t)best.splits * p.M * ((p.N + 31) / 32 * 32) * 4;
  return best;
}

cudaError_t launch_linear_tc(const Product& p, const TilePlan& t, float* part, cudaStream_t s) {
  TcProduct q{};
  q.mode = p.mode; q.experts = p.experts; q.splits = t.splits; q.offsets = p.offsets;
  q.K = (int)p.K;
  if (t.bn == 0) {
    q.rows = (int)p.M;
    q.M = (int)p.N;
    q.tiles_m = (int)((p.N + BM - 1) / BM);
    q.tile_rows = t.tile_rows;
    q.stages = rows_stages(t.tile_rows);
  } else {
    q.M = (int)p.M;
    q.N = (int)p.N;
    q.tiles_m = (int)((p.M + BM - 1) / BM);
    q.tiles_n = (int)((p.N + t.bn - 1) / t.bn);
  }
  q.type = p.dtype;
  q.first = p.dtype == DT_F32 ? 0 : kProducts - 1;
  q.act = p.act;
  q.D = p.D; q.bias = p.bias; q.residual = p.residual; q.r_m = p.r_m; q.preact = p.preact;
  q.vec = aligned_rows(p.D, p.N, q.type) && (!p.bias || aligned_rows(p.bias, p.N, q.type)) &&
          (!p.residual || aligned_rows(p.residual, p.r_m, q.type)) && (!p.preact || aligned_rows(p.preact, p.N, q.type));
  q.part = part;
  q.part_pitch = (p.N + 31) / 32 * 32;
  q.err = p.err;
  cudaError_t e = t.bn == 0 ? run_rows(p, q, s) : (t.bn == 256 ? run_sum<256>(p, q, s) : run_sum<128>(p, q, s));
  if (e == cudaSuccess && t.splits > 1) {
    // (vec: columns are whole pieces of 8)
    const bool vec = q.vec && q.type != DT_F32;
    const int64_t n = (vec ? p.N / 8 : p.N) * p.M;
    const dim3 grid((unsigned)((n + 255) / 256));
    e = vec ? launch_early(k_linear_join<8>, grid, dim3(256), 0, s, q, (int)p.M, (int)p.N)
            : launch_early(k_linear_join<1>, grid, dim3(256), 0, s, q, (int)p.M, (int)p.N);
  }
  return e;
}

cudaError_t launch_prepare_rows(bool split, const RowsJob& first, const RowsJob& second, cudaStream_t s) {
  unsigned threads = 32;
  const auto blocks = [&](const RowsJob& j) {
    PrepBlocks p{j, 0, 1, 1, 1};
    if (j.batch == 0) return p;
    const int64_t pieces = j.pitch / 8;
    p.col_blocks = (int)((pieces + 255) / 256);
    p.per = (int)((pieces + p.col_blocks - 1) / p.col_blocks);
    p.row_blocks = (j.rows + kPrepRows - 1) / kPrepRows;
    p.blocks = j.batch * p.row_blocks * p.col_blocks;
    threads = std::max(threads, (unsigned)((p.per + 31) / 32 * 32));
    return p;
  };
  const PrepBlocks a = blocks(first), b = blocks(second);
  const dim3 grid((unsigned)(a.blocks + b.blocks));
  return split ? launch_early(k_prepare_rows<true>, grid, dim3(threads), 0, s, a, b)
               : launch_early(k_prepare_rows<false>, grid, dim3(threads), 0, s, a, b);
}

}  // namespace muon
