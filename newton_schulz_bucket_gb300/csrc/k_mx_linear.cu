// A layer's product of microscaled 4-bit operands on the tensor cores: y =
// act(x W + b) + r with the weights held in 4 bits and the token rows rounded to 4
// bits before (k_mx_quantize.cu), fp32 sums.
//
// The block-scaled MMA (tcgen05.mma kind::mxf4) multiplies 64 steps of the sum at a
// time and takes the operands' scales from TMEM: for every 128 steps a 32-bit word a row
// (four scales), row r in lane r % 32, column r / 32, the same in all four quarters of
// the lanes.  Scales are held by rows in memory, [rows][steps / 32]; four warps read
// 16 of them a lane (512 steps), scatter the words into that order in shared
// memory, and tcgen05.cp spreads them over TMEM just before the MMAs that use them.
// Each stage of the ring has scale columns of its own in TMEM, so the wait for the
// stage covers them too.
//
// Tiles are those of k_linear_tc.cu's rows form: a CTA pair computes 256 features x up
// to 192 tokens (two accumulators of 192 columns and 5 x 24 columns of scales fill
// TMEM), each CTA stages its 128 rows of weights and its half of the tokens, 256 steps a
// stage.  Up to 64 rows of one matrix take the form of k_linear_few.cu: 128 features a
// cluster of up to eight CTAs that share the sum.
#include <cuda.h>

#include <mutex>

#include "linear_tiles.cuh"
#include "mx.cuh"

namespace muon {

namespace {

constexpr int kStep = 256;                    // steps of the sum in a stage: 128 bytes a row
constexpr uint32_t kRowBytes = 128;
constexpr uint32_t kScaleA = 1024;            // a stage's scales: two words a row, 128 rows
constexpr int kScaleWarps = 4;

// ---- block-scaled MMA ----

// Instruction descriptor, kind::mxf4: both operands e2m1 along the sum, scales of 8
// exponent bits; `half`: which two of a word's four scales.
__host__ __device__ constexpr uint32_t mx_desc(int M, int N, uint32_t half) {
  return (2 * half) << 4 | 1u << 7 | 1u << 10 | (uint32_t)(N >> 3) << 17 | 1u << 23 | (uint32_t)(M >> 4) << 24 |
         (2 * half) << 29;
}
template <bool kPair>
__device__ __forceinline__ void umma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                        uint32_t accumulate) {
  if constexpr (kPair) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb)
        : "memory");
  }
}
// 32 lanes x 16 bytes of shared memory to four TMEM columns, in all four quarters.
template <bool kPair>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (kPair)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Descriptor of such a block: no swizzle, groups of eight 16-byte rows 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

// ---- scales ----

struct MxScales {
  const uint8_t* w;
  const uint8_t* x;
  int64_t w_pitch, x_pitch;
  int64_t w_matrix;            // bytes between experts' scales
  int blocks;                  // of a row
};

// Scales at .. at + 15 of a row, zero past the row's blocks.
__device__ __forceinline__ uint4 fetch_scales(const uint8_t* row, int at, int blocks, bool vec) {
  if (vec && at + 16 <= blocks) return *reinterpret_cast<const uint4*>(row + at);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at + 4 * i + k < blocks) w[i] |= (uint32_t)row[at + 4 * i + k] << (8 * k);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Word i of a lane's 16 scales into a stage: row group j of block `base`.
__device__ __forceinline__ void put_word(uint8_t* base, int lane, int j, uint32_t w) {
  *reinterpret_cast<uint32_t*>(base + lane * 16 + j * 4) = w;
}

// 16 scales of the lane's row of weights and of its token rows (one in each group of
// 128), on their way from memory to a stage.
template <int G>
struct ScaleSet {
  uint4 a, b[G];
  int stages;                  // of this set: 1 where the sum ends in its first half, 0: no set
  // weight row m, token rows n, n + 128 ..: absent ones (>= their ends) are zero
  __device__ __forceinline__ void fetch(const MxScales& q, int64_t mat, int m, int m_end, int n, int n_end, int k,
                                        int K, bool vw, bool vx) {
    const int at = k / kMxBlock;
    a = make_uint4(0, 0, 0, 0);
    if (m < m_end) a = fetch_scales(q.w + mat * q.w_matrix + m * q.w_pitch, at, q.blocks, vw);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      b[g] = make_uint4(0, 0, 0, 0);
      if (n + 128 * g < n_end) b[g] = fetch_scales(q.x + (n + 128 * g) * q.x_pitch, at, q.blocks, vx);
    }
    stages = K - k > kStep ? 2 : 1;
  }
  // Half h (256 steps) into a stage's scales.
  __device__ __forceinline__ void put(uint8_t* sa, uint8_t* sb, int lane, int j, int h) const {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      put_word(sa + c * 512, lane, j, h ? (c ? a.w : a.z) : (c ? a.y : a.x));
#pragma unroll
      for (int g = 0; g < G; ++g)
        put_word(sb + (c * G + g) * 512, lane, j, h ? (c ? b[g].w : b[g].z) : (c ? b[g].y : b[g].x));
    }
  }
};

__device__ __forceinline__ bool row_vec(const uint8_t* p, int64_t pitch) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && pitch % 16 == 0;
}

// ---- tiles in CTA pairs ----

constexpr int kThreads = 32 * (2 + kEpiWarps + kScaleWarps);
constexpr int kMaxStages = 9;
constexpr uint32_t kWeights = 128 * kRowBytes;
constexpr uint32_t kScaleB = 2048;
constexpr int kScaleCols = 8 + 16;             // of a stage in TMEM
__host__ __device__ constexpr uint32_t stage_bytes_of(int tile_rows) {
  return kWeights + (uint32_t)(tile_rows / 2) * kRowBytes + kScaleA + kScaleB;
}
constexpr uint32_t kRing = 221184;             // 8 stages of 128 tokens
__host__ __device__ constexpr int stages_of(int tile_rows) {
  const int smem = (int)(kRing / stage_bytes_of(tile_rows)), tmem = (512 - 2 * tile_rows) / kScaleCols;
  const int n = smem < tmem ? smem : tmem;
  return n < kMaxStages ? n : kMaxStages;
}
static_assert(stages_of(192) == 5 && stages_of(128) == 8 && stages_of(64) == kMaxStages, "ring depths");
static_assert(stage_bytes_of(192) % 1024 == 0 && stage_bytes_of(128) % 1024 == 0 && stage_bytes_of(64) % 1024 == 0,
              "stages start where the swizzle does");
constexpr uint32_t kSmem = kRing + 512 + 1024;
static_assert((2 * kMaxStages + 5) * 8 + 8 <= 512 && kSmem <= 227 * 1024, "shared memory layout");

__global__ void __launch_bounds__(kThreads, 1)
    k_mx_tiles(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ NMaps mapsX,
               const __grid_constant__ TcProduct p, const __grid_constant__ MxScales q) {
  const int S = p.stages;
  const uint32_t stage_bytes = stage_bytes_of(p.tile_rows);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kRing);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  const uint32_t bar0 = saddr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto tfull = [&](int a) { return bar0 + 8u * (2 * kMaxStages + a); };
  auto tempty = [&](int a) { return bar0 + 8u * (2 * kMaxStages + 2 + a); };
  const uint32_t done = bar0 + 8u * (2 * kMaxStages + 4);
  const uint32_t acc_cols = (uint32_t)p.tile_rows;
  // the scales' place in a stage
  const uint32_t sa_at = kWeights + (uint32_t)(p.tile_rows / 2) * kRowBytes, sb_at = sa_at + kScaleA;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1 + 2 * kScaleWarps);  // the copies of both CTAs, and their scale warps
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) { mbar_init(tfull(a), 1); mbar_init(tempty(a), 2 * kEpiWarps); }
    mbar_init(done, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mapW) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mapsX.box[0]) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(saddr(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_barrier();  // both CTAs' barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_launch_next();
  grid_wait();  // all that runs before this launch is done: its results may be read, its inputs overwritten
  Walk<0> walk(p);
  Item it;
  bool more = walk.next(p, it);

  if (warp == 0) {  // ---- TMA producer (both CTAs) ----
    const uint32_t ring = saddr(smem), full_leader = map_to(full(0), 0);
    int s = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (; ok && more; more = walk.next(p, it)) {
      const int wrow = it.m0 + (int)rank * 128;
      const int half = mma_cols(it) / 2, xrow = it.n0 + (int)rank * half;
      int box = 0;
      while (box_rows(box) < half) ++box;
      const CUtensorMap* mapX = &mapsX.box[box];
      const uint32_t bytes = kWeights + (uint32_t)box_rows(box) * kRowBytes;
      for (int k = 0; k < p.K; k += kStep) {
        if (!(ok = mbar_wait(empty(s), ph, abort_flag, p.err, 512))) break;
        if (elect_lane()) {
          const uint32_t sw = ring + s * stage_bytes, bar = full_leader + 8u * s;
          if (rank == 0) mbar_expect_tx(full(s), 2 * bytes);
          tma_load_3d_pair(sw, &mapW, bar, k / 4, wrow, it.e);
          tma_load_3d_pair(sw + kWeights, mapX, bar, k / 4, xrow, 0);
        }
        __syncwarp();
        if (++s == S) { s = 0; ph ^= 1; }
      }
    }
    if (!ok) {  // gave up: let the copies in flight land before the block leaves
      const long long t0 = clock64();
      while (clock64() - t0 < (1ll << 21)) {}
    }
  } else if (warp == 1) {
    if (rank == 0) {  // ---- MMA issuer (leader only) ----
      const uint64_t da = smem_desc(saddr(smem), 16, 1024), db = smem_desc(saddr(smem) + kWeights, 16, 1024);
      const uint64_t dsa = scale_desc(saddr(smem) + sa_at), dsb = scale_desc(saddr(smem) + sb_at);
      const uint32_t scales = tmem_base + 2 * acc_cols;
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 1;
      bool ok = true;
      for (; more; more = walk.next(p, it)) {
        if (!(ok = mbar_wait(tempty(acc), aph, abort_flag, p.err, 1024))) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)acc * acc_cols;
        const int cols = mma_cols(it);
        const uint32_t first = mx_desc(BM, cols, 0), second = mx_desc(BM, cols, 1);
        uint32_t add = 0;  // the tile's first MMA overwrites
        for (int k = 0; k < p.K; k += kStep) {
          if (!(ok = mbar_wait(full(s), ph, abort_flag, p.err, 2048))) break;
          mbar_acquire_cluster(full(s), ph);  // the other CTA's scales
          tc_fence_after();
          const uint64_t at = s * (stage_bytes >> 4);
          if (elect_lane()) {
            const uint32_t ta = scales + (uint32_t)(s * kScaleCols), tb = ta + 8;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (c && p.K - k <= 128) break;
              copy_scales<true>(ta + 4 * c, dsa + at + c * (512 >> 4));
              copy_scales<true>(tb + 8 * c, dsb + at + c * (1024 >> 4));
              if (cols > 128) copy_scales<true>(tb + 8 * c + 4, dsb + at + c * (1024 >> 4) + (512 >> 4));
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk * 64 >= p.K - k) break;
              umma_mx<true>(d_tmem, da + at + kk * 2, db + at + kk * 2, kk & 1 ? second : first, ta + 4 * (kk >> 1),
                            tb + 8 * (kk >> 1), add);
              add = 1;
            }
            umma_commit_pair(empty(s), 3);  // frees the stage in both CTAs once these MMAs retire
          }
          __syncwarp();
          add = 1;
          if (++s == S) { s = 0; ph ^= 1; }
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
    const int half = (warp - 2) >> 2; // the warps of a quarter take turns at 32 tokens
    int acc = 0;
    uint32_t aph = 0;
    for (; more; more = walk.next(p, it)) {
      if (!mbar_wait(tfull(acc), aph, abort_flag, p.err, 8, sum_wait(p.K, 1))) break;
      tc_fence_after();
      const uint32_t tacc = tmem_base + (uint32_t)acc * acc_cols + ((uint32_t)(quarter * 32) << 16);
      const int row0 = it.m0 + (int)rank * 128 + quarter * 32;
      for (int c = half * 32; row0 < p.M && it.n0 + c < it.n_end; c += 64) {
        float v[32];
        __syncwarp();  // lanes without a feature skip the rest of the loop
        tmem_ld32(tacc + (uint32_t)c, reinterpret_cast<uint32_t*>(v));
        const int n = min(32, it.n_end - it.n0 - c), f = row0 + lane;
        const int64_t t0 = it.n0 + c;
        if (f >= p.M) continue;
        if (p.type == DT_BF16) write_tokens<__nv_bfloat16>(p, v, it.e, f, t0, n);
        else if (p.type == DT_F16) write_tokens<__half>(p, v, it.e, f, t0, n);
        else write_tokens<float>(p, v, it.e, f, t0, n);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to(tempty(acc), 0));
      if (++acc == 2) { acc = 0; aph ^= 1; }
    }
    if (p.mode == GROUP_ROWS) {  // rows of no expert: before the first range and behind the last
      const int64_t row = (p.type == DT_F32 ? 2ll : 1ll) * p.M;  // in 16-bit units
      const int64_t head = row * range_at(p, 0, p.rows);
      const int64_t from = max(head, row * range_at(p, p.experts, p.rows)), to = row * p.rows;
      const int64_t tid = (int64_t)blockIdx.x * (32 * kEpiWarps) + threadIdx.x - 64;
      const int64_t n_threads = (int64_t)gridDim.x * (32 * kEpiWarps);
      zero_span(p.D, 0, head, tid, n_threads);
      zero_span(p.D, from, to, tid, n_threads);
    }
  } else {  // ---- scales (both CTAs) ----
    constexpr int kSets = 2;  // sets in flight: one is stored while the others' loads are under way
    const int j = warp - 2 - kEpiWarps;
    const bool vw = row_vec(q.w, q.w_pitch) && q.w_matrix % 16 == 0, vx = row_vec(q.x, q.x_pitch);
    ScaleSet<2> set[kSets];
    int k = 0;
    auto fetch = [&](ScaleSet<2>& t) {  // the next 512 steps of this tile, or of the next one
      t.stages = 0;
      if (!more) return;
      const int cols = mma_cols(it);
      t.fetch(q, it.e, it.m0 + (int)rank * 128 + 32 * j + lane, p.M, it.n0 + 32 * j + lane, min(it.n0 + cols, p.rows), k,
              p.K, vw, vx);
      k += 2 * kStep;
      if (k >= p.K) {
        k = 0;
        more = walk.next(p, it);
      }
    };
    const uint32_t full_leader = map_to(full(0), 0);
    int s = 0;
    uint32_t ph = 1;
    bool ok = true;
#pragma unroll
    for (int i = 0; i < kSets; ++i) fetch(set[i]);
    while (ok && set[0].stages) {
#pragma unroll
      for (int i = 0; i < kSets; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!ok || h >= set[i].stages) continue;
          if (!(ok = mbar_wait(empty(s), ph, abort_flag, p.err, 4096))) continue;
          uint8_t* stage = smem + s * stage_bytes;
          set[i].put(stage + sa_at, stage + sb_at, lane, j, h);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive_release_cluster(full_leader + 8u * s);
          if (++s == S) { s = 0; ph ^= 1; }
        }
        fetch(set[i]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // neither CTA leaves while the pair's MMAs or copies may touch it
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem_base) : "memory");
  }
}

// ---- few rows ----

constexpr int kFewThreads = 192;  // producer, MMA issuer, four warps for the scales and then the epilogue
constexpr uint32_t kFewRing = 110592;  // 5 stages of 128 + 16 rows; two CTAs an SM
constexpr uint32_t kFewSmem = kFewRing + 256 + 1024;
constexpr int kFewStages = 5;
constexpr uint32_t kFewScaleB = 1024;
constexpr int kFewScaleCols = 16;
constexpr int kFewTmem = 256;     // 64 of sums, 16 for each stage's scales
constexpr int kMaxShares = 8;

struct FewArgs {
  int rows, M, K;           // token rows, features, length of the sum
  int cols;                 // columns of an MMA: rows in steps of 16
  int stages;
  uint32_t stage_bytes;
  int type, act;
  void* D;
  const void* bias;
  const void* residual;
  int64_t r_m;
  int* err;
};

__device__ __forceinline__ float ld_shared_of(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_to(addr, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}

__global__ void __launch_bounds__(kFewThreads, 2)
    k_mx_few(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapX,
             const __grid_constant__ FewArgs p, const __grid_constant__ MxScales q) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kFewRing);  // full, empty, all
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kFewStages + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t bar0 = saddr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kFewStages + s); };
  const uint32_t all = bar0 + 8u * (2 * kFewStages);
  const int shares = (int)cluster_ctas(), rank = (int)cta_rank();
  const int m0 = (int)(blockIdx.x / shares) * 128;
  const uint32_t sa_at = kWeights + (uint32_t)p.cols * kRowBytes, sb_at = sa_at + kScaleA;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) { mbar_init(full(s), 1 + kScaleWarps); mbar_init(empty(s), 1); }
    mbar_init(all, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mapW) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mapX) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)),
                 "r"(kFewTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_launch_next();
  grid_wait();

  // this CTA's share of the sum, in pieces of 512 steps (a lane's 16 scales)
  const int pieces = (p.K + 2 * kStep - 1) / (2 * kStep);  // pieces * shares stays below 2^31
  const int k0 = pieces * rank / shares * (2 * kStep);
  const int k1 = rank + 1 == shares ? p.K : pieces * (rank + 1) / shares * (2 * kStep);
  if (warp == 0) {  // ---- TMA producer ----
    const uint32_t ring = saddr(smem);
    int s = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int k = k0; k < k1; k += kStep) {
      if (!(ok = mbar_wait(empty(s), ph, abort_flag, p.err, 8192))) break;
      if (elect_lane()) {
        const uint32_t sw = ring + s * p.stage_bytes;
        mbar_expect_tx(full(s), kWeights + (uint32_t)p.cols * kRowBytes);
        tma_load_3d(sw, &mapW, full(s), k / 4, m0, 0);
        tma_load_3d(sw + kWeights, &mapX, full(s), k / 4, 0, 0);
      }
      __syncwarp();
      if (++s == p.stages) { s = 0; ph ^= 1; }
    }
    if (!ok) {  // gave up: let the copies in flight land before the block leaves
      const long long t0 = clock64();
      while (clock64() - t0 < (1ll << 21)) {}
    }
  } else if (warp == 1) {  // ---- MMA issuer ----
    const uint64_t da = smem_desc(saddr(smem), 16, 1024), db = smem_desc(saddr(smem) + kWeights, 16, 1024);
    const uint64_t dsa = scale_desc(saddr(smem) + sa_at), dsb = scale_desc(saddr(smem) + sb_at);
    const uint32_t first = mx_desc(128, p.cols, 0), second = mx_desc(128, p.cols, 1);
    int s = 0;
    uint32_t ph = 0, add = 0;
    for (int k = k0; k < k1; k += kStep) {
      if (!mbar_wait(full(s), ph, abort_flag, p.err, 16384)) break;
      tc_fence_after();
      const uint64_t at = s * (p.stage_bytes >> 4);
      if (elect_lane()) {
        const uint32_t ta = tmem + 64 + (uint32_t)(s * kFewScaleCols), tb = ta + 8;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c && k1 - k <= 128) break;
          copy_scales<false>(ta + 4 * c, dsa + at + c * (512 >> 4));
          copy_scales<false>(tb + 4 * c, dsb + at + c * (512 >> 4));
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk * 64 >= k1 - k) break;
          umma_mx<false>(tmem, da + at + kk * 2, db + at + kk * 2, kk & 1 ? second : first, ta + 4 * (kk >> 1),
                         tb + 4 * (kk >> 1), add);
          add = 1;
        }
        umma_commit(empty(s));
      }
      __syncwarp();
      add = 1;
      if (++s == p.stages) { s = 0; ph ^= 1; }
    }
    if (elect_lane()) umma_commit(all);
    __syncwarp();
    volatile int keep_waiting = 0;
    mbar_wait(all, 0, &keep_waiting, p.err, 256);  // every MMA is done before the ring is reused
  } else {  // ---- scales ----
    constexpr int kSets = 3;
    const int j = warp - 2;
    const bool vw = row_vec(q.w, q.w_pitch), vx = row_vec(q.x, q.x_pitch);
    ScaleSet<1> set[kSets];
    int next = k0;
    auto fetch = [&](ScaleSet<1>& t) {
      t.stages = 0;
      if (next >= k1) return;
      t.fetch(q, 0, m0 + 32 * j + lane, p.M, 32 * j + lane, p.rows, next, k1, vw, vx);
      next += 2 * kStep;
    };
    int s = 0;
    uint32_t ph = 1;
    bool ok = true;
#pragma unroll
    for (int i = 0; i < kSets; ++i) fetch(set[i]);
    while (ok && set[0].stages) {
#pragma unroll
      for (int i = 0; i < kSets; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!ok || h >= set[i].stages) continue;
          if (!(ok = mbar_wait(empty(s), ph, abort_flag, p.err, 32768))) continue;
          uint8_t* stage = smem + s * p.stage_bytes;
          set[i].put(stage + sa_at, stage + sb_at, lane, j, h);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(full(s));
          if (++s == p.stages) { s = 0; ph ^= 1; }
        }
        fetch(set[i]);
      }
    }
  }
  // every copy has landed and been read, so the ring can take the partial sums:
  // [token][128 features]
  float* part = reinterpret_cast<float*>(smem);
  __syncthreads();
  if (warp >= 2) {
    tc_fence_after();
    const int quarter = warp & 3;
#pragma unroll 1
    for (int c = 0; c < p.rows; c += 32) {
      uint32_t v[32];
      tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c, v);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c + i < p.rows) part[(c + i) * 128 + quarter * 32 + lane] = __uint_as_float(v[i]);
    }
    tc_fence_before();
  }
  cluster_barrier();  // the partial sums of every share are in place
  for (int i = (int)threadIdx.x + rank * kFewThreads; i < p.rows * 128; i += kFewThreads * shares) {
    const int64_t t = i >> 7, f = m0 + (i & 127);
    if (f >= p.M) continue;
    float z = 0.f;
    for (int r = 0; r < shares; ++r) z += ld_shared_of(saddr(part + i), (uint32_t)r);
    if (p.bias) z += ld_el(p.bias, f, p.type);
    z = p.type == DT_F32 ? activate<false>(z, p.act) : activate<true>(z, p.act);
    if (p.residual) z += ld_el(p.residual, t * p.r_m + f, p.type);
    st_el(p.D, t * p.M + f, z, p.type);
  }
  cluster_barrier();  // no CTA leaves while another reads its sums
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kFewTmem) : "memory");
  }
}

// Shared memory beyond the default (once per device and kernel).
template <typename F>
cudaError_t prepare(F fn, uint32_t smem, bool* ready, std::mutex& mu) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 64 && ready[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && dev < 64) ready[dev] = true;
  return e;
}

template <typename F, typename... A>
cudaError_t launch_cluster(F fn, unsigned grid, unsigned threads, size_t smem, unsigned cluster, cudaStream_t s,
                           A... args) {
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(grid);
  lc.blockDim = dim3(threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 2;
  return cudaLaunchKernelEx(&lc, fn, args...);
}

// Rows of `blocks` 16-byte blocks as 16-bit elements (a stage's rows are 64 of them).
cudaError_t encode(CUtensorMap* m, const uint8_t* values, int64_t blocks, int64_t rows, int64_t mats, uint32_t box) {
  return tc_encode_map(m, values, NS_F16, blocks * 8, rows, mats, blocks * 8, rows * blocks * 8, 64, box);
}

cudaError_t run_few(const MxProduct& p, const MxScales& q, cudaStream_t s) {
  static bool ready[64] = {};
  static std::mutex mu;
  cudaError_t e = prepare(k_mx_few, kFewSmem, ready, mu);
  if (e != cudaSuccess) return e;
  FewArgs a{};
  a.rows = (int)p.rows; a.M = (int)p.out; a.K = q.blocks * kMxBlock;
  a.cols = (a.rows + 15) / 16 * 16;
  a.stage_bytes = kWeights + (uint32_t)a.cols * kRowBytes + kScaleA + kFewScaleB;
  a.stages = (int)(kFewRing / a.stage_bytes);
  if (a.stages > kFewStages) a.stages = kFewStages;
  a.type = p.dtype; a.act = p.act; a.D = p.y; a.bias = p.bias; a.residual = p.residual; a.r_m = p.r_stride;
  a.err = p.err;
  CUtensorMap mw, mx;
  e = encode(&mw, p.w_values, q.blocks, p.out, 1, 128);
  if (e == cudaSuccess) e = encode(&mx, p.x_values, q.blocks, p.rows, 1, (uint32_t)a.cols);
  if (e != cudaSuccess) return e;
  // shares of the sum: as many as one wave of two CTAs an SM takes, as in k_linear_few.cu
  const int tiles = (a.M + 127) / 128, pieces = (a.K + 2 * kStep - 1) / (2 * kStep), places = 2 * num_sms();
  int shares = places / tiles < kMaxShares ? places / tiles : kMaxShares;
  if (shares > pieces) shares = pieces;
  if (shares < 1) shares = 1;
  return launch_cluster(k_mx_few, (unsigned)(tiles * shares), kFewThreads, kFewSmem, (unsigned)shares, s, mw, mx, a, q);
}

cudaError_t run_tiles(const MxProduct& p, const MxScales& q, cudaStream_t s) {
  static bool ready[64] = {};
  static std::mutex mu;
  cudaError_t e = prepare(k_mx_tiles, kSmem, ready, mu);
  if (e != cudaSuccess) return e;
  TcProduct a{};
  a.mode = p.experts ? GROUP_ROWS : GROUP_NONE;
  a.experts = p.experts; a.offsets = p.offsets; a.splits = 1;
  a.rows = (int)p.rows; a.K = q.blocks * kMxBlock; a.M = (int)p.out;
  a.tiles_m = (a.M + BM - 1) / BM;
  a.type = p.dtype; a.act = p.act; a.D = p.y; a.bias = p.bias; a.residual = p.residual; a.r_m = p.r_stride;
  a.err = p.err;
  const int64_t pairs = num_sms() / 2;
  const int64_t ranges = p.experts ? (p.rows < p.experts ? p.rows : p.experts) : 1;
  const int64_t each = (p.rows + ranges - 1) / ranges;
  const auto items = [&](int tile) { return ranges * ((each + tile - 1) / tile) * a.tiles_m; };
  a.tile_rows = each <= 32 ? 64 : (each <= 64 ? 128 : 192);
  if (!p.experts) a.tile_rows = items(192) >= pairs ? 192 : (items(128) >= pairs ? 128 : 64);
  a.stages = stages_of(a.tile_rows);
  CUtensorMap mw;
  NMaps mx;
  e = encode(&mw, p.w_values, q.blocks, p.out, p.experts ? p.experts : 1, 128);
  for (int b = 0; b < kBoxes && e == cudaSuccess; ++b)
    e = encode(&mx.box[b], p.x_values, q.blocks, p.rows, 1, (uint32_t)box_rows(b));
  if (e != cudaSuccess) return e;
  int64_t most = (p.rows + a.tile_rows - 1) / a.tile_rows;
  if (p.experts) most = p.rows / a.tile_rows + ranges;  // at most
  most *= a.tiles_m;
  const unsigned grid = (unsigned)(2 * (most < 1 ? 1 : (most < pairs ? most : pairs)));
  return launch_cluster(k_mx_tiles, grid, kThreads, kSmem, 2, s, mw, mx, a, q);
}

}  // namespace

cudaError_t launch_mx_linear(const MxProduct& p, cudaStream_t s) {
  MxScales q{};
  q.blocks = (int)((p.in + kMxBlock - 1) / kMxBlock);
  q.w = p.w_scales; q.w_pitch = q.blocks; q.w_matrix = p.out * q.blocks;
  q.x = p.x_scales; q.x_pitch = p.x_pitch;
  return !p.experts && p.rows <= 64 ? run_few(p, q, s) : run_tiles(p, q, s);
}

}  // namespace muon
