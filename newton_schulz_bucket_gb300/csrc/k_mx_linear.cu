// A layer's product of microscaled 4-bit operands on the tensor cores: y =
// act(x W + b) + r with the weights held in 4 bits and the token rows rounded to 4
// bits before, fp32 sums.
//
// The block-scaled MMA (tcgen05.mma kind::mxf4) multiplies 64 steps of the sum at a
// time and takes the operands' scales from TMEM: for every 128 steps a 32-bit word a row
// (four scales), row r in lane r % 32, column r / 32, the same in all four quarters of
// the lanes.  The launch before (k_mx_quantize.cu) has put the scales of 128 rows x 128
// steps into blocks of 512 bytes in that order, so that they come by TMA with the
// operands, and tcgen05.cp spreads them over TMEM just before the MMAs that use them.
// Sets of scale columns are used in turn, each once the MMAs that read it are done.  (Put
// in order here, by warps that read them from memory and handed them to the leader, they
// cost a release and an acquire at cluster scope a stage: 1800 cycles a stage of 384 of
// MMAs.)
//
// Tiles are those of k_linear_tc.cu's rows form: a CTA pair computes 256 features x up
// to 192 tokens (two accumulators of 192 columns and 5 x 24 columns of scales fill
// TMEM), each CTA stages its 128 rows of weights and its half of the tokens, 256 steps a
// stage.  Waits, scale copies, MMAs and commits are issued by three warps: in one they
// took 800 cycles a stage, where the MMAs take 384.  [8192 x 8192] x [8192, 8192] 190 us with
// the rounding (5790 TFLOP/s): the tensor pipe is 82% busy and the clock at 1.58 GHz, under
// the power cap.
//
// Up to 64 rows of one matrix can take the form of k_linear_few.cu: 128 features a cluster of
// up to eight CTAs that share the sum.  Up to 16 of them need no launch before: the warps
// that wait for the sum round the rows and order the scales meanwhile.  Bound by latency: one
// token, 4096 -> 12288, 27 MB, takes 10 us (2.7 TB/s), 4096 -> 4096 6.2.
#include <cuda.h>

#include <mutex>

#include "linear_tiles.cuh"
#include "mx.cuh"

namespace muon {

namespace {

constexpr int kStep = 256;                    // steps of the sum in a stage: 128 bytes a row
constexpr uint32_t kRowBytes = 128;
constexpr uint32_t kWeights = 128 * kRowBytes;
constexpr uint32_t kScaleBlock = 512;         // scales of 128 rows x 128 steps
constexpr uint32_t kScaleA = 2 * kScaleBlock;

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
// A block of scales, 32 lanes x 16 bytes, to four TMEM columns in all four quarters.
template <bool kPair>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (kPair)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Arrives on the leader's barrier alone when what this thread issued has completed.
__device__ __forceinline__ void commit_leader(uint32_t mbar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(mbar) : "memory");
}
// Descriptor of such a block: no swizzle, groups of eight 16-byte rows 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

// A stage's scales to TMEM, the weights' at ta and the tokens' behind, for `steps` steps of
// the sum (256 at most).  NB: blocks of scales of the tile's tokens.
template <bool kPair, int NB>
__device__ __forceinline__ void stage_scales(uint32_t ta, uint64_t dsa, uint64_t dsb, int steps) {
  constexpr uint64_t kBlock = kScaleBlock >> 4;
  const uint32_t tb = ta + 8;
  copy_scales<kPair>(ta, dsa);
  copy_scales<kPair>(tb, dsb);
  if (NB == 2) copy_scales<kPair>(tb + 4, dsb + kBlock);
  if (steps > 128) {
    copy_scales<kPair>(ta + 4, dsa + kBlock);
    copy_scales<kPair>(tb + 4 * NB, dsb + NB * kBlock);
    if (NB == 2) copy_scales<kPair>(tb + 12, dsb + 3 * kBlock);
  }
}
// Its MMAs, 64 steps each; behind the sum's end there are only zeros.
template <bool kPair, int NB>
__device__ __forceinline__ void stage_mmas(uint32_t d, uint32_t ta, uint64_t da, uint64_t db, uint32_t first,
                                           uint32_t second, int steps, uint32_t add) {
  const uint32_t tb = ta + 8;
  umma_mx<kPair>(d, da, db, first, ta, tb, add);
  if (steps > 192) {
    umma_mx<kPair>(d, da + 2, db + 2, second, ta, tb, 1);
    umma_mx<kPair>(d, da + 4, db + 4, first, ta + 4, tb + 4 * NB, 1);
    umma_mx<kPair>(d, da + 6, db + 6, second, ta + 4, tb + 4 * NB, 1);
  } else {
    if (steps > 64) umma_mx<kPair>(d, da + 2, db + 2, second, ta, tb, 1);
    if (steps > 128) umma_mx<kPair>(d, da + 4, db + 4, first, ta + 4, tb + 4 * NB, 1);
  }
}

// ---- tiles in CTA pairs ----

constexpr int kThreads = 32 * (4 + kEpiWarps);  // producer, MMA issuer, epilogue, two that copy scales
constexpr int kMaxStages = 9;
constexpr uint32_t kRing = 222208;             // 7 stages of 192 tokens, 8 of 128, 9 of 64
__host__ __device__ constexpr uint32_t stage_bytes_of(int tile_rows) {
  return kWeights + (uint32_t)(tile_rows / 2) * kRowBytes + kScaleA + (uint32_t)mx_token_blocks(tile_rows) * kScaleA;
}
__host__ __device__ constexpr int stages_of(int tile_rows) { return (int)(kRing / stage_bytes_of(tile_rows)); }
static_assert(stages_of(192) == 7 && stages_of(128) == 8 && stages_of(64) == kMaxStages, "ring depths");
static_assert(2 * 192 + 5 * 24 <= 512 && 2 * 128 + kMaxStages * 16 <= 512, "accumulators and scales in TMEM");
static_assert(stage_bytes_of(192) % 1024 == 0 && stage_bytes_of(128) % 1024 == 0 && stage_bytes_of(64) % 1024 == 0,
              "stages start where the swizzle does");
constexpr uint32_t kSmem = kRing + 512 + 1024;
static_assert((3 * kMaxStages + 5) * 8 + 8 <= 512 && kSmem <= 227 * 1024, "shared memory layout");

struct ScaleMaps {
  CUtensorMap w, x;            // [block][128 steps][512 or 1024 bytes]
};

// NB: blocks of scales of a tile's tokens (2 for tiles of more than 128).
template <int NB>
__global__ void __launch_bounds__(kThreads, 1)
    k_mx_tiles(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ NMaps mapsX,
               const __grid_constant__ ScaleMaps scales, const __grid_constant__ TcProduct p) {
  const int S = p.stages;
  const uint32_t stage_bytes = stage_bytes_of(p.tile_rows);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kRing);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * kMaxStages + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  const uint32_t bar0 = saddr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto tfull = [&](int a) { return bar0 + 8u * (2 * kMaxStages + a); };
  auto tempty = [&](int a) { return bar0 + 8u * (2 * kMaxStages + 2 + a); };
  const uint32_t done = bar0 + 8u * (2 * kMaxStages + 4);
  auto ready = [&](int s) { return bar0 + 8u * (2 * kMaxStages + 5 + s); };
  const uint32_t acc_cols = (uint32_t)p.tile_rows;
  constexpr int kScaleCols = 8 + 8 * NB, kSets = NB == 2 ? 5 : kMaxStages;  // sets of scale columns
  // the scales' place in a stage
  const uint32_t sa_at = kWeights + (uint32_t)(p.tile_rows / 2) * kRowBytes, sb_at = sa_at + kScaleA;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(full(s), 1); mbar_init(ready(s), 1); mbar_init(empty(s), 1); }
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
  // The launch before (k_mx_prepare) lets this one start only once all that ran before
  // it is done, so that offsets and weights may be read here; what it writes itself, and
  // what y takes the place of, waits.
  Walk<0> walk(p);
  Item it;
  bool more = walk.next(p, it);
  if (warp != 0) grid_wait();

  if (warp == 0) {  // ---- TMA producer (both CTAs) ----
    const uint32_t ring = saddr(smem), full_leader = map_to(full(0), 0);
    int s = 0;
    uint32_t ph = 1;
    bool ok = true;
    const int ahead = min(S, (p.K + kStep - 1) / kStep);  // stages of the first tile whose weights come early
    if (more && elect_lane()) {
      for (int i = 0; i < ahead; ++i)
        tma_load_3d_pair(ring + i * stage_bytes, &mapW, full_leader + 8u * i, i * (kStep / 4), it.m0 + (int)rank * 128,
                         it.e);
    }
    __syncwarp();
    grid_wait();
    int early = ahead;
    for (; ok && more; more = walk.next(p, it)) {
      const int wrow = it.m0 + (int)rank * 128, e = it.e;
      const int half = mma_cols(it) / 2, xrow = it.n0 + (int)rank * half;
      int box = 0;
      while (box_rows(box) < half) ++box;
      const CUtensorMap* mapX = &mapsX.box[box];
      const uint32_t bytes = kWeights + (uint32_t)box_rows(box) * kRowBytes + kScaleA + NB * kScaleA;
      const int wblock = e * p.tiles_n + wrow / 128;  // (tiles_n: blocks of 128 features)
      const int xblock = mx_token_slot(walk.lo, it.e, p.tile_rows) + it.tile;
      for (int k = 0; k < p.K; k += kStep) {
        if (!(ok = mbar_wait(empty(s), ph, abort_flag, p.err, 512))) break;
        if (elect_lane()) {
          const uint32_t sw = ring + s * stage_bytes, bar = full_leader + 8u * s;
          if (rank == 0) mbar_expect_tx(full(s), 2 * bytes);
          if (early == 0) tma_load_3d_pair(sw, &mapW, bar, k / 4, wrow, e);
          tma_load_3d_pair(sw + kWeights, mapX, bar, k / 4, xrow, 0);
          tma_load_3d_pair(sw + sa_at, &scales.w, bar, 0, k / 128, wblock);
          tma_load_3d_pair(sw + sb_at, &scales.x, bar, 0, k / 128, xblock);
        }
        __syncwarp();
        if (early) --early;
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
      const uint32_t apart = stage_bytes >> 4;
      const int whole = p.K / kStep, rest = p.K % kStep;
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 1, at = 0, ta = 2 * acc_cols;  // (all of TMEM is this CTA's: it starts at 0)
      const uint32_t ta_end = ta + kSets * kScaleCols;
      bool ok = true;
      const auto next_stage = [&] {
        at += apart;
        ta += kScaleCols;
        if (ta == ta_end) ta = 2 * acc_cols;
        if (++s == S) { s = 0; at = 0; ph ^= 1; }
      };
      for (; more; more = walk.next(p, it)) {
        if (!(ok = mbar_wait(tempty(acc), aph, abort_flag, p.err, 1024))) break;
        tc_fence_after();
        const uint32_t d_tmem = (uint32_t)acc * acc_cols;
        const int cols = mma_cols(it);
        const uint32_t first = mx_desc(BM, cols, 0), second = mx_desc(BM, cols, 1);
        uint32_t add = 0;
        for (int i = 0; i < whole; ++i) {
          if (!(ok = mbar_wait(ready(s), ph, abort_flag, p.err, 2048))) break;
          tc_fence_after();
          if (elect_lane()) {
            stage_mmas<true, NB>(d_tmem, ta, da + at, db + at, first, second, kStep, add);
            umma_commit_pair(empty(s), 3);  // frees the stage in both CTAs once these MMAs retire
          }
          __syncwarp();
          add = 1;
          next_stage();
        }
        if (ok && rest) {
          if (!(ok = mbar_wait(ready(s), ph, abort_flag, p.err, 2048))) break;
          tc_fence_after();
          if (elect_lane()) {
            stage_mmas<true, NB>(d_tmem, ta, da + at, db + at, first, second, rest, add);
            umma_commit_pair(empty(s), 3);
          }
          __syncwarp();
          next_stage();
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
  } else if (warp >= 2 + kEpiWarps) {
    if (rank == 0) {  // ---- scales from shared memory to TMEM, of both CTAs (leader only) ----
      // Two warps, one for the even stages and one for the odd: one alone needs 540 cycles a
      // stage for its waits and copies, the MMAs 384.  (Not in turns: a barrier's phases
      // are told apart by their parity, so that whoever waits on a stage has to wait for
      // each of its phases.)
      const uint64_t dsa = scale_desc(saddr(smem) + sa_at), dsb = scale_desc(saddr(smem) + sb_at);
      const uint32_t apart = stage_bytes >> 4;
      int s = 0, used = 0, old = 0;  // sets in use; the stage whose MMAs read the next set before
      const int which = warp - 2 - kEpiWarps;
      uint32_t ph = 0, oph = 0, at = 0, ta = 2 * acc_cols;
      const uint32_t ta_end = ta + kSets * kScaleCols;
      bool ok = true;
      for (; ok && more; more = walk.next(p, it)) {
        for (int k = 0; k < p.K; k += kStep) {
          if ((s & 1) == which) {
            // (as many sets as stages: the stage's own wait will do)
            if (NB == 2 && used == kSets && !(ok = mbar_wait(empty(old), oph, abort_flag, p.err, 4096))) break;
            if (!(ok = mbar_wait(full(s), ph, abort_flag, p.err, 8192))) break;
            tc_fence_after();
            if (elect_lane()) {
              stage_scales<true, NB>(ta, dsa + at, dsb + at, p.K - k);
              commit_leader(ready(s));
            }
            __syncwarp();
          }
          if (used < kSets) ++used;
          else if (++old == S) { old = 0; oph ^= 1; }
          at += apart;
          ta += kScaleCols;
          if (ta == ta_end) ta = 2 * acc_cols;
          if (++s == S) { s = 0; at = 0; ph ^= 1; }
        }
      }
      // (the last copies are done when the MMAs that wait for them are; after an abort they
      // are waited for here)
      if (!ok) {
        const long long t0 = clock64();
        while (clock64() - t0 < (1ll << 21)) {}
      }
    }
  } else {  // ---- epilogue ----
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

constexpr int kFewThreads = 192;  // producer, MMA issuer, four epilogue warps
constexpr uint32_t kFewRing = 112640;  // 5 stages of 128 + 16 rows, 4 of 128 + 64; two CTAs an SM
constexpr uint32_t kFewSmem = kFewRing + 256 + 1024;
constexpr int kFewStages = 5;
constexpr int kFewTmem = 256;     // 64 of sums, 16 for each stage's scales
constexpr int kMaxShares = 8;
static_assert(2 * (kFewSmem + 1024) <= 228 * 1024, "two CTAs an SM");

struct FewArgs {
  const void* x;            // with kOwn: the rows, and the weights' scales as they are held
  int64_t x_stride;
  const uint8_t* w_scales;
  int in, x_vec;
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

// What one of the four warps puts into a stage itself (kOwn): the scales of 32 weight
// rows, and of the 16 token rows every fourth, 256 steps each, eight a lane.
template <typename T>
struct OwnStage {
  uint2 w;
  Eight<T> x[4];
  __device__ __forceinline__ void fetch(const FewArgs& p, int m0, int warp, int lane, int k) {
    const int kb = p.K / kMxBlock, at = k / kMxBlock, row = m0 + 32 * warp + lane;
    w = make_uint2(0, 0);
    if (row < p.M) {
      const uint8_t* q = p.w_scales + (int64_t)row * kb + at;
      if (at + 8 <= kb && (reinterpret_cast<uintptr_t>(q) & 7) == 0) {
        w = *reinterpret_cast<const uint2*>(q);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (at + i < kb) (i < 4 ? w.x : w.y) |= (uint32_t)q[i] << (8 * (i & 3));
      }
    }
    const int col = k + 8 * lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = warp + 4 * i;
      x[i].zero();
      if (t >= p.rows || col >= p.in) continue;
      const T* src = static_cast<const T*>(p.x) + t * p.x_stride + col;
      if (p.x_vec && col + 8 <= p.in) x[i].fetch(src);
      else x[i].fetch_some(src, p.in - col);
    }
  }
  __device__ __forceinline__ void put(const FewArgs& p, uint8_t* rows, uint8_t* sa, uint8_t* sb, int warp, int lane) const {
    *reinterpret_cast<uint32_t*>(sa + lane * 16 + warp * 4) = w.x;
    *reinterpret_cast<uint32_t*>(sa + kScaleBlock + lane * 16 + warp * 4) = w.y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = warp + 4 * i, block = lane >> 2;
      if (t >= p.rows) break;  // (the same for the warp; columns of no token take what is there)
      uint32_t top = x[i].top();
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t s = Eight<T>::scale(top);
      // (the copies' 128-byte swizzle)
      *reinterpret_cast<uint32_t*>(rows + t * 128 + ((block ^ (t & 7)) << 4) + (lane & 3) * 4) = x[i].packed(mx_inverse(s));
      if ((lane & 3) == 0) sb[(block >> 2) * kScaleBlock + t * 16 + (block & 3)] = (uint8_t)s;
    }
  }
};

// kOwn (up to 16 rows): no launch before this one has rounded the rows or ordered the
// scales.
template <bool kOwn, typename T>
__global__ void __launch_bounds__(kFewThreads, 2)
    k_mx_few(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapX,
             const __grid_constant__ ScaleMaps scales, const __grid_constant__ FewArgs p) {
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
    for (int s = 0; s < p.stages; ++s) { mbar_init(full(s), kOwn ? 5 : 1); mbar_init(empty(s), 1); }
    mbar_init(all, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mapW) : "memory");
    if (!kOwn) asm volatile("prefetch.tensormap [%0];" ::"l"(&mapX) : "memory");
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
  if (kOwn || warp != 0) grid_wait();  // (the producer's weights come early, as in k_mx_tiles)

  const int blocks = (p.K + kStep - 1) / kStep;  // blocks * shares stays below 2^31
  const int k0 = blocks * rank / shares * kStep;
  const int k1 = rank + 1 == shares ? p.K : blocks * (rank + 1) / shares * kStep;
  if (warp == 0) {  // ---- TMA producer ----
    const uint32_t ring = saddr(smem);
    int s = 0;
    uint32_t ph = 1;
    bool ok = true;
    int early = kOwn ? 0 : min(p.stages, (k1 - k0 + kStep - 1) / kStep);
    if (!kOwn && elect_lane())
      for (int i = 0; i < early; ++i)
        tma_load_3d(ring + i * p.stage_bytes, &mapW, full(i), (k0 + i * kStep) / 4, m0, 0);
    __syncwarp();
    if (!kOwn) grid_wait();
    for (int k = k0; k < k1; k += kStep) {
      if (!(ok = mbar_wait(empty(s), ph, abort_flag, p.err, 4096))) break;
      if (elect_lane()) {
        const uint32_t sw = ring + s * p.stage_bytes;
        mbar_expect_tx(full(s), kOwn ? kWeights : p.stage_bytes);
        if (early == 0) tma_load_3d(sw, &mapW, full(s), k / 4, m0, 0);
        if constexpr (!kOwn) {
          tma_load_3d(sw + kWeights, &mapX, full(s), k / 4, 0, 0);
          tma_load_3d(sw + sa_at, &scales.w, full(s), 0, k / 128, m0 / 128);
          tma_load_3d(sw + sb_at, &scales.x, full(s), 0, k / 128, 0);
        }
      }
      __syncwarp();
      if (early) --early;
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
    uint32_t ph = 0;
    for (int k = k0; k < k1; k += kStep) {
      if (!mbar_wait(full(s), ph, abort_flag, p.err, 8192)) break;
      tc_fence_after();
      const uint64_t at = s * (p.stage_bytes >> 4);
      const uint32_t ta = tmem + 64 + (uint32_t)(s * 16);
      if (elect_lane()) {
        stage_scales<false, 1>(ta, dsa + at, dsb + at, k1 - k);
        stage_mmas<false, 1>(tmem, ta, da + at, db + at, first, second, k1 - k, k > k0 ? 1 : 0);
        umma_commit(empty(s));
      }
      __syncwarp();
      if (++s == p.stages) { s = 0; ph ^= 1; }
    }
    if (elect_lane()) umma_commit(all);
    __syncwarp();
    volatile int keep_waiting = 0;
    mbar_wait(all, 0, &keep_waiting, p.err, 256);  // every MMA is done before the ring is reused
  } else if constexpr (kOwn) {  // ---- rows and scales ----
    constexpr int kSets = 2;  // one is put into its stage while the other's loads are under way
    OwnStage<T> set[kSets];
    int s = 0;
    uint32_t ph = 1;
    bool ok = true;
#pragma unroll
    for (int i = 0; i < kSets; ++i)
      if (k0 + i * kStep < k1) set[i].fetch(p, m0, warp - 2, lane, k0 + i * kStep);
    for (int k = k0; ok && k < k1; k += kSets * kStep) {
#pragma unroll
      for (int i = 0; i < kSets; ++i) {
        const int at = k + i * kStep;
        if (!ok || at >= k1) continue;
        if (!(ok = mbar_wait(empty(s), ph, abort_flag, p.err, 16384))) continue;
        uint8_t* stage = smem + s * p.stage_bytes;
        set[i].put(p, stage + kWeights, stage + sa_at, stage + sb_at, warp - 2, lane);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(full(s));
        if (++s == p.stages) { s = 0; ph ^= 1; }
        if (at + kSets * kStep < k1) set[i].fetch(p, m0, warp - 2, lane, at + kSets * kStep);
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
  // four features a thread, every share's sums in flight together
  for (int i = (int)threadIdx.x + rank * kFewThreads; i < p.rows * 32; i += kFewThreads * shares) {
    const int64_t t = i >> 5, f = m0 + (i & 31) * 4;
    if (f >= p.M) continue;
    float4 v[kMaxShares];
#pragma unroll
    for (int r = 0; r < kMaxShares; ++r)
      if (r < shares) v[r] = ld_shared_of<float4>(saddr(part + 4 * i), (uint32_t)r);
    float z[4] = {};
#pragma unroll
    for (int r = 0; r < kMaxShares; ++r)
      if (r < shares) { z[0] += v[r].x; z[1] += v[r].y; z[2] += v[r].z; z[3] += v[r].w; }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (f + c >= p.M) break;
      if (p.bias) z[c] += ld_el(p.bias, f + c, p.type);
      z[c] = p.type == DT_F32 ? activate<false>(z[c], p.act) : activate<true>(z[c], p.act);
      if (p.residual) z[c] += ld_el(p.residual, t * p.r_m + f + c, p.type);
      st_el(p.D, t * p.M + f + c, z[c], p.type);
    }
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

// Rows of `blocks` 16-byte blocks as 16-bit elements (a stage's rows are 64 of them).
cudaError_t encode(CUtensorMap* m, const uint8_t* values, int64_t blocks, int64_t rows, int64_t mats, uint32_t box) {
  return tc_encode_map(m, values, NS_F16, blocks * 8, rows, mats, blocks * 8, rows * blocks * 8, 64, box);
}
// Ordered scales as 32-bit words: two times 128 steps a stage.
cudaError_t encode_scales(ScaleMaps* m, const MxProduct& p, int64_t w_blocks, int64_t x_slots, int nb) {
  const int64_t parts = mx_parts(p.in);
  cudaError_t e = tc_encode_words(&m->w, p.w_scales, 128, parts, w_blocks, 2);
  if (e == cudaSuccess) e = tc_encode_words(&m->x, p.x_scales, 128 * nb, parts, x_slots, 2);
  return e;
}

template <bool kOwn, typename T>
cudaError_t run_few(const MxProduct& p, cudaStream_t s) {
  static bool ready[64] = {};
  static std::mutex mu;
  auto fn = k_mx_few<kOwn, T>;
  cudaError_t e = prepare(fn, kFewSmem, ready, mu);
  if (e != cudaSuccess) return e;
  const int64_t kb = mx_blocks_of(p.in);
  FewArgs a{};
  a.rows = (int)p.rows; a.M = (int)p.out; a.K = (int)kb * kMxBlock;
  a.cols = (a.rows + 15) / 16 * 16;
  a.stage_bytes = kWeights + (uint32_t)a.cols * kRowBytes + 2 * kScaleA;
  a.stages = (int)(kFewRing / a.stage_bytes);
  if (a.stages > kFewStages) a.stages = kFewStages;
  a.type = p.dtype; a.act = p.act; a.D = p.y; a.bias = p.bias; a.residual = p.residual; a.r_m = p.r_stride;
  a.err = p.err;
  const int tiles = (a.M + 127) / 128, blocks = (a.K + kStep - 1) / kStep, places = 2 * num_sms();
  CUtensorMap mw, mx{};
  ScaleMaps ms{};
  e = encode(&mw, p.w_values, kb, p.out, 1, 128);
  if (kOwn) {
    a.x = p.x;
    a.x_stride = p.x_stride;
    a.w_scales = p.w_scales;
    a.in = (int)p.in;
    a.x_vec = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && (p.rows == 1 || p.x_stride * (int64_t)sizeof(T) % 16 == 0);
  } else {
    if (e == cudaSuccess) e = encode(&mx, p.x_values, kb, p.rows, 1, (uint32_t)a.cols);
    if (e == cudaSuccess) e = encode_scales(&ms, p, tiles, 1, 1);
  }
  if (e != cudaSuccess) return e;
  // shares of the sum: as many as one wave of two CTAs an SM takes, as in k_linear_few.cu
  int shares = places / tiles < kMaxShares ? places / tiles : kMaxShares;
  if (shares > blocks) shares = blocks;
  if (shares < 1) shares = 1;
  return launch_early_cluster(fn, (unsigned)(tiles * shares), kFewThreads, kFewSmem, (unsigned)shares, s, mw, mx, ms, a);
}

template <int NB>
cudaError_t run_tiles(const MxProduct& p, cudaStream_t s) {
  static bool ready[64] = {};
  static std::mutex mu;
  cudaError_t e = prepare(k_mx_tiles<NB>, kSmem, ready, mu);
  if (e != cudaSuccess) return e;
  const int64_t kb = mx_blocks_of(p.in), mats = p.experts ? p.experts : 1;
  TcProduct a{};
  a.mode = p.experts ? GROUP_ROWS : GROUP_NONE;
  a.experts = p.experts; a.offsets = p.offsets; a.splits = 1;
  a.rows = (int)p.rows; a.K = (int)kb * kMxBlock; a.M = (int)p.out;
  a.tiles_m = (a.M + BM - 1) / BM;
  a.tiles_n = (a.M + 127) / 128;
  a.type = p.dtype; a.act = p.act; a.D = p.y; a.bias = p.bias; a.residual = p.residual; a.r_m = p.r_stride;
  a.err = p.err;
  a.tile_rows = p.tile_rows;
  a.stages = stages_of(a.tile_rows);
  CUtensorMap mw;
  NMaps mx;
  ScaleMaps ms;
  e = encode(&mw, p.w_values, kb, p.out, mats, 128);
  for (int b = 0; b < kBoxes && e == cudaSuccess; ++b)
    e = encode(&mx.box[b], p.x_values, kb, p.rows, 1, (uint32_t)box_rows(b));
  if (e == cudaSuccess) e = encode_scales(&ms, p, mats * a.tiles_n, mx_token_slots(p.rows, p.experts, a.tile_rows), NB);
  if (e != cudaSuccess) return e;
  const int64_t pairs = num_sms() / 2;
  int64_t most = (p.rows + a.tile_rows - 1) / a.tile_rows;
  if (p.experts) most = p.rows / a.tile_rows + (p.rows < mats ? p.rows : mats);  // at most
  most *= a.tiles_m;
  const unsigned grid = (unsigned)(2 * (most < 1 ? 1 : (most < pairs ? most : pairs)));
  return launch_early_cluster(k_mx_tiles<NB>, grid, kThreads, kSmem, 2, s, mw, mx, ms, a);
}

}  // namespace

// Most token rows of a tile: as many as fill the tensor cores' columns, fewer where that
// leaves pairs without a tile (512 rows, 4096 -> 16384: 25.3 us with 192, 26.9 with 128;
// 4096 -> 4096: 14.6 and 14.3; with 64 35 and 17).  An expert often has more rows than the
// average, which is all the host knows: not where that would need another tile (64 experts
// [7168, 2048] of 32 rows 113 us with 64, 115 with 192; of 64 rows 125 with 128, 131 with 64;
// of 128 rows 147 with 192, 152 with 128).
int mx_tile_rows(int64_t rows, int32_t experts, int64_t out) {
  if (experts) {
    const int64_t ranges = rows < experts ? rows : experts, each = ranges ? (rows + ranges - 1) / ranges : 0;
    return each <= 32 ? 64 : (each <= 64 ? 128 : 192);
  }
  if (rows <= 64) return 64;
  return (out + BM - 1) / BM * ((rows + 191) / 192) >= num_sms() / 2 ? 192 : 128;
}

// Few rows of one matrix, where four CTAs or more can share a sum (32 rows, 4096 -> 4096: 9.4
// us, 10.9 in tiles; 64 rows, 16384 -> 4096: 16.3 and 20.8; with three shares 64 rows, 4096
// -> 12288 16.8 and 13.2).  (Rows that a product rounds itself always.)
static bool few_rows(const MxProduct& p) {
  return !p.experts && p.rows <= 64 && 4 * ((p.out + 127) / 128) <= 2 * num_sms();
}

cudaError_t launch_mx_linear(const MxProduct& p, cudaStream_t s) {
  if (mx_own_rows(p.rows, p.experts)) {
    switch (p.dtype) {
      case DT_F16: return run_few<true, __half>(p, s);
      case DT_BF16: return run_few<true, __nv_bfloat16>(p, s);
      default: return run_few<true, float>(p, s);
    }
  }
  if (few_rows(p)) return run_few<false, float>(p, s);
  return mx_token_blocks(p.tile_rows) == 2 ? run_tiles<2>(p, s) : run_tiles<1>(p, s);
}

}  // namespace muon
