// A layer's product for few token rows (up to 64): the time it takes to read the
// weights once.
//
// A cluster of up to eight CTAs shares one tile of 128 features: each takes a
// share of the sum, streams its weights (the M operand of tcgen05.mma, one CTA
// each, 16 to 64 columns of tokens) through a ring of TMA tiles, and the partial
// sums are added through distributed shared memory in the order of the ranks.
// So every SM has weights in flight, and nothing is written but the result (one
// token, [4096, 12288] bf16: 18.7 us, 5.4 TB/s; [1024, 1024]: 4.6 us): no
// scratch, no second launch.  Two CTAs fit on an SM.  fp32 tensors take the six partial
// products of three bf16 planes, as the tile kernels do.
#include <cuda.h>

#include <mutex>

#include "internal.h"
#include "linear.cuh"

namespace muon {

namespace {

constexpr int kThreads = 192;  // producer, MMA issuer, four epilogue warps
constexpr uint32_t kW = 128 * BK * 2;
constexpr uint32_t kRingBytes = 110592;  // 6 stages of 128 + 16 rows; two CTAs an SM
constexpr uint32_t kSmemBytes = kRingBytes + 256 + 1024;
constexpr int kMaxStages = 6;
constexpr int kMaxShares = 8;

struct FewArgs {
  int rows, M, K;           // token rows, features, length of the sum
  int cols;                 // columns of an MMA: rows in steps of 16
  int stages;
  uint32_t stage_bytes;
  int type, act, first;     // DType, Act, first partial product
  void* D;
  const void* bias;
  const void* residual;
  int64_t r_m;
  void* preact;
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

// ACROSS: weights stored across the sum ([in][out] for y).
template <bool ACROSS>
__global__ void __launch_bounds__(kThreads, 2)
    k_linear_few(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapX,
                 const __grid_constant__ FewArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kRingBytes);  // full, empty, all
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t bar0 = saddr(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  const uint32_t all = bar0 + 8u * (2 * kMaxStages);
  const int shares = (int)cluster_ctas(), rank = (int)cta_rank();
  const int m0 = (int)(blockIdx.x / shares) * 128;
  const uint32_t tmem_cols = p.cols > 32 ? 64 : 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) { mbar_init(full(s), 1); mbar_init(empty(s), 1); }
    mbar_init(all, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mapW) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mapX) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)),
                 "r"(tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_launch_next();
  grid_wait();

  const int blocks = (p.K + BK - 1) / BK;  // blocks * shares stays below 2^31
  const int k0 = blocks * rank / shares * BK;
  const int k1 = rank + 1 == shares ? p.K : blocks * (rank + 1) / shares * BK;
  if (warp == 0) {  // ---- TMA producer ----
    const uint32_t ring = saddr(smem);
    int s = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int i = p.first; ok && i < kProducts; ++i) {
      const int wp = plane_m(i), xp = plane_n(i);
      for (int k = k0; k < k1; k += BK) {
        if (!(ok = mbar_wait(empty(s), ph, abort_flag, p.err, 64))) break;
        if (elect_lane()) {
          const uint32_t sw = ring + s * p.stage_bytes;
          mbar_expect_tx(full(s), p.stage_bytes);
          if (ACROSS) {
            tma_load_3d(sw, &mapW, full(s), m0, k, wp);
            tma_load_3d(sw + 64 * BK * 2, &mapW, full(s), m0 + 64, k, wp);
          } else {
            tma_load_3d(sw, &mapW, full(s), k, m0, wp);
          }
          tma_load_3d(sw + kW, &mapX, full(s), k, 0, xp);
        }
        __syncwarp();
        if (++s == p.stages) { s = 0; ph ^= 1; }
      }
    }
    if (!ok) {  // gave up: let the copies in flight land before the block leaves
      const long long t0 = clock64();
      while (clock64() - t0 < (1ll << 21)) {}
    }
  } else if (warp == 1) {  // ---- MMA issuer ----
    const uint64_t da = ACROSS ? smem_desc(saddr(smem), 64 * BK * 2, 1024) : smem_desc(saddr(smem), 16, 1024);
    const uint64_t db = smem_desc(saddr(smem) + kW, 16, 1024);
    constexpr uint64_t kStepA = ACROSS ? 2048 / 16 : 32 / 16, kStepB = 32 / 16;
    const uint32_t idesc = instr_desc(p.type == DT_F16 ? 0u : 1u, 128, p.cols, false, ACROSS);
    int s = 0;
    uint32_t ph = 0, add = 0;
    bool ok = true;
    for (int i = p.first; ok && i < kProducts; ++i) {
      for (int k = k0; k < k1; k += BK) {
        if (!(ok = mbar_wait(full(s), ph, abort_flag, p.err, 128))) break;
        tc_fence_after();
        const uint64_t a = da + s * (p.stage_bytes >> 4), b = db + s * (p.stage_bytes >> 4);
        if (elect_lane()) {
          umma(tmem, a, b, idesc, add);
          umma(tmem, a + kStepA, b + kStepB, idesc, 1);
          umma(tmem, a + 2 * kStepA, b + 2 * kStepB, idesc, 1);
          umma(tmem, a + 3 * kStepA, b + 3 * kStepB, idesc, 1);
          umma_commit(empty(s));
        }
        __syncwarp();
        add = 1;
        if (++s == p.stages) { s = 0; ph ^= 1; }
      }
    }
    if (elect_lane()) umma_commit(all);
    __syncwarp();
    volatile int keep_waiting = 0;
    mbar_wait(all, 0, &keep_waiting, p.err, 256);  // every MMA is done before the ring is reused
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
  for (int i = (int)threadIdx.x + rank * kThreads; i < p.rows * 128; i += kThreads * shares) {
    const int64_t t = i >> 7, f = m0 + (i & 127);
    if (f >= p.M) continue;
    float z = 0.f;
    for (int r = 0; r < shares; ++r) z += ld_shared_of(saddr(part + i), (uint32_t)r);
    if (p.bias) z += ld_el(p.bias, f, p.type);
    if (p.preact) st_el(p.preact, t * p.M + f, z, p.type);
    z = p.type == DT_F32 ? activate<false>(z, p.act) : activate<true>(z, p.act);
    if (p.residual) z += ld_el(p.residual, t * p.r_m + f, p.type);
    st_el(p.D, t * p.M + f, z, p.type);
  }
  cluster_barrier();  // no CTA leaves while another reads its sums
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(tmem_cols) : "memory");
  }
}

template <bool ACROSS>
cudaError_t launch(const CUtensorMap& mw, const CUtensorMap& mx, const FewArgs& q, int tiles, int shares,
                   cudaStream_t s) {
  auto fn = k_linear_few<ACROSS>;
  static bool ready[64] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !ready[dev]) {
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
      if (e != cudaSuccess) return e;
      if (dev < 64) ready[dev] = true;
    }
  }
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3((unsigned)(tiles * shares));
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = kSmemBytes;
  lc.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)shares;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 2;
  return cudaLaunchKernelEx(&lc, fn, mw, mx, q);
}

}  // namespace

bool linear_few_fits(const Product& p) {
  return p.mode == GROUP_NONE && p.a_k == 1 && p.M <= 64 && (p.K + BK - 1) / BK * kMaxShares < (1ll << 31) / BK &&
         (p.N + 127) / 128 * kMaxShares < (1ll << 31);
}

cudaError_t launch_linear_few(const Product& p, cudaStream_t s) {
  FewArgs q{};
  q.rows = (int)p.M; q.M = (int)p.N; q.K = (int)p.K;
  q.cols = (q.rows + 15) / 16 * 16;
  q.stage_bytes = kW + (uint32_t)q.cols * BK * 2;
  q.stages = (int)(kRingBytes / q.stage_bytes);
  q.type = p.dtype; q.act = p.act;
  q.first = p.dtype == DT_F32 ? 0 : kProducts - 1;
  q.D = p.D; q.bias = p.bias; q.residual = p.residual; q.r_m = p.r_m; q.preact = p.preact; q.err = p.err;
  const int type = p.dtype == DT_F16 ? NS_F16 : NS_BF16, planes = p.dtype == DT_F32 ? 3 : 1;
  const bool across = p.b_k != 1;
  CUtensorMap mw, mx;
  cudaError_t e = across ? tc_encode_map(&mw, p.B, type, p.N, p.K, planes, p.b_k, p.K * p.b_k, 64, 64)
                         : tc_encode_map(&mw, p.B, type, p.K, p.N, planes, p.b_n, p.N * p.b_n, 64, 128);
  if (e == cudaSuccess)
    e = tc_encode_map(&mx, p.A, type, p.K, p.M, planes, p.a_m, p.M * p.a_m, 64, (uint32_t)q.cols);
  if (e != cudaSuccess) return e;
  // shares of the sum: as many as one wave of two CTAs an SM takes, of at least
  // two blocks each (equal shares of a stream that HBM bounds end together; a
  // second wave would start when the first one's copies have drained)
  const int tiles = (q.M + 127) / 128, blocks = (q.K + BK - 1) / BK, places = 2 * num_sms();
  int shares = places / tiles < kMaxShares ? places / tiles : kMaxShares;
  if (shares > blocks / 2) shares = blocks / 2;
  if (shares < 1) shares = 1;
  return across ? launch<true>(mw, mx, q, tiles, shares, s) : launch<false>(mw, mx, q, tiles, shares, s);
}

}  // namespace muon
