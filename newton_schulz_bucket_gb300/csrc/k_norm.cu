// Layer norm of rows, y = (x - mean) rstd w + b with rstd = (var + eps)^-1/2, and its
// gradient: with xh = (x - mean) rstd and g = dy w,
//   dx = rstd (g - mean(g) - xh mean(g xh)) + r,   dw = sum over rows of dy xh,   db = sum of dy.
//
// Rows of up to 16384 elements cross HBM once.  Up to 512 of them belong to 1 to 32 lanes
// of a warp, more to a block.  A row stays in the registers of its threads (16 or 32
// elements each) between the sums over it and its result; where those hold the sums over
// rows already (back, beyond 8192 elements) it stays in shared memory and is read twice from
// there.  The next rows are on their way meanwhile: several, by bulk copies into a ring in
// shared memory, where a row belongs to a block; else the next one, into registers.  Rows
// beyond 16384 elements are read again for each sum (from L2, where they are not too long).
// The variance is the sum of squares about the mean, not a difference of two large sums.
// Blocks stay for many rows, so that the weights are read once a block and the sums over
// rows (dw, db) grow in registers too; each part of rows leaves one partial sum, and a second
// kernel adds the parts in a fixed order.  No atomics: the same bits every time.
//
// Bound by HBM where rows are whole 16-byte pieces ([8192, 4096] bf16 24.1 us, 5.6 TB/s; its
// gradient with a residual 51, without 43; [65536, 512] fp32 gradient 73, 5.5 TB/s).  Where
// they are not, an element is a load from the ring and a store of its own: loads of one
// element and fixed latencies are what warps wait for, at 52% (back 62%) of the SM's busiest
// unit ([8192, 4095] bf16 50.5 and 82 us, fp32 49 and 72; read from memory by the lanes,
// without the ring: 106 and 188, 123 and 206).  Few rows are bound by latency: one of 4096
// 3.1 us, its gradient 5.5 in two launches.
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "mbarrier.cuh"
#include "ops.h"

namespace muon {

namespace {

constexpr int kEach = 16;        // elements of a row that a thread holds
constexpr int kSmallBlock = 128; // threads of a block whose warps hold whole rows
// Blocks of them on an SM, by the elements of a load: as many as the registers allow
// without spills that cost more than a block less ([131072, 256] bf16 back: 45 us with
// four, 47 with three; [131072, 255]: 142 with four, 88 with two; forward: 51 with four,
// 116 with six).
constexpr int small_blocks(int n, bool backward) { return backward ? (n == 1 ? 2 : n == 4 ? 3 : 4) : (n == 1 ? 4 : 6); }
constexpr int kMostThreads = 512;
constexpr int kMostHeld = 1024;  // of k_norm_backward_held
constexpr int kPartRows = 512;   // most rows a thread adds up one after another

// N neighbouring elements (16 bytes of them if N > 1) in the form they are loaded in.
template <typename T, int N>
struct Piece {
  static constexpr int kLoads = N == 1 ? 1 : N * (int)sizeof(T) / 16;
  uint4 u[kLoads];
  T one;
  __device__ __forceinline__ void fetch(const T* p) {
    if constexpr (N == 1) {
      one = *p;
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
    }
  }
  __device__ __forceinline__ void stream(const T* p) {  // read once
    if constexpr (N == 1) {
      one = *p;
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) u[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
  }
  __device__ __forceinline__ void zero() {
    if constexpr (N == 1) {
      one = T(0.f);
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) u[i] = make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void open(float* f) const {
    if constexpr (N == 1) {
      f[0] = to_f32(one);
    } else {
      const T* h = reinterpret_cast<const T*>(u);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = to_f32(h[i]);
    }
  }
};
template <typename T, int N>
__device__ __forceinline__ void put(T* p, const float* f) {
  if constexpr (N == 1) {
    *p = from_f32<T>(f[0]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
    uint4 u;
    uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(p) = u;
  }
}

// Two elements at a time.
__device__ __forceinline__ float2 at2(const float* f, int i) { return make_float2(f[2 * i], f[2 * i + 1]); }
__device__ __forceinline__ void set2(float* f, int i, float2 v) { f[2 * i] = v.x; f[2 * i + 1] = v.y; }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Sums over the threads of a row: lanes of a warp (lanes of them, a power of two),
// or the block.  A block's sums alternate between two buffers, so that one barrier
// each is enough.
using Sums = float[2][2][32];  // [buffer][value][warp], zeros behind the last warp
template <bool kWarp>
struct RowSum {
  Sums* red;
  int lanes, turn;
  __device__ __forceinline__ void init() {
    if constexpr (!kWarp) {
      for (int i = threadIdx.x; i < 128; i += blockDim.x) (&(*red)[0][0][0])[i] = 0.f;
      __syncthreads();
    }
  }
  __device__ __forceinline__ float join(int value) {
    const float4* r = reinterpret_cast<const float4*>((*red)[turn][value]);
    float4 t = r[0];
    for (int w = 1; 128 * w < (int)blockDim.x; ++w) {
      const float4 u = r[w];
      t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
    }
    return (t.x + t.y) + (t.z + t.w);
  }
  __device__ __forceinline__ float lanes_sum(float a) {
    for (int o = lanes >> 1; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
  }
  __device__ __forceinline__ void operator()(float& a, float& b) {
    if constexpr (kWarp) {
      a = lanes_sum(a);
      b = lanes_sum(b);
    } else {
      a = warp_sum(a);
      b = warp_sum(b);
      if ((threadIdx.x & 31) == 0) { (*red)[turn][0][threadIdx.x >> 5] = a; (*red)[turn][1][threadIdx.x >> 5] = b; }
      __syncthreads();
      a = join(0);
      b = join(1);
      turn ^= 1;
    }
  }
  __device__ __forceinline__ void operator()(float& a) {
    if constexpr (kWarp) {
      a = lanes_sum(a);
    } else {
      a = warp_sum(a);
      if ((threadIdx.x & 31) == 0) (*red)[turn][0][threadIdx.x >> 5] = a;
      __syncthreads();
      a = join(0);
      turn ^= 1;
    }
  }
};

// Rows of a block on their way: `kTensors` tensors' rows to a slot, by bulk copies that
// one thread issues and a barrier counts.  A slot is free once every thread of the block
// has taken its pieces: after the next __syncthreads.  A row that starts or ends between
// two 16-byte boundaries comes with the bytes around it up to them (of the same 16 as its
// own ends, so of the same allocation), which nobody looks at.
//
// A wait that runs out ends the block: who gave up sets the row's flag, which all of its
// threads read after the next __syncthreads (gave_up), so that they agree; nothing more is
// fetched or stored, the copies in flight land, and the block leaves.  A flag is set
// again only behind a further barrier that everyone comes to after having read it:
// rows with one barrier take turns at two flags.
constexpr int kMostSlots = 8;
template <int kTensors, bool kWhole>  // kWhole: rows start and end on 16 bytes
struct RowRing {
  uint8_t* slots;
  uint64_t* full;
  volatile int* state;         // two flags; the waits' limit in 1024 cycles
  const NormArgs& a;
  uint32_t row_bytes;
  int n, at;                   // slots, the current one
  uint32_t phase;
  const uint8_t* src[kTensors];  // nullable
  int64_t pitch[kTensors];       // bytes between rows

  static __device__ __forceinline__ uint32_t shared(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
  __device__ __forceinline__ void init() {
    const int i = threadIdx.x;  // (a barrier a thread: all by one took 0.1 us of the latency of few rows)
    if (i < n) {
      mbar_init(shared(full + i), i == a.lost_slot - 1 && (int)blockIdx.x == a.lost_block ? 2 : 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (i < 2) state[i] = 0;
    if (i == 2) state[2] = a.wait_limit;
    __syncthreads();
  }
  __device__ __forceinline__ uintptr_t start(int t, int64_t row) const {
    return reinterpret_cast<uintptr_t>(src[t]) + row * pitch[t];
  }
  __device__ __forceinline__ uint32_t window(uintptr_t p) const {
    return kWhole ? row_bytes : ((uint32_t)(p & 15) + row_bytes + 15) & ~15u;
  }
  __device__ __forceinline__ void fetch(int slot, int64_t row) {  // one thread
    const uint32_t bar = shared(full + slot);
    uint32_t to = shared(slots) + slot * a.slot_bytes, bytes = 0;
#pragma unroll
    for (int t = 0; t < kTensors; ++t) bytes += src[t] ? window(start(t, row)) : 0;
    mbar_expect_tx(bar, bytes);
#pragma unroll
    for (int t = 0; t < kTensors; ++t, to += a.part_bytes) {
      if (!src[t]) continue;
      const uintptr_t p = start(t, row);
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
                   "l"(p & ~(uintptr_t)15), "r"(window(p)), "r"(bar)
                   : "memory");
    }
  }
  // Waits for the current slot's rows: there unless a thread gave up.
  __device__ __forceinline__ void take(int flag) {
    mbar_wait_within(shared(full + at), phase, state + flag, a.err, 1 << 16, [&] { return (long long)state[2] << 10; });
  }
  __device__ __forceinline__ bool gave_up(int flag) const { return state[flag] != 0; }
  // The copies in flight land before the block's shared memory goes to another.
  __device__ __forceinline__ void drain() const {
    if (threadIdx.x != 0) return;
    const long long t0 = clock64();
    while (clock64() - t0 < (1ll << 21)) {}
  }
  __device__ __forceinline__ const uint8_t* row_of(int t, int64_t row) const {
    return slots + at * a.slot_bytes + t * a.part_bytes + (kWhole ? 0 : start(t, row) & 15);
  }
  __device__ __forceinline__ void next() {
    if (++at == n) { at = 0; phase ^= 1; }
  }
};

// Where a thread stands: its row within the block's round, and its first column of
// each piece (col + p * step).
struct Place {
  int row, rows;   // of this round, rows a round
  int col, step;
};
template <bool kWarp, int N>
__device__ __forceinline__ Place place(int lanes) {
  if constexpr (kWarp) {
    const int t = threadIdx.x & (lanes - 1);
    return {(int)threadIdx.x / lanes, (int)blockDim.x / lanes, t * N, lanes * N};
  } else {
    return {0, 1, (int)threadIdx.x * N, (int)blockDim.x * N};
  }
}

template <typename W, int N>
__device__ __forceinline__ void load_weights(const void* w, int col, bool live, float fill, float* f) {
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = fill;
  if (w && live) {
    Piece<W, N> v;
    v.fetch(static_cast<const W*>(w) + col);
    v.open(f);
  }
}

template <int N>
__device__ __forceinline__ void put_sums(float* out, const float* s) {
  if constexpr (N == 1) {
    *out = *s;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(out + i) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
  }
}

// E elements a thread; kThreads: most threads of a block, kBlocks of which fit on an SM.
template <typename T, typename W, int N, int E, bool kWarp, int kThreads, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) k_norm(NormArgs a, int lanes) {
  constexpr int P = E / N;
  constexpr bool kRing = !kWarp;
  __shared__ __align__(16) Sums red;
  extern __shared__ __align__(128) uint8_t ring_bytes[];
  __shared__ uint64_t full[kMostSlots];
  __shared__ int state[3];
  grid_launch_next();
  const Place at = place<kWarp, N>(lanes);
  RowSum<kWarp> sum{&red, lanes, 0};
  sum.init();
  const int h = (int)a.width;
  bool live[P];
#pragma unroll
  for (int p = 0; p < P; ++p) live[p] = at.col + p * at.step < h;
  grid_wait();
  const T* x = static_cast<const T*>(a.x) + at.col;
  T* y = static_cast<T*>(a.y) + at.col;
  const int64_t by = (int64_t)gridDim.x * at.rows;
  int64_t first = (int64_t)blockIdx.x * at.rows;  // the round's first row: the same for the block
  RowRing<1, (N > 1)> ring{ring_bytes, full, state, a, (uint32_t)(h * sizeof(T)), a.slots, 0, 0,
                  {static_cast<const uint8_t*>(a.x)}, {a.x_stride * (int64_t)sizeof(T)}};
  Piece<T, N> v[P];
  if constexpr (kRing) {
    ring.init();
    if (threadIdx.x == 0)
      for (int i = 0; i < a.slots && first + i * by < a.rows; ++i) ring.fetch(i, first + i * by);
  } else {
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (live[p] && first + at.row < a.rows) v[p].stream(x + (first + at.row) * a.x_stride + p * at.step);
  }
  float w[E], b[E];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    load_weights<W, N>(a.w, at.col + p * at.step, live[p], 1.f, w + p * N);
    load_weights<W, N>(a.bias, at.col + p * at.step, live[p], 0.f, b + p * N);
  }
  // (a running address costs less than a product a row: [65536, 520] bf16 46.5 us against 49.2; the
  // forms with more pieces have no registers left for it)
  constexpr bool kRunning = kRing && N == 8;
  T* out = y + first * h;
  const int64_t out_step = by * h;
  for (; first < a.rows; first += by) {
    const int64_t row = first + at.row;
    float f[E];
    if constexpr (kRing) {
      ring.take(0);
      const T* sx = reinterpret_cast<const T*>(ring.row_of(0, row)) + at.col;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        Piece<T, N> u;
        u.zero();
        if (live[p]) u.fetch(sx + p * at.step);
        u.open(f + p * N);
      }
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        if (live[p] && row < a.rows) {
          v[p].open(f + p * N);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) f[p * N + i] = 0.f;
        }
        if (live[p] && row + by < a.rows) v[p].stream(x + (row + by) * a.x_stride + p * at.step);
      }
    }
    float2 s2 = at2(f, 0);
#pragma unroll
    for (int i = 1; i < E / 2; ++i) s2 = __fadd2_rn(s2, at2(f, i));
    float s = s2.x + s2.y;
    sum(s);
    if constexpr (kRing) {  // (every thread has its pieces: the sum was a barrier)
      if (ring.gave_up(0)) { ring.drain(); return; }
      if (threadIdx.x == 0 && row + a.slots * by < a.rows) ring.fetch(ring.at, row + a.slots * by);
      ring.next();
    }
    const float mean = s / (float)h;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) set2(f, i, __fadd2_rn(at2(f, i), both(-mean)));
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (live[p]) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) f[p * N + i] = 0.f;
    }
    float2 q2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) q2 = __ffma2_rn(at2(f, i), at2(f, i), q2);
    float q = q2.x + q2.y;
    sum(q);
    const float rstd = 1.f / sqrtf(q / (float)h + a.eps);
    if (row >= a.rows) continue;  // (after the sums, which every lane takes part in)
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
      set2(f, i, __ffma2_rn(__fmul2_rn(at2(f, i), both(rstd)), at2(w, i), at2(b, i)));
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (live[p]) put<T, N>((kRunning ? out : y + row * h) + p * at.step, f + p * N);
    if (kRunning) out += out_step;
    if (at.col == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// Rows first .. last - 1 of a part; its sums go to row `part` of a.part.
template <typename T, typename W, int N, bool kWarp>
__global__ void __launch_bounds__(kWarp ? kSmallBlock : kMostThreads, kWarp ? small_blocks(N, true) : 1)
    k_norm_backward(NormArgs a, int lanes) {
  constexpr int P = kEach / N;
  constexpr bool kRing = !kWarp;
  __shared__ __align__(16) Sums red;
  extern __shared__ __align__(128) uint8_t ring_bytes[];
  float* fold = reinterpret_cast<float*>(ring_bytes);  // kWarp: [warps][2][width]
  __shared__ uint64_t full[kMostSlots];
  __shared__ int state[3];
  grid_launch_next();
  const Place at = place<kWarp, N>(lanes);
  RowSum<kWarp> sum{&red, lanes, 0};
  sum.init();
  const int h = (int)a.width;
  bool live[P];
#pragma unroll
  for (int p = 0; p < P; ++p) live[p] = at.col + p * at.step < h;
  grid_wait();
  const T* x = static_cast<const T*>(a.x) + at.col;
  const T* dy = static_cast<const T*>(a.dy) + at.col;
  const T* res = static_cast<const T*>(a.residual) + at.col;
  T* dx = static_cast<T*>(a.dx) + at.col;
  float w[kEach];
#pragma unroll
  for (int p = 0; p < P; ++p) load_weights<W, N>(a.w, at.col + p * at.step, live[p], 1.f, w + p * N);
  const float per = 1.f / (float)h;
  RowRing<3, (N > 1)> ring{ring_bytes, full, state, a, (uint32_t)(h * sizeof(T)), a.slots, 0, 0,
                  {static_cast<const uint8_t*>(a.x), static_cast<const uint8_t*>(a.dy),
                   a.dx ? static_cast<const uint8_t*>(a.residual) : nullptr},
                  {a.x_stride * (int64_t)sizeof(T), a.dy_stride * (int64_t)sizeof(T), a.r_stride * (int64_t)sizeof(T)}};
  if constexpr (kRing) ring.init();
  for (int64_t part = blockIdx.x; part < a.parts; part += gridDim.x) {
    const int64_t last = min(a.rows, (part + 1) * a.part_rows);
    int64_t first = part * a.part_rows;
    if constexpr (kRing) {  // (the part before has used up what it fetched)
      if (threadIdx.x == 0)
        for (int i = 0; i < a.slots && first + i < last; ++i)
          ring.fetch(ring.at + i < a.slots ? ring.at + i : ring.at + i - a.slots, first + i);
    }
    float sw[kEach] = {}, sb[kEach] = {};
    Piece<T, N> vx[P], vd[P];
    float mean = 0.f, rstd = 0.f;
    if (first + at.row < last) {
      const int64_t row = first + at.row;
      mean = a.mean[row];
      rstd = a.rstd[row];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        if (kRing || !live[p]) continue;
        vx[p].stream(x + row * a.x_stride + p * at.step);
        vd[p].stream(dy + row * a.dy_stride + p * at.step);
      }
    }
    for (; first < last; first += at.rows) {
      const int64_t row = first + at.row, next = row + at.rows;
      const bool mine = row < last;
      float xh[kEach], d[kEach];
      float s1, s2;
      Piece<T, N> vr[P];
      if constexpr (kRing) {
        ring.take(sum.turn);
        const T* sx = reinterpret_cast<const T*>(ring.row_of(0, row)) + at.col;
        const T* sd = reinterpret_cast<const T*>(ring.row_of(1, row)) + at.col;
        const T* sr = reinterpret_cast<const T*>(ring.row_of(2, row)) + at.col;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          Piece<T, N> ux, ud;
          ud.zero();
          if (live[p]) {
            ux.fetch(sx + p * at.step);
            ud.fetch(sd + p * at.step);
            if (ring.src[2]) vr[p].fetch(sr + p * at.step);
          }
          ux.open(xh + p * N);
          ud.open(d + p * N);
          if (live[p]) continue;
#pragma unroll
          for (int i = 0; i < N; ++i) xh[p * N + i] = mean;
        }
      } else {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          if (mine && live[p]) {
            vx[p].open(xh + p * N);
            vd[p].open(d + p * N);
          } else {
#pragma unroll
            for (int i = 0; i < N; ++i) xh[p * N + i] = mean, d[p * N + i] = 0.f;
          }
          if (next < last && live[p]) {
            vx[p].stream(x + next * a.x_stride + p * at.step);
            vd[p].stream(dy + next * a.dy_stride + p * at.step);
          }
        }
      }
      const float r = rstd;
      {
        float2 t1 = make_float2(0.f, 0.f), t2 = t1;
#pragma unroll
        for (int i = 0; i < kEach / 2; ++i) {
          const float2 x2 = __fmul2_rn(__fadd2_rn(at2(xh, i), both(-mean)), both(r)), d2 = at2(d, i);
          const float2 g = __fmul2_rn(d2, at2(w, i));
          t1 = __fadd2_rn(t1, g);
          t2 = __ffma2_rn(g, x2, t2);
          set2(sw, i, __ffma2_rn(d2, x2, at2(sw, i)));
          set2(sb, i, __fadd2_rn(at2(sb, i), d2));
          set2(xh, i, x2);
        }
        s1 = t1.x + t1.y;
        s2 = t2.x + t2.y;
      }
      if (next < last) {
        mean = a.mean[next];
        rstd = a.rstd[next];
      } else {
        mean = rstd = 0.f;
      }
      if (!kRing && !a.dx) continue;
      if (!kRing && a.residual && mine) {
#pragma unroll
        for (int p = 0; p < P; ++p)
          if (live[p]) vr[p].stream(res + row * a.r_stride + p * at.step);
      }
      sum(s1, s2);
      if constexpr (kRing) {  // (every thread has its pieces: the sum was a barrier)
        if (ring.gave_up(sum.turn ^ 1)) { ring.drain(); return; }
        if (threadIdx.x == 0 && row + a.slots < last) ring.fetch(ring.at, row + a.slots);
        ring.next();
        if (!a.dx) continue;
      }
      s1 *= per;
      s2 *= per;
      if (!mine) continue;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        if (!live[p]) continue;
        float o[N], add[N] = {};
        if (a.residual) vr[p].open(add);
        if constexpr (N == 1) {
          o[0] = fmaf(r, fmaf(-xh[p], s2, fmaf(d[p], w[p], -s1)), add[0]);
        } else {
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            const int j = p * (N / 2) + i;
            const float2 t = __ffma2_rn(at2(d, j), at2(w, j), both(-s1));
            set2(o, i, __ffma2_rn(both(r), __ffma2_rn(at2(xh, j), both(-s2), t), at2(add, i)));
          }
        }
        put<T, N>(dx + row * h + p * at.step, o);
      }
    }
    if (!a.part) continue;
    float* out = a.part + part * 2 * h + at.col;
    if constexpr (kWarp) {  // the rows of a round, then the warps
      const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        for (int o = lanes; o < 32; o <<= 1) {
          sw[i] += __shfl_xor_sync(0xffffffffu, sw[i], o);
          sb[i] += __shfl_xor_sync(0xffffffffu, sb[i], o);
        }
      }
      __syncthreads();
      if (lane < lanes) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          if (!live[p]) continue;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            fold[warp * 2 * h + at.col + p * at.step + i] = sw[p * N + i];
            fold[warp * 2 * h + h + at.col + p * at.step + i] = sb[p * N + i];
          }
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 2 * h; i += blockDim.x) {
        float s = 0.f;
        for (int k = 0; k < warps; ++k) s += fold[k * 2 * h + i];
        a.part[part * 2 * h + i] = s;
      }
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        if (!live[p]) continue;
        put_sums<N>(out + p * at.step, sw + p * N);
        put_sums<N>(out + h + p * at.step, sb + p * N);
      }
    }
  }
}

// The gradient of rows that fill a block's registers with their sums over rows alone:
// they stay in the ring, and are read twice from there ([2048, 16384] bf16 79 us, [3000,
// 9000] 64; read again from memory, and once more for dw: 120 and 118).
template <typename T, typename W, int N>
__global__ void __launch_bounds__(kMostHeld) k_norm_backward_held(NormArgs a) {
  constexpr int P = kEach / N;
  __shared__ __align__(16) Sums red;
  extern __shared__ __align__(128) uint8_t ring_bytes[];
  __shared__ uint64_t full[kMostSlots];
  __shared__ int state[3];
  grid_launch_next();
  RowSum<false> sum{&red, 32, 0};
  sum.init();
  const int h = (int)a.width, step = (int)blockDim.x * N, col = (int)threadIdx.x * N;
  grid_wait();
  const float per = 1.f / (float)h;
  RowRing<3, (N > 1)> ring{ring_bytes, full, state, a, (uint32_t)(h * sizeof(T)), a.slots, 0, 0,
                           {static_cast<const uint8_t*>(a.x), static_cast<const uint8_t*>(a.dy),
                            a.dx ? static_cast<const uint8_t*>(a.residual) : nullptr},
                           {a.x_stride * (int64_t)sizeof(T), a.dy_stride * (int64_t)sizeof(T),
                            a.r_stride * (int64_t)sizeof(T)}};
  ring.init();
  int flag = 0;
  for (int64_t part = blockIdx.x; part < a.parts; part += gridDim.x) {
    const int64_t first = part * a.part_rows, last = min(a.rows, first + a.part_rows);
    if (threadIdx.x == 0)
      for (int i = 0; i < a.slots && first + i < last; ++i)
        ring.fetch(ring.at + i < a.slots ? ring.at + i : ring.at + i - a.slots, first + i);
    float sw[kEach] = {}, sb[kEach] = {};
    float next_mean = a.mean[first], next_rstd = a.rstd[first];
    for (int64_t row = first; row < last; ++row) {
      const float mean = next_mean, rstd = next_rstd;
      if (row + 1 < last) {
        next_mean = a.mean[row + 1];
        next_rstd = a.rstd[row + 1];
      }
      ring.take(flag);
      const T* sx = reinterpret_cast<const T*>(ring.row_of(0, row)) + col;
      const T* sd = reinterpret_cast<const T*>(ring.row_of(1, row)) + col;
      const T* sr = reinterpret_cast<const T*>(ring.row_of(2, row)) + col;
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        if (col + p * step >= h) continue;
        Piece<T, N> v;
        float x[N], d[N], w[N];
        v.fetch(sx + p * step);
        v.open(x);
        v.fetch(sd + p * step);
        v.open(d);
        load_weights<W, N>(a.w, col + p * step, true, 1.f, w);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float xh = (x[i] - mean) * rstd, g = d[i] * w[i];
          s1 += g;
          s2 = fmaf(g, xh, s2);
          sw[p * N + i] = fmaf(d[i], xh, sw[p * N + i]);
          sb[p * N + i] += d[i];
        }
      }
      if (a.dx) {
        sum(s1, s2);
        if (ring.gave_up(flag)) { ring.drain(); return; }
        s1 *= per;
        s2 *= per;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          if (col + p * step >= h) continue;
          Piece<T, N> v;
          float x[N], d[N], w[N], add[N] = {};
          v.fetch(sx + p * step);
          v.open(x);
          v.fetch(sd + p * step);
          v.open(d);
          if (a.residual) {
            v.fetch(sr + p * step);
            v.open(add);
          }
          load_weights<W, N>(a.w, col + p * step, true, 1.f, w);
#pragma unroll
          for (int i = 0; i < N; ++i)
            x[i] = fmaf(rstd, fmaf((mean - x[i]) * rstd, s2, fmaf(d[i], w[i], -s1)), add[i]);
          put<T, N>(static_cast<T*>(a.dx) + row * h + col + p * step, x);
        }
      }
      __syncthreads();  // everyone is done with the slot
      if (ring.gave_up(flag)) { ring.drain(); return; }
      if (threadIdx.x == 0 && row + a.slots < last) ring.fetch(ring.at, row + a.slots);
      ring.next();
      flag ^= 1;
    }
    if (!a.part) continue;
    float* out = a.part + part * 2 * h + col;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (col + p * step >= h) continue;
      put_sums<N>(out + p * step, sw + p * N);
      put_sums<N>(out + h + p * step, sb + p * N);
    }
  }
}

// A thread's sum over a row of any length (up to 2^20 numbers of 2^30): each addition's
// rounding error, which two differences give exactly, is kept and added at the end.  In a
// running sum alone a row of 4 million equal numbers is off by 6e-5, its mean and rstd with
// it; this costs 1 to 7% ([400, 40000] bf16 26.7 -> 27.5 us, back 77 -> 78).  Sums in
// levels of 64 pieces cost more: the loops over pieces are then unrolled less ([8, 2^21]
// bf16 257 us as a running sum, 272 so, 334 in levels).
struct LongSum {
  float s = 0.f, low = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float t = s + v, b = t - s;
    low += (s - (t - b)) + (v - b);
    s = t;
  }
  // (beyond the largest number there is no error to tell)
  __device__ __forceinline__ float total() const { return fabsf(s) < __int_as_float(0x7f800000) ? s + low : s; }
};

// Rows that no block holds: read again for each sum (from L2).  One block a row.
template <typename T, typename W, int N>
__global__ void __launch_bounds__(1024) k_norm_wide(NormArgs a) {
  __shared__ __align__(16) Sums red;
  grid_launch_next();
  grid_wait();
  RowSum<false> sum{&red, 32, 0};
  sum.init();
  const int64_t h = a.width, step = (int64_t)blockDim.x * N, c0 = (int64_t)threadIdx.x * N;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    LongSum s_sum, q_sum;
    for (int64_t c = c0; c < h; c += step) {
      Piece<T, N> v;
      float f[N], t = 0.f;
      v.fetch(x + c);
      v.open(f);
#pragma unroll
      for (int i = 0; i < N; ++i) t += f[i];
      s_sum.add(t);
    }
    float s = s_sum.total();
    sum(s);
    const float mean = s / (float)h;
    for (int64_t c = c0; c < h; c += step) {
      Piece<T, N> v;
      float f[N], t = 0.f;
      v.fetch(x + c);
      v.open(f);
#pragma unroll
      for (int i = 0; i < N; ++i) t = fmaf(f[i] - mean, f[i] - mean, t);
      q_sum.add(t);
    }
    float q = q_sum.total();
    sum(q);
    const float rstd = 1.f / sqrtf(q / (float)h + a.eps);
    for (int64_t c = c0; c < h; c += step) {
      Piece<T, N> v;
      float f[N], w[N], b[N];
      v.fetch(x + c);
      v.open(f);
      load_weights<W, N>(a.w, (int)c, true, 1.f, w);
      load_weights<W, N>(a.bias, (int)c, true, 0.f, b);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = fmaf((f[i] - mean) * rstd, w[i], b[i]);
      put<T, N>(static_cast<T*>(a.y) + row * h + c, f);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

template <typename T, typename W, int N>
__global__ void __launch_bounds__(1024) k_norm_wide_dx(NormArgs a) {
  __shared__ __align__(16) Sums red;
  grid_launch_next();
  grid_wait();
  RowSum<false> sum{&red, 32, 0};
  sum.init();
  const int64_t h = a.width, step = (int64_t)blockDim.x * N, c0 = (int64_t)threadIdx.x * N;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
    const float mean = a.mean[row], rstd = a.rstd[row];
    LongSum sum1, sum2;
    float s1 = 0.f, s2 = 0.f;
    for (int pass = 0; pass < 2; ++pass) {
      for (int64_t c = c0; c < h; c += step) {
        Piece<T, N> v;
        float f[N], d[N], w[N], add[N] = {}, t1 = 0.f, t2 = 0.f;
        v.fetch(x + c);
        v.open(f);
        v.fetch(dy + c);
        v.open(d);
        load_weights<W, N>(a.w, (int)c, true, 1.f, w);
        if (pass && a.residual) {
          v.fetch(static_cast<const T*>(a.residual) + row * a.r_stride + c);
          v.open(add);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float xh = (f[i] - mean) * rstd, g = d[i] * w[i];
          if (pass) {
            f[i] = fmaf(rstd, g - s1 - xh * s2, add[i]);
          } else {
            t1 += g;
            t2 = fmaf(g, xh, t2);
          }
        }
        if (!pass) {
          sum1.add(t1);
          sum2.add(t2);
        }
        if (pass) put<T, N>(static_cast<T*>(a.dx) + row * h + c, f);
      }
      if (pass) break;
      s1 = sum1.total();
      s2 = sum2.total();
      sum(s1, s2);
      s1 /= (float)h;
      s2 /= (float)h;
    }
  }
}

// Partial sums of dw and db for the same: a thread's columns over a part's rows.
template <typename T, int N>
__global__ void __launch_bounds__(256) k_norm_wide_dw(NormArgs a, int col_blocks) {
  grid_launch_next();
  grid_wait();
  const int64_t h = a.width, c = ((int64_t)(blockIdx.x % col_blocks) * 256 + threadIdx.x) * N;
  const int64_t part = blockIdx.x / col_blocks;
  if (c >= h) return;
  float sw[N] = {}, sb[N] = {};
  const int64_t last = min(a.rows, (part + 1) * a.part_rows);
#pragma unroll 4
  for (int64_t row = part * a.part_rows; row < last; ++row) {
    Piece<T, N> vx, vd;
    float f[N], d[N];
    vx.fetch(static_cast<const T*>(a.x) + row * a.x_stride + c);
    vd.fetch(static_cast<const T*>(a.dy) + row * a.dy_stride + c);
    vx.open(f);
    vd.open(d);
    const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      sw[i] = fmaf(d[i], (f[i] - mean) * rstd, sw[i]);
      sb[i] += d[i];
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a.part[part * 2 * h + c + i] = sw[i];
    a.part[part * 2 * h + h + c + i] = sb[i];
  }
}

// dw and db from the parts' sums: 32 columns a block, the parts shared out over 32
// warps and added in order, then the warps'.
template <typename W>
__global__ void __launch_bounds__(1024) k_norm_join(NormArgs a) {
  __shared__ float red[32][33];
  grid_launch_next();
  grid_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t h = a.width, c = (int64_t)blockIdx.x * 32 + lane;  // column of [dw, db]
  float s = 0.f;
  if (c < 2 * h) {
#pragma unroll 8
    for (int64_t p = warp; p < a.parts; p += 32) s += a.part[p * 2 * h + c];
  }
  red[warp][lane] = s;
  __syncthreads();
  s = warp_sum(red[lane][warp]);  // column `warp` of the block
  const int64_t mine = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && mine < 2 * h) {
    if (mine < h) {
      if (a.dw) static_cast<W*>(a.dw)[mine] = from_f32<W>(s);
    } else if (a.db) {
      static_cast<W*>(a.db)[mine - h] = from_f32<W>(s);
    }
  }
}

// How rows of this width are held: by lanes of a warp, by a block (`each` elements a
// thread, `blocks` blocks an SM), in the ring, or by none.  Forward, rows but fp32 ones in
// whole pieces take 32 elements a thread where there are rows enough to fill the GPU: the
// sums over a row then cost half as much of a thread ([8192, 4096] bf16: 24.1 us, 29.2 with
// 16; fp32 in whole pieces is bound by HBM with either, 48.4 with 16, 47.7 with 32).  Rows
// that 256 threads of 16 do not hold take 32 too ([2000, 12001] bf16 47.7 us; read again for
// each sum 83).
struct Form {
  bool warp, held, wide;
  int lanes, threads, each, blocks;
};
Form form_of(int64_t rows, int64_t width, int n, bool backward) {
  const auto threads_of = [&](int64_t each) { return ((width + n - 1) / n * n + each - 1) / each; };
  const int64_t t = threads_of(kEach), t2 = threads_of(2 * kEach);
  Form f{false, false, false, 32, 0, kEach, 1};
  if (t <= 32) {
    f.warp = true;
    f.lanes = 1;
    while (f.lanes < t) f.lanes *= 2;
    f.threads = kSmallBlock;
    f.blocks = small_blocks(n, backward);
  } else if (backward ? t <= 512 : (t <= 256 && (n == 4 || rows < 2 * num_sms() || t2 < 64))) {
    f.threads = (int)((t + 31) / 32 * 32);
    f.blocks = f.threads > 256 ? 1 : (backward ? 512 : 768) / f.threads;
  } else if (!backward && t2 <= 512) {
    f.each = 2 * kEach;
    f.threads = (int)((t2 + 31) / 32 * 32);
    f.blocks = 512 / f.threads;
  } else if (backward && t <= kMostHeld) {
    f.held = true;
    f.threads = (int)((t + 31) / 32 * 32);
  } else {
    f.wide = true;
    f.threads = 1024;
    f.blocks = 2;
  }
  return f;
}

bool aligned(const void* p, int64_t stride, int64_t size) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride * size % 16 == 0;
}
template <typename T, typename W>
bool vector_rows(const NormArgs& a) {
  constexpr int64_t b = sizeof(T);
  return a.width * b % 16 == 0 && aligned(a.x, a.rows > 1 ? a.x_stride : 0, b) && aligned(a.y, 0, b) &&
         aligned(a.dy, a.rows > 1 ? a.dy_stride : 0, b) && aligned(a.dx, 0, b) &&
         aligned(a.residual, a.rows > 1 ? a.r_stride : 0, b) && aligned(a.w, 0, sizeof(W)) &&
         aligned(a.bias, 0, sizeof(W));
}

// Parts of the sum over rows: one a resident block (about 512 threads an SM), and
// no more than kPartRows rows one after another.
void set_parts(NormArgs* a, int n) {
  const Form f = form_of(a->rows, a->width, n, true);
  int64_t each, most;
  if (f.wide) {
    const int64_t col_blocks = (a->width + 256ll * n - 1) / (256ll * n);
    most = (8ll * num_sms() + col_blocks - 1) / col_blocks;
    each = 1;
  } else {
    most = (int64_t)num_sms() * f.blocks;
    each = f.warp ? f.threads / f.lanes : 1;  // rows a round
  }
  int64_t rows = (a->rows + most - 1) / most;
  rows = (rows + each - 1) / each * each;
  if (rows > kPartRows * each) rows = kPartRows * each;
  a->part_rows = rows < 1 ? 1 : rows;
  a->parts = (a->rows + a->part_rows - 1) / a->part_rows;
}

// The ring of a block: what fits of `blocks` blocks an SM.
constexpr int64_t kRingBytes = 208 * 1024;
size_t set_slots(NormArgs* a, int64_t row_bytes, int tensors, bool whole, int64_t blocks) {
  a->part_bytes = (uint32_t)(whole ? row_bytes : (row_bytes + 15) / 16 * 16 + 16);
  const int64_t slot_bytes = (int64_t)tensors * a->part_bytes;
  const int64_t n = kRingBytes / (blocks < 1 ? 1 : blocks) / slot_bytes;
  a->slot_bytes = (uint32_t)slot_bytes;
  a->slots = (int)(n < 1 ? 1 : (n < kMostSlots ? n : kMostSlots));
  return (size_t)(a->slots * slot_bytes);
}
// Shared memory beyond the default (once per device and kernel; kernels of one type
// share a table).
template <typename F>
cudaError_t allow(F fn) {
  static std::mutex mu;
  static struct {
    F fn;
    bool ready[64];
  } table[40] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  bool* ready = nullptr;
  for (auto& t : table) {
    if (t.fn == nullptr) t.fn = fn;
    if (t.fn != fn) continue;
    if (dev < 64) ready = &t.ready[dev];
    break;
  }
  if (ready && *ready) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes);
  if (e == cudaSuccess && ready) *ready = true;
  return e;
}

template <typename T, typename W, int N>
cudaError_t forward(NormArgs a, cudaStream_t s) {
  const Form f = form_of(a.rows, a.width, N, false);
  const int64_t each = f.warp ? f.threads / f.lanes : 1;
  const int64_t rounds = (a.rows + each - 1) / each, most = (int64_t)num_sms() * f.blocks;
  const dim3 grid((unsigned)(rounds < most ? rounds : most)), block((unsigned)f.threads);
  if (f.wide) return launch_early(k_norm_wide<T, W, N>, grid, block, 0, s, a);
  if (f.warp) return launch_early(k_norm<T, W, N, kEach, true, kSmallBlock, small_blocks(N, false)>, grid, block, 0, s, a, f.lanes);
  auto fn = k_norm<T, W, N, kEach, false, 256, 3>;
  if (f.each > kEach)
    fn = f.threads > 256 ? k_norm<T, W, N, 2 * kEach, false, 512, 1> : k_norm<T, W, N, 2 * kEach, false, 256, 2>;
  size_t smem = 0;
  cudaError_t e = ops_error_word(&a.err);
  if (a.wait_limit == 0) a.wait_limit = (int32_t)(kWaitCycles >> 10);
  if (e == cudaSuccess) {
    smem = set_slots(&a, a.width * (int64_t)sizeof(T), 1, N > 1, f.blocks);
    e = allow(fn);
  }
  return e == cudaSuccess ? launch_early(fn, grid, block, smem, s, a, f.lanes) : e;
}

template <typename T, typename W, int N>
cudaError_t backward(NormArgs a, cudaStream_t s) {
  set_parts(&a, N);
  const Form f = form_of(a.rows, a.width, N, true);
  cudaError_t e = cudaSuccess;
  if (f.wide) {
    const int64_t most = (int64_t)num_sms() * 2;
    if (a.dx)
      e = launch_early(k_norm_wide_dx<T, W, N>, dim3((unsigned)(a.rows < most ? a.rows : most)), dim3(1024), 0, s, a);
    const int col_blocks = (int)((a.width + 256ll * N - 1) / (256ll * N));
    if (e == cudaSuccess && a.part)
      e = launch_early(k_norm_wide_dw<T, N>, dim3((unsigned)(col_blocks * a.parts)), dim3(256), 0, s, a, col_blocks);
  } else {
    const int64_t most = (int64_t)num_sms() * f.blocks;
    const dim3 grid((unsigned)(a.parts < most ? a.parts : most)), block((unsigned)f.threads);
    size_t smem = f.warp ? sizeof(float) * 2 * a.width * (f.threads / 32) : 0;
    e = ops_error_word(&a.err);
    if (a.wait_limit == 0) a.wait_limit = (int32_t)(kWaitCycles >> 10);
    if (e == cudaSuccess && !f.warp) {
      smem = set_slots(&a, a.width * (int64_t)sizeof(T), a.dx && a.residual ? 3 : 2, N > 1, f.blocks);
      e = f.held ? allow(k_norm_backward_held<T, W, N>) : allow(k_norm_backward<T, W, N, false>);
    }
    if (e != cudaSuccess) return e;
    if (f.held) e = launch_early(k_norm_backward_held<T, W, N>, grid, block, smem, s, a);
    else e = f.warp ? launch_early(k_norm_backward<T, W, N, true>, grid, block, smem, s, a, f.lanes)
                    : launch_early(k_norm_backward<T, W, N, false>, grid, block, smem, s, a, f.lanes);
  }
  if (e == cudaSuccess && a.part)
    e = launch_early(k_norm_join<W>, dim3((unsigned)((2 * a.width + 31) / 32)), dim3(1024), 0, s, a);
  return e;
}

template <typename T, typename W>
cudaError_t run(const NormArgs& a, bool back, cudaStream_t s) {
  constexpr int N = 16 / (int)sizeof(T);
  if (vector_rows<T, W>(a)) return back ? backward<T, W, N>(a, s) : forward<T, W, N>(a, s);
  return back ? backward<T, W, 1>(a, s) : forward<T, W, 1>(a, s);
}

cudaError_t dispatch(const NormArgs& a, bool back, cudaStream_t s) {
  const bool wide_w = a.w_dtype == DT_F32;
  switch (a.dtype) {
    case DT_F16: return wide_w ? run<__half, float>(a, back, s) : run<__half, __half>(a, back, s);
    case DT_BF16: return wide_w ? run<__nv_bfloat16, float>(a, back, s) : run<__nv_bfloat16, __nv_bfloat16>(a, back, s);
    default: return run<float, float>(a, back, s);
  }
}

}  // namespace

int64_t norm_part_rows(int64_t rows, int64_t width) {
  int64_t most = 0;
  for (const int n : {1, 4, 8}) {  // (whichever the pointers' alignment will allow)
    NormArgs a{};
    a.rows = rows;
    a.width = width;
    set_parts(&a, n);
    if (a.parts > most) most = a.parts;
  }
  return most;
}
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) { return dispatch(a, false, s); }
cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t s) { return dispatch(a, true, s); }

}  // namespace muon
