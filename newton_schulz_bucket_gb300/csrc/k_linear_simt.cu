// A layer's product in fp32 FMA: D(m, n) = act(sum_k A(m, k) B(k, n) + bias)
// + residual, for any strides, sizes and expert ranges.
//
// 64 x 64 output tiles, 16 steps of the sum at a time in shared memory, 4 x 4
// accumulators a thread; sums run in k order, so they do not depend on the
// grid.
#include "act.cuh"
#include "common.cuh"

namespace muon {

namespace {

constexpr int TM = 64, TN = 64, TK = 16;

__device__ __forceinline__ int64_t clamp_off(const int32_t* off, int e, int64_t hi) {
  const int64_t v = off[e];
  return v < 0 ? 0 : (v > hi ? hi : v);
}

template <typename T>
__global__ void __launch_bounds__(256) k_linear_simt(Product p) {
  __shared__ float As[TK][TM + 4], Bs[TK][TN + 4];
  __shared__ int64_t range[3];  // first row, end row, expert of this tile
  constexpr bool kFast = sizeof(T) == 2;
  const int tid = threadIdx.x;
  int64_t n0 = (int64_t)blockIdx.y * TN, m0 = (int64_t)blockIdx.x * TM, m_end = p.M;
  int64_t k0 = 0, k1 = p.K;
  int e = 0;
  if (p.mode == GROUP_ROWS) {
    if (tid == 0) {  // tile blockIdx.x of the ranges' tiles, range by range; past them, the unowned rows
      int64_t t = blockIdx.x, lo = 0, hi = 0;
      int g = 0;
      for (; g <= p.experts; ++g) {
        lo = clamp_off(p.offsets, g, p.M);
        hi = g < p.experts ? clamp_off(p.offsets, g + 1, p.M) : p.M;
        const int64_t tiles = hi > lo ? (hi - lo + TM - 1) / TM : 0;
        if (t < tiles) break;
        t -= tiles;
      }
      range[0] = g <= p.experts ? lo + t * TM : p.M;
      range[1] = g <= p.experts ? hi : p.M;
      range[2] = g;
    }
    __syncthreads();
    m0 = range[0];
    m_end = range[1];
    e = (int)range[2];
    if (m0 >= m_end) return;
  } else if (p.mode == GROUP_SUM) {
    e = blockIdx.z;
    k0 = clamp_off(p.offsets, e, p.K);
    k1 = clamp_off(p.offsets, e + 1, p.K);
  }
  const bool unowned = p.mode == GROUP_ROWS && e == p.experts;
  if (unowned) k1 = k0;
  const T* A = static_cast<const T*>(p.A);
  const T* B = static_cast<const T*>(p.B) + (p.mode == GROUP_ROWS && !unowned ? e * p.b_e : 0);
  float acc[4][4] = {};
  const int ty = tid >> 4, tx = tid & 15;
  for (int64_t kb = k0; kb < k1; kb += TK) {
    for (int i = tid; i < TK * TM; i += 256) {
      // consecutive threads along the operand's contiguous dimension
      const int k = p.a_k == 1 ? i % TK : i / TM, m = p.a_k == 1 ? i / TK : i % TM;
      const bool in = kb + k < k1 && m0 + m < m_end;
      As[k][m] = in ? to_f32(A[(m0 + m) * p.a_m + (kb + k) * p.a_k]) : 0.f;
      const int kk = p.b_k == 1 ? i % TK : i / TN, n = p.b_k == 1 ? i / TK : i % TN;
      const bool inb = kb + kk < k1 && n0 + n < p.N;
      Bs[kk][n] = inb ? to_f32(B[(kb + kk) * p.b_k + (n0 + n) * p.b_n]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < TK; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) { a[i] = As[k][ty * 4 + i]; b[i] = Bs[k][tx * 4 + i]; }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
  T* D = static_cast<T*>(p.D) + (p.mode == GROUP_SUM ? (int64_t)e * p.M * p.N : 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + ty * 4 + i;
    if (m >= m_end) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + tx * 4 + j;
      if (n >= p.N) continue;
      float z = acc[i][j], y = 0.f;
      if (unowned) {
        z = 0.f;
      } else {
        if (p.bias) z += to_f32(static_cast<const T*>(p.bias)[(int64_t)e * p.N + n]);
        y = activate<kFast>(z, p.act);
        if (p.residual) y += to_f32(static_cast<const T*>(p.residual)[m * p.r_m + n]);
      }
      if (p.preact) static_cast<T*>(p.preact)[m * p.N + n] = from_f32<T>(z);
      D[m * p.N + n] = from_f32<T>(y);
    }
  }
}

template <typename T>
cudaError_t run(const Product& p, cudaStream_t s) {
  const int64_t tm = (p.M + TM - 1) / TM + (p.mode == GROUP_ROWS ? p.experts + 1 : 0);
  const dim3 grid((unsigned)tm, (unsigned)((p.N + TN - 1) / TN), p.mode == GROUP_SUM ? p.experts : 1);
  k_linear_simt<T><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_simt(const Product& p, cudaStream_t s) {
  switch (p.dtype) {
    case DT_F16: return run<__half>(p, s);
    case DT_BF16: return run<__nv_bfloat16>(p, s);
    default: return run<float>(p, s);
  }
}

}  // namespace muon
