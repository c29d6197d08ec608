// Internal structures of the layer operators (include/muon_ops.h).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace muon {

enum DType : int32_t { DT_F32 = 0, DT_F16 = 1, DT_BF16 = 2 };
enum Act : int32_t { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4 };

// Which dimension the experts' row ranges cut.
enum GroupMode : int32_t {
  GROUP_NONE = 0,  // one product
  GROUP_ROWS = 1,  // output rows: rows of range e with matrix e (y and dx)
  GROUP_SUM = 2    // the sum: output matrix e sums over the rows of range e (dw)
};

// One product of a layer: D(m, n) = epilogue(sum_k A(m, k) B(k, n)).
struct Product {
  int32_t dtype;
  int32_t mode;                // GroupMode
  int32_t experts;             // ranges (mode != NONE)
  const int32_t* offsets;      // device [experts + 1]
  int64_t M, N, K;             // GROUP_ROWS: M = all rows; GROUP_SUM: K = all rows
  const void* A;               // element (m, k) at m * a_m + k * a_k: one of the two is 1
  int64_t a_m, a_k;
  const void* B;               // element (k, n) at k * b_k + n * b_n: one of the two is 1
  int64_t b_k, b_n, b_e;       // b_e: between matrices (GROUP_ROWS)
  void* D;                     // row pitch N; GROUP_SUM: [experts][M][N]
  // epilogue: z = sum + bias; preact = z; D = act(z) + residual
  int32_t act;
  const void* bias;            // nullable [N], or [experts][N]
  const void* residual;        // nullable, row stride r_m
  int64_t r_m;
  void* preact;                // nullable, row pitch N
  int* err;                    // device error word of the bounded waits
};

// dz = dy * act'(z) (rounded to dtype; not written if act is NONE) and the
// column sums of the unrounded dz per expert (db), each nullable.
struct GradPrep {
  int32_t dtype;
  int32_t act;
  int32_t experts;             // 0: all rows are one range
  const int32_t* offsets;
  int64_t rows, cols;
  const void* dy;
  int64_t dy_stride;
  const void* z;
  void* dz;                    // row pitch dz_stride
  int64_t dz_stride;
  float* part;                 // rows > kGradSingle: [chunks + ranges][cols] partial sums
  void* db;                    // [ranges][cols]
};

// How the tensor-core form runs a product (chosen on the host from sizes).
struct TilePlan {
  int bn;                      // sum form (dw): columns of a pair's tile, 256 or 128; 0: rows form
  int tile_rows;               // rows form: most token rows of a tile, 256, 128 or 64
  int splits;                  // parts of the sum, joined by a second kernel
  int64_t part_bytes;          // scratch of the parts
};
TilePlan tile_plan(const Product& p);
cudaError_t launch_linear_tc(const Product& p, const TilePlan& t, float* part, cudaStream_t s);
// Few token rows: one launch, no scratch (operands as launch_linear_tc's).
bool linear_few_fits(const Product& p);
cudaError_t launch_linear_few(const Product& p, cudaStream_t s);
int num_sms();
// Rows made readable for TMA: 16-bit ones copied to a pitch of whole 16 bytes, dst
// [batch][rows][pitch]; fp32 ones as three bf16 planes, dst [batch][3][rows][pitch].
// batch 0: no job.
struct RowsJob {
  const void* src;
  int64_t stride, batch_stride;
  uint16_t* dst;
  int64_t pitch, rows, cols, batch;
  const int32_t* offsets;      // nullable: matrix b is wanted where offsets[b] < offsets[b + 1]
};
cudaError_t launch_prepare_rows(bool split, const RowsJob& first, const RowsJob& second, cudaStream_t s);
cudaError_t ops_error_word(int** err);  // device address of the error word of the current device

constexpr int kGradChunk = 128;   // rows of one partial column sum
constexpr int kGradSingle = 256;  // up to these rows are summed at once

cudaError_t launch_grad_prep(const GradPrep& g, cudaStream_t s);

struct GateArgs {
  int32_t dtype, experts, top_k, renormalize;
  int64_t tokens, stride;
  const void* logits;
  int32_t* indices;
  float* weights;
  const float* dweights;       // backward
  void* dlogits;
};
cudaError_t launch_gate(const GateArgs& g, cudaStream_t s);
cudaError_t launch_gate_backward(const GateArgs& g, cudaStream_t s);

struct SortArgs {
  int32_t dtype, top_k, experts, index_bits;
  int64_t tokens, hidden;
  const void* x;               // dispatch: token rows
  int64_t x_stride;
  const void* indices;
  void* xs;
  int32_t* slot;
  int32_t* offsets;
  int32_t* counts;             // workspace [chunks][experts], then
  int32_t* total;              // [experts]
  const void* ys;              // rows in expert order
  int64_t ys_stride;
  const float* weights;        // nullable: every weight is 1
  const void* residual;        // nullable
  int64_t r_stride;
  void* y;
  const void* dy;
  int64_t dy_stride;
  void* dys;
  float* dweights;
};
constexpr int kSortChunk = 1024;  // assignments one block counts and places
// Up to these are ordered by one cluster of blocks, without workspace (8000
// assignments 6.3 us against 8.8 in three launches, 32000 14.7 against 11.6).
constexpr int kSortCluster = 1 << 14;
cudaError_t launch_dispatch(const SortArgs& a, cudaStream_t s);
cudaError_t launch_combine(const SortArgs& a, cudaStream_t s);
cudaError_t launch_combine_backward(const SortArgs& a, cudaStream_t s);

}  // namespace muon
