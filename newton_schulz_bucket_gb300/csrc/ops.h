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


// Layer norm and its gradient (w_dtype: of w, bias, dw and db).
struct NormArgs {
  int32_t dtype, w_dtype;
  int64_t rows, width;
  float eps;
  const void* x;
  int64_t x_stride;
  const void* w;               // nullable: ones
  const void* bias;            // nullable
  void* y;                     // row pitch width
  float* mean;                 // forward: nullable
  float* rstd;
  const void* dy;              // backward
  int64_t dy_stride;
  const void* residual;        // nullable
  int64_t r_stride;
  void* dx;                    // nullable, row pitch width
  void* dw;                    // nullable
  void* db;                    // nullable
  float* part;                 // nullable: [parts][2][width] sums of dw and db
  int64_t parts, part_rows;    // set by the launch, as what follows
  uint32_t part_bytes, slot_bytes;  // of the ring of rows on their way
  int32_t slots;
  int* err;
  // Of the waits for a row: their limit in 1024 cycles (0: the library's); and for a test of
  // one that runs out, the slot (from 1; 0: none) of a block whose barrier nothing completes.
  int32_t wait_limit, lost_slot, lost_block;
};
int64_t norm_part_rows(int64_t rows, int64_t width);  // most parts that launch_norm_backward uses
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s);
cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t s);

// A router's balance loss and its gradient.
struct BalanceArgs {
  int32_t dtype, experts, top_k;
  int64_t tokens, stride;
  float coef;
  const void* logits;
  const int32_t* indices;
  float* loss;
  int32_t* counts;             // [experts]
  int32_t* live;
  float* part;                 // [blocks][experts] sums of probabilities, then
  int32_t* part_counts;        // [blocks][experts + 1] assignments and tokens
  int32_t blocks;
  const float* dloss;          // backward
  const void* residual;        // nullable
  int64_t r_stride;
  void* dlogits;
};
int balance_blocks(int64_t tokens, int32_t experts);
cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s);
cudaError_t launch_balance_backward(const BalanceArgs& a, cudaStream_t s);

// Rows of numbers into microscaled 4-bit form and back: values [rows][blocks of 32]
// [16 bytes], scales [rows][blocks], or for a product in the MMA's order (below).
struct MxRows {
  const void* src;             // stored along the sum (rows x cols), or across it (cols x rows)
  int64_t stride, batch_stride;
  int64_t rows, mat_rows, cols;  // rows of all matrices, of one, steps of the sum
  uint8_t* values;
  uint8_t* scales;
  void* dst;                   // back: [rows][cols]
  uint32_t col_blocks;         // set by the launch: column blocks of the grid, and of a row
  int32_t col_total;
  int log_across;
  bool vec;
};
enum MxOp : int32_t { MX_ALONG = 0, MX_ACROSS = 1, MX_BACK = 2 };
int64_t mx_blocks(int64_t rows, int64_t mat_rows, int64_t cols);
cudaError_t launch_mx_rows(int32_t dtype, MxOp op, const MxRows& q, cudaStream_t s);

// Scales in the MMA's order, for a product: a block of 512 bytes holds those of 128 rows
// x 128 steps of the sum (a part), byte (r % 32) * 16 + r / 32 * 4 + block of 32 steps.
// Weights: [matrix][128 features][part][512].  Token rows: a slot for every tile of the
// product, [slot][part][1 or 2 blocks][512], row 0 of a tile at its start.  A range's
// slots start at mx_token_slot, which leaves as many as its tiles can be.
__host__ __device__ constexpr int mx_token_blocks(int tile_rows) { return tile_rows > 128 ? 2 : 1; }
__host__ __device__ constexpr int mx_token_slot(int first_row, int range, int tile_rows) {
  return first_row / tile_rows + range;
}
__host__ __device__ constexpr uint32_t mx_scale_byte(int r, int block) {
  return (uint32_t)((r & 31) * 16 + (r >> 5 & 3) * 4 + (block & 3));
}
inline int64_t mx_blocks_of(int64_t n) { return (n + 31) / 32; }
inline int64_t mx_parts(int64_t n) { return (n + 127) / 128; }
inline int64_t mx_token_slots(int64_t rows, int32_t experts, int tile_rows) {
  return rows / tile_rows + (experts ? experts : 1);
}
int mx_tile_rows(int64_t rows, int32_t experts, int64_t out);

// What a product starts from: the token rows rounded, and both operands' scales in order.
struct MxPrepare {
  MxRows x;                    // scales: [slots]
  int32_t experts;
  const int32_t* offsets;
  int32_t tile_rows;
  const uint8_t* w_scales;     // [matrices][out][blocks]
  int64_t out, mats;
  uint8_t* w_ordered;
  int64_t x_blocks, w_parts;   // set by the launch: blocks of the first job, runs of parts
};
int64_t mx_prepare_blocks(int64_t rows, int64_t in, int64_t out, int64_t mats);
cudaError_t launch_mx_prepare(int32_t dtype, const MxPrepare& q, cudaStream_t s);

// y = act(x W + b) + r of microscaled operands, rows in expert order if experts > 0.
struct MxProduct {
  int32_t dtype, act, experts, tile_rows;
  const int32_t* offsets;
  int64_t rows, in, out;
  const void* x;               // mx_own_rows: as they are
  int64_t x_stride;
  const uint8_t* x_values;     // else [rows][blocks][16]
  const uint8_t* x_scales;     // and in order
  const uint8_t* w_values;     // [matrices][out][blocks][16]
  const uint8_t* w_scales;     // mx_own_rows: [out][blocks]; else in order
  const void* bias;
  const void* residual;
  int64_t r_stride;
  void* y;
  int* err;
};
// Rows so few that the product rounds them itself, without launch_mx_prepare (one token,
// 4096 -> 12288: 10.4 us, 12.2 with it, and 15 against 20 of host time).
inline bool mx_own_rows(int64_t rows, int32_t experts) { return !experts && rows <= 16; }
cudaError_t launch_mx_linear(const MxProduct& p, cudaStream_t s);

}  // namespace muon
