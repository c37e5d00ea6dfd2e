// Launch interface of the row kernels (rows_*.cu): layer norm, its backward
// pass, row quantisation to int8 and back.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace twell {

constexpr int kRowThreads = 256;     // of a block at most
constexpr int kMaxGroups = 8;        // rows that a block works on at once
constexpr int kMaxGroupWarps = 8;    // of a row
constexpr int kNormChunks = 10;      // of eight elements that a thread holds at most
// Joining the pieces of unaligned rows wants more warps (bf16, 8191 x 1535: 30 us with 6 chunks, 25 with 5; 8191 x 4095:
// 66 with 8, 55), unless so all rows are at work at once (2047 x 1535: 7.3 us with 6, 8.1 with 5).
constexpr int norm_chunks_unaligned(int M, int sms) { return M <= 16 * sms ? 6 : 5; }
constexpr int kQuantizeChunks = 6;   // as long as kMaxGroupWarps warps hold the row so
constexpr int kNormFewWarps = 8;     // per SM, up to which a row is spread over more warps than hold it
constexpr int kQuantizeFewWarps = 32;
constexpr int kBwdThreads = 512;     // of a block at most, backward
constexpr int kLayerNormMaxD = 16384;
constexpr int kQuantizeMaxRow = 8 * kNormChunks * kRowThreads;  // longer rows are read twice

// Blocks that share an SM's registers.
constexpr int norm_blocks(int chunks) { return chunks <= 2 ? 4 : chunks <= 5 ? 3 : 2; }
constexpr int quantize_blocks(int chunks, int element) { return chunks * element <= 12 ? 4 : chunks * element <= 20 ? 3 : 2; }

// Registers of a thread, backward: chunks it holds of a row, rows at a time.  (Shifted rows take a warp more; with 72
// registers three groups of nine fit an SM: fp16 16384 x 2047 70 us, with 80 83.)
constexpr int bwd_registers(int chunks, int rows, bool shifted) { return chunks > 1 ? 128 : rows > 1 ? (shifted ? 72 : 80) : 64; }

// How a launch lays out rows over blocks (see rows.cuh): warps per row; rows
// [begin, end) are those whose aligned pieces lie inside the matrix.
struct RowPlan {
  int warps;
  uint32_t begin, end;
  __host__ __device__ bool whole_pieces(uint32_t row) const { return row >= begin && row < end; }
};
// Backward: shifted rows, `classes` of them by where a row starts (see rows_bwd.cuh).
struct BwdPlan : RowPlan {
  uint32_t classes;
};

// Rows are `ld` elements apart; a row's elements are contiguous.  Types are
// twell_dtype values; out_type TWELL_I8 writes quantised rows and y_scale.
struct LayerNormParams {
  const void* x;
  const void* weight;  // [D] of w_type, or NULL (ones)
  const void* bias;    // [D] of w_type, or NULL (zeros)
  void* y;
  float* y_scale;      // [M], int8 output only
  float* mean;         // [M] or NULL
  float* rstd;         // [M] or NULL
  int64_t ldx, ldy;
  int M, D;
  float eps, inv_d;    // inv_d: 1 / D
  int x_type, y_type, w_type;
};
cudaError_t launch_layer_norm(const LayerNormParams& p, int sms, cudaStream_t s);

struct LayerNormBwdParams {
  const void* dy;
  const void* x;
  const void* weight;  // or NULL
  const float* mean;
  const float* rstd;
  void* dx;            // x_type
  float* partial;      // [parts][2][D]; NULL: no parameter gradients
  float* dweight;      // [D] or NULL
  float* dbias;        // [D] or NULL
  int64_t lddy, ldx, lddx;
  int M, D;
  float inv_d;         // 1 / D
  int dy_type, x_type, w_type;
};
// Most partial rows of the parameter gradients that a call writes, for any alignment.
int layer_norm_bwd_max_parts(int M, int D, int sms);
// `parts`: the partial rows it writes.
cudaError_t launch_layer_norm_bwd(const LayerNormBwdParams& p, int sms, int& parts, cudaStream_t s);
cudaError_t launch_layer_norm_bwd_reduce(const LayerNormBwdParams& p, int parts, cudaStream_t s);

struct QuantizeParams {
  const void* x;   // quantize: x_type rows; dequantize: int8 rows
  void* y;         // quantize: int8 rows; dequantize: y_type rows
  float* scale;    // [M], written by quantize, read by dequantize
  int64_t ldx, ldy;
  int M, K;
  int type;        // the floating type of either side
};
cudaError_t launch_quantize_rows(const QuantizeParams& p, int sms, cudaStream_t s);
cudaError_t launch_dequantize_rows(const QuantizeParams& p, int sms, cudaStream_t s);

}  // namespace twell
