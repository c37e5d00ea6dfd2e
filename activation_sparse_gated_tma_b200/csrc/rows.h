// Launch interface of the row kernels (rows.cu): layer norm, its backward
// pass, row quantisation to int8 and back.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace twell {

constexpr int kLayerNormMaxD = 16384;  // a row stays in the registers of at most 512 threads, 32 elements each

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
  float eps;
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
  int dy_type, x_type, w_type;
};
// Row groups that write a partial sum each (a function of the sizes and the SM count only).
int layer_norm_bwd_parts(int M, int D, int sms);
cudaError_t launch_layer_norm_bwd(const LayerNormBwdParams& p, int sms, cudaStream_t s);
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
