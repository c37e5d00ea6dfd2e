// Launch interface of the 8-bit integer products (int8_gemm.cu).  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace twell {

constexpr int kI8BK = 128;            // int8 elements per 128-byte swizzle row
constexpr int kI8MaxK = 131071;       // 128 * 128 * K stays within a 32-bit sum
constexpr int kI8ChannelTile = 128;   // rows of a weight box

// y[m][n] = f(x_scale[m] w_scale[n] sum_k x[m][k] w[n][k]); plain: + bias[n];
// gated: u * max(g, 0) with g from w / w_scale and u from w2 / w2_scale.
struct Int8GemmParams {
  const float* x_scale;
  const float* w_scale;
  const float* w2_scale;  // gated only
  const float* bias;      // plain only, or NULL
  void* y;                // y_type, rows ldy elements apart
  int64_t ldy;
  int M, N, K;
  int y_type;
};

// How a product is cut: tokens per tile and CTAs (a cluster) that share a tile's reduction.
struct Int8Plan {
  int token_tile;
  int k_splits;
};
Int8Plan int8_plan(int M, int N, int K, bool gated, int sms);

// tm_x's box is token_tile rows, tm_w's and tm_w2's kI8ChannelTile rows, all kI8BK wide.
cudaError_t launch_int8_gemm(const Int8Plan& plan, bool gated, const CUtensorMap& tm_x, const CUtensorMap& tm_w,
                             const CUtensorMap& tm_w2, const Int8GemmParams& p, cudaStream_t s);

}  // namespace twell
