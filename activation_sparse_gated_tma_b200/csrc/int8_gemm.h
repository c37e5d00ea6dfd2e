// Launch interface of the 8-bit integer products (int8_gemm.cu).  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace twell {

constexpr int kI8BK = 128;            // int8 elements per 128-byte swizzle row
constexpr int kI8MaxK = 131071;       // 128 * 128 * K stays within a 32-bit sum
constexpr int kI8MaxRows = 0x7fffffff - 1024;  // M and N: tile counts and padded rows stay within 32 bits
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
  unsigned long long wait_limit_ns;  // of every wait for a barrier
  bool lost;                         // test: MMAs are given up on (a tile of a CTA, all but a pair's first tile)
};

// How a product is cut: CTA pairs on 256 x 256 tiles, or tiles of 128 channels
// by `token_tile` tokens whose reduction k_splits CTAs (a cluster) share.
struct Int8Plan {
  bool pairs;
  int token_tile;
  int k_splits;
};
// Whether a product can be cut as `plan` (no share of a reduction may be empty).
bool int8_can_cut(const Int8Plan& plan, int K, bool gated, int sms);
// aligned_rows: the output's rows start on 16 bytes.
Int8Plan int8_plan(int M, int N, int K, bool gated, bool aligned_rows, int sms);
// Rows of the boxes of the operands' tensor maps (all kI8BK wide).
inline int int8_token_box(const Int8Plan& plan) { return plan.pairs ? 128 : plan.token_tile; }
constexpr int kI8ChannelBox = 128;

cudaError_t launch_int8_gemm(const Int8Plan& plan, bool gated, const CUtensorMap& tm_x, const CUtensorMap& tm_w,
                             const CUtensorMap& tm_w2, const Int8GemmParams& p, int sms, cudaStream_t s);

}  // namespace twell
