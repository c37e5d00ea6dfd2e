// Launches of the 8-bit integer products (int8_gemm.cuh) and how they are cut.
#include "int8_gemm.cuh"

#include "launch.h"

namespace twell {

// Tokens per tile: the smallest of 16, 32, 64, 128 that holds the batch (128
// for larger ones).  Reduction splits (a cluster, 1 to 8): as many as keep the
// CTAs within two per SM, each with at least two k blocks and none empty.
Int8Plan int8_plan(int M, int N, int K, bool gated, int sms) {
  Int8Plan plan;
  plan.token_tile = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  const int64_t tiles = static_cast<int64_t>((N + kI8ChannelTile - 1) / kI8ChannelTile) *
                        ((M + plan.token_tile - 1) / plan.token_tile);
  const int kb = (K + kI8BK - 1) / kI8BK;
  int s = gated && plan.token_tile == 128 ? 1 : 8;
  for (; s > 1; s /= 2) {
    const int per = (kb + s - 1) / s;
    if (tiles * s <= 2 * sms && per >= 2 && (kb + per - 1) / per == s) break;
  }
  plan.k_splits = s;
  return plan;
}

namespace {

template <int BT, bool GATED>
cudaError_t split(const CUtensorMap& tm_x, const CUtensorMap& tm_w, const CUtensorMap& tm_w2, const Int8GemmParams& p,
                  int splits, cudaStream_t s) {
  auto kern = int8_split_kernel<BT, GATED>;
  constexpr int smem = Int8SplitSmem<BT, GATED>::kTotal;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((p.N + kI8ChannelTile - 1) / kI8ChannelTile) * ((p.M + BT - 1) / BT);
  if (tiles * splits > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl_cluster(splits, kern, static_cast<int>(tiles * splits), 192, smem, s, tm_x, tm_w, tm_w2, p, splits);
}

template <bool GATED>
cudaError_t by_tile(const Int8Plan& plan, const CUtensorMap& tm_x, const CUtensorMap& tm_w, const CUtensorMap& tm_w2,
                    const Int8GemmParams& p, cudaStream_t s) {
  switch (plan.token_tile) {
    case 16: return split<16, GATED>(tm_x, tm_w, tm_w2, p, plan.k_splits, s);
    case 32: return split<32, GATED>(tm_x, tm_w, tm_w2, p, plan.k_splits, s);
    case 64: return split<64, GATED>(tm_x, tm_w, tm_w2, p, plan.k_splits, s);
    case 128: return split<128, GATED>(tm_x, tm_w, tm_w2, p, plan.k_splits, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_int8_gemm(const Int8Plan& plan, bool gated, const CUtensorMap& tm_x, const CUtensorMap& tm_w,
                             const CUtensorMap& tm_w2, const Int8GemmParams& p, cudaStream_t s) {
  return gated ? by_tile<true>(plan, tm_x, tm_w, tm_w2, p, s) : by_tile<false>(plan, tm_x, tm_w, tm_w2, p, s);
}

}  // namespace twell
