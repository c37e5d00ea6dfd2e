// Launches of the 8-bit integer products (int8_gemm.cuh) and how they are cut.
#include "int8_gemm.cuh"

#include "launch.h"

namespace twell {

namespace {

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Estimated microseconds of a product cut as `plan`.  A wave of CTAs costs a
// start, its k blocks at the rate operands arrive (an SM takes 159 KB a
// microsecond, one CTA's ring half of that), a tail by columns, and for a
// shared reduction the exchange.  Constants fitted to 28 products timed in all
// their cuts on one B200 (M 1 to 4096, N 1535 to 10240, K 1536 to 10240, plain
// and gated, operands rotating through L2): the estimate is within 11% rms, and
// its choice is the fastest cut or within 3% of it for 25 of them, 27% at most.
// Two of them: M=300 N=5632 K=2048, tiles of 64 tokens 9.5 us (pairs 11.9,
// 128 tokens 11.7); M=1000 N=K=4096, pairs 17.6 us (64 tokens 28, 128 tokens 19.4).
double int8_cost(const Int8Plan& plan, int M, int N, int K, bool gated, bool aligned_rows, int sms) {
  const double kb = static_cast<double>(div_up(K, kI8BK));
  if (plan.pairs) {
    const int64_t tiles = div_up(M, 256) * div_up(N, gated ? 128 : 256);
    const double waves = static_cast<double>(div_up(tiles, sms / 2));
    // Gated tiles store by rows: elements, if those are unaligned.
    return 5.1 + waves * (0.311 * kb + 1.7 + (gated && !aligned_rows ? 14.0 : 0.0));
  }
  const int g = gated ? 2 : 1;
  const int64_t ctas = div_up(N, kI8ChannelTile) * div_up(M, plan.token_tile) * plan.k_splits;
  const double waves = static_cast<double>(div_up(ctas, 2 * sms));
  const double stage = 16.0 * g + plan.token_tile / 8.0;  // KB
  const double resident = static_cast<double>(ctas < 2 * sms ? ctas : 2 * sms) / sms;
  const double per_kb = stage * (resident / 159.0 > 1 / 72.0 ? resident / 159.0 : 1 / 72.0);
  double t = 2.8 + static_cast<double>(div_up(static_cast<int64_t>(kb), plan.k_splits)) * per_kb + 0.0193 * plan.token_tile * g;
  if (plan.k_splits > 1) t += 1.03 + 0.0168 * plan.token_tile * g;
  return waves * t;
}

}  // namespace

// (Gated tiles of 128 tokens have no room to share a reduction.)
bool int8_can_cut(const Int8Plan& plan, int K, bool gated, int sms) {
  if (plan.pairs) return sms >= 2;
  const int64_t kb = div_up(K, kI8BK);
  return div_up(kb, div_up(kb, plan.k_splits)) == plan.k_splits && !(gated && plan.token_tile == 128 && plan.k_splits > 1);
}

// The cut with the least estimated time: CTA pairs, or tiles of 16 to 128
// tokens (no more than hold the batch) with a reduction of 1 to 8 shares, none
// of them empty.
Int8Plan int8_plan(int M, int N, int K, bool gated, bool aligned_rows, int sms) {
  Int8Plan best{false, 16, 1};
  double least = int8_cost(best, M, N, K, gated, aligned_rows, sms);
  auto consider = [&](const Int8Plan& plan) {
    if (!int8_can_cut(plan, K, gated, sms)) return;
    const double t = int8_cost(plan, M, N, K, gated, aligned_rows, sms);
    if (t < least) {
      least = t;
      best = plan;
    }
  };
  for (int tile = 16; tile <= 128; tile *= 2) {
    if (tile > 16 && tile / 2 >= M) break;
    for (int s = 1; s <= 8; s *= 2) consider(Int8Plan{false, tile, s});
  }
  consider(Int8Plan{true, 128, 1});
  return best;
}

namespace {

template <int BT, bool GATED, class TY>
cudaError_t split(const CUtensorMap& tm_x, const CUtensorMap& tm_w, const CUtensorMap& tm_w2, const Int8GemmParams& p,
                  int splits, cudaStream_t s) {
  auto kern = int8_split_kernel<BT, GATED, TY>;
  constexpr int smem = Int8SplitSmem<BT, GATED>::kTotal;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((p.N + kI8ChannelTile - 1) / kI8ChannelTile) * ((p.M + BT - 1) / BT);
  if (tiles * splits > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl_cluster(splits, kern, static_cast<int>(tiles * splits), 192, smem, s, tm_x, tm_w, tm_w2, p, splits);
}

template <bool GATED, class TY>
cudaError_t by_tile(const Int8Plan& plan, const CUtensorMap& tm_x, const CUtensorMap& tm_w, const CUtensorMap& tm_w2,
                    const Int8GemmParams& p, cudaStream_t s) {
  switch (plan.token_tile) {
    case 16: return split<16, GATED, TY>(tm_x, tm_w, tm_w2, p, plan.k_splits, s);
    case 32: return split<32, GATED, TY>(tm_x, tm_w, tm_w2, p, plan.k_splits, s);
    case 64: return split<64, GATED, TY>(tm_x, tm_w, tm_w2, p, plan.k_splits, s);
    case 128: return split<128, GATED, TY>(tm_x, tm_w, tm_w2, p, plan.k_splits, s);
  }
  return cudaErrorInvalidValue;
}

template <bool GATED, class TY>
cudaError_t pair(const CUtensorMap& tm_x, const CUtensorMap& tm_w, const CUtensorMap& tm_w2, const Int8GemmParams& p,
                 int sms, cudaStream_t s) {
  auto kern = int8_pair_kernel<GATED, TY>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Int8PairSmem::kTotal);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((p.M + 255) / 256) * ((p.N + (GATED ? 127 : 255)) / (GATED ? 128 : 256));
  if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
  const int clusters = static_cast<int>(tiles < sms / 2 ? tiles : sms / 2);
  const CUtensorMap& a = GATED ? tm_x : tm_w;
  const CUtensorMap& b0 = GATED ? tm_w : tm_x;
  return launch_pdl_pair(kern, 2 * clusters, Int8PairSmem::kThreads, Int8PairSmem::kTotal, s, a, b0, tm_w2, p);
}

template <bool GATED, class TY>
cudaError_t by_plan(const Int8Plan& plan, const CUtensorMap& tm_x, const CUtensorMap& tm_w, const CUtensorMap& tm_w2,
                    const Int8GemmParams& p, int sms, cudaStream_t s) {
  return plan.pairs ? pair<GATED, TY>(tm_x, tm_w, tm_w2, p, sms, s) : by_tile<GATED, TY>(plan, tm_x, tm_w, tm_w2, p, s);
}

template <class TY>
cudaError_t by_form(bool gated, const Int8Plan& plan, const CUtensorMap& tm_x, const CUtensorMap& tm_w,
                    const CUtensorMap& tm_w2, const Int8GemmParams& p, int sms, cudaStream_t s) {
  return gated ? by_plan<true, TY>(plan, tm_x, tm_w, tm_w2, p, sms, s)
               : by_plan<false, TY>(plan, tm_x, tm_w, tm_w2, p, sms, s);
}

}  // namespace

cudaError_t launch_int8_gemm(const Int8Plan& plan, bool gated, const CUtensorMap& tm_x, const CUtensorMap& tm_w,
                             const CUtensorMap& tm_w2, const Int8GemmParams& p, int sms, cudaStream_t s) {
  if (p.y_type == TWELL_F32) return by_form<float>(gated, plan, tm_x, tm_w, tm_w2, p, sms, s);
  if (p.y_type == TWELL_BF16) return by_form<__nv_bfloat16>(gated, plan, tm_x, tm_w, tm_w2, p, sms, s);
  return by_form<__half>(gated, plan, tm_x, tm_w, tm_w2, p, sms, s);
}

}  // namespace twell
