// Layer norm's backward pass: launches and type dispatch (kernels in rows_bwd.cuh).
#include "rows_bwd.cuh"
#include "rows_launch.h"

namespace twell {
namespace {

// Sums `parts` partial rows of 2 D values: a block takes 32 columns with 16
// warps, each adding every 16th row, then the warps' sums in a fixed order.
constexpr int kReduceWarps = 16;
__global__ void __launch_bounds__(32 * kReduceWarps)
    layer_norm_bwd_reduce_kernel(const float* __restrict__ partial, int parts, int D, float* dweight, float* dbias) {
  __shared__ float sums[kReduceWarps][32];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.f;
  if (c < 2 * static_cast<int64_t>(D))
#pragma unroll 8
    for (int r = warp; r < parts; r += kReduceWarps) s += partial[static_cast<int64_t>(r) * 2 * D + c];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < 2 * static_cast<int64_t>(D)) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < kReduceWarps; ++k) s += sums[k][lane];
    if (c < D) {
      if (dweight) dweight[c] = s;
    } else if (dbias) {
      dbias[c - D] = s;
    }
  }
}

// Chunks a thread owns: the fewest of 1, 2, 4 with which kBwdThreads threads
// own a row; two rows at a time where one chunk of aligned rows leaves the
// registers for it (4099 x 2047, f16, unaligned: 39 us with two, 32 with one).
struct BwdShape {
  int chunks, warps, groups, rows, grid;
};
BwdShape bwd_shape(int M, int D, bool aligned, int sms) {
  BwdShape r;
  r.chunks = D <= 8 * kBwdThreads ? 1 : D <= 16 * kBwdThreads ? 2 : 4;
  r.rows = r.chunks == 1 && aligned ? 2 : 1;
  r.warps = (D + 256 * r.chunks - 1) / (256 * r.chunks);
  r.groups = r.warps < kMaxGroups ? kMaxGroups / r.warps : 1;
  const int64_t each = (static_cast<int64_t>(M) + static_cast<int64_t>(sms) * r.rows - 1) / (static_cast<int64_t>(sms) * r.rows);
  if (r.groups > each) r.groups = static_cast<int>(each);
  const int threads = 32 * r.warps * r.groups;
  const int resident = 65536 / bwd_registers(r.chunks);
  const int per_sm = resident / threads > 1 ? resident / threads : 1;
  const int64_t need = (static_cast<int64_t>(M) + r.groups * r.rows - 1) / (r.groups * r.rows);
  const int64_t most = static_cast<int64_t>(sms) * per_sm;
  r.grid = static_cast<int>(need < most ? need : most);
  return r;
}

template <class TX, class TDY>
cudaError_t norm_bwd(const LayerNormBwdParams& p, bool aligned, int sms, int& parts, cudaStream_t s) {
  const BwdShape r = bwd_shape(p.M, p.D, aligned, sms);
  parts = r.grid;
  BwdPlan plan{r.warps, 0, static_cast<uint32_t>(p.M)};
  rows_inside(p.x, p.ldx, p.M, p.D, p.x_type, plan.begin, plan.end);
  rows_inside(p.dy, p.lddy, p.M, p.D, p.dy_type, plan.begin, plan.end);
  auto kern = r.chunks == 1   ? (aligned ? layer_norm_bwd_kernel<TX, TDY, 1, 2, true> : layer_norm_bwd_kernel<TX, TDY, 1, 1, false>)
              : r.chunks == 2 ? (aligned ? layer_norm_bwd_kernel<TX, TDY, 2, 1, true> : layer_norm_bwd_kernel<TX, TDY, 2, 1, false>)
                              : (aligned ? layer_norm_bwd_kernel<TX, TDY, 4, 1, true> : layer_norm_bwd_kernel<TX, TDY, 4, 1, false>);
  const size_t smem = r.groups > 1 ? static_cast<size_t>(r.groups) * 2 * p.D * sizeof(float) : 0;  // 16 KB at most
  return launch_pdl(kern, r.grid, 32 * r.warps * r.groups, smem, s, p, plan);
}

}  // namespace

int layer_norm_bwd_max_parts(int M, int D, int sms) {
  const int a = bwd_shape(M, D, true, sms).grid, b = bwd_shape(M, D, false, sms).grid;
  return a > b ? a : b;
}

cudaError_t launch_layer_norm_bwd(const LayerNormBwdParams& p, int sms, int& parts, cudaStream_t s) {
  const bool vec = p.D % 8 == 0 && chunk_rows(p.x, p.ldx, p.x_type) && chunk_rows(p.dx, p.lddx, p.x_type) &&
                   chunk_rows(p.dy, p.lddy, p.dy_type);
  if (p.x_type == TWELL_F32) {
    if (p.dy_type == TWELL_F32) return norm_bwd<float, float>(p, vec, sms, parts, s);
    if (p.dy_type == TWELL_BF16) return norm_bwd<float, bf16>(p, vec, sms, parts, s);
    return norm_bwd<float, __half>(p, vec, sms, parts, s);
  }
  if (p.x_type == TWELL_BF16)
    return p.dy_type == TWELL_F32 ? norm_bwd<bf16, float>(p, vec, sms, parts, s)
                                  : norm_bwd<bf16, bf16>(p, vec, sms, parts, s);
  return p.dy_type == TWELL_F32 ? norm_bwd<__half, float>(p, vec, sms, parts, s)
                                : norm_bwd<__half, __half>(p, vec, sms, parts, s);
}

cudaError_t launch_layer_norm_bwd_reduce(const LayerNormBwdParams& p, int parts, cudaStream_t s) {
  return launch_pdl(layer_norm_bwd_reduce_kernel, (2 * p.D + 31) / 32, 32 * kReduceWarps, 0, s,
                    static_cast<const float*>(p.partial), parts, p.D, p.dweight, p.dbias);
}

}  // namespace twell
