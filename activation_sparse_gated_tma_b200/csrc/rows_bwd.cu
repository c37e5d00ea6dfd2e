// Layer norm's backward pass: launches and type dispatch (kernels in rows.cuh).
#include "rows_bwd.cuh"
#include "rows_launch.h"

namespace twell {
namespace {

constexpr int64_t kSmShared = 220 * 1024;  // of an SM's 227 KB, for the dynamic shared memory of its blocks
constexpr int64_t kBlockFixed = 3 * 1024;  // of a block besides: static and reserved

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

// Layers of four columns a thread owns: the fewest of 2, 4, 8 with which kBwdThreads threads own a row.
int bwd_layers(int D) { return D <= 8 * kBwdThreads ? 2 : D <= 16 * kBwdThreads ? 4 : 8; }
int bwd_threads(int D) {
  const int span = 128 * bwd_layers(D);
  return (D + span - 1) / span * 32;
}
int bwd_blocks(int D) {
  const int threads = bwd_layers(D) == 2 ? 1024 : 512;  // what the registers allow an SM
  const int blocks = threads / bwd_threads(D);
  return blocks < 1 ? 1 : blocks > 8 ? 8 : blocks;
}

template <class TX, class TDY>
cudaError_t norm_bwd(const LayerNormBwdParams& p, bool vec, int sms, int& parts, cudaStream_t s) {
  const int layers = bwd_layers(p.D), threads = bwd_threads(p.D), warps = threads / 32;
  const int64_t row = row_slot_bytes(p.D * sizeof(TX)) + row_slot_bytes(p.D * sizeof(TDY));
  const int64_t vector = 4 * 4 * layers * threads;
  // Blocks per SM and rows per batch: the most blocks with which two batches
  // of two rows fit (else one block), batches as large as two of them fit.
  int per_sm = bwd_blocks(p.D);
  auto room = [&](int n) { return kSmShared / n - kBlockFixed - vector; };
  while (per_sm > 1 && room(per_sm) < 4 * row) --per_sm;
  int rows = static_cast<int>(room(per_sm) / (2 * row));
  if (rows > kMaxBatch) rows = kMaxBatch;
  // Few rows: batches small enough to occupy every block.
  const int64_t spread = (static_cast<int64_t>(p.M) + static_cast<int64_t>(sms) * per_sm - 1) / (static_cast<int64_t>(sms) * per_sm);
  if (rows > spread) rows = static_cast<int>(spread);
  if (rows < 1) rows = 1;
  // Whole numbers of warps per row, if a slightly smaller batch has one.
  for (int k = rows; k > rows / 2; --k)
    if (warps % k == 0) {
      rows = k;
      break;
    }
  BatchPlan plan;
  plan.rows = rows;
  plan.batches = (static_cast<uint32_t>(p.M) + rows - 1) / rows;
  const int64_t most = static_cast<int64_t>(sms) * per_sm;
  const int grid = static_cast<int>(plan.batches < most ? plan.batches : most);
  const int64_t each = (plan.batches + grid - 1) / grid;
  int64_t slots = room(per_sm) / (rows * row);
  if (slots > 4) slots = 4;
  if (slots > each) slots = each;
  plan.slots = static_cast<int>(slots < 1 ? 1 : slots);
  plan.ring_begin = 0;
  plan.ring_end = p.M;
  rows_inside(p.x, p.ldx, p.M, p.D, p.x_type, plan.ring_begin, plan.ring_end);
  rows_inside(p.dy, p.lddy, p.M, p.D, p.dy_type, plan.ring_begin, plan.ring_end);
  const size_t smem = static_cast<size_t>(vector + plan.slots * rows * row);
  auto kern = layers == 2   ? (vec ? layer_norm_bwd_kernel<TX, TDY, 2, true> : layer_norm_bwd_kernel<TX, TDY, 2, false>)
              : layers == 4 ? (vec ? layer_norm_bwd_kernel<TX, TDY, 4, true> : layer_norm_bwd_kernel<TX, TDY, 4, false>)
                            : (vec ? layer_norm_bwd_kernel<TX, TDY, 8, true> : layer_norm_bwd_kernel<TX, TDY, 8, false>);
  parts = grid;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, grid, threads, smem, s, p, plan);
}

}  // namespace

int layer_norm_bwd_max_parts(int M, int D, int sms) {
  const int64_t most = static_cast<int64_t>(sms) * bwd_blocks(D);
  return static_cast<int>(M < most ? M : most);
}

cudaError_t launch_layer_norm_bwd(const LayerNormBwdParams& p, int sms, int& parts, cudaStream_t s) {
  const bool vec = p.D % 4 == 0 && aligned_rows(p.x, p.ldx * type_size(p.x_type), 16) &&
                   aligned_rows(p.dx, p.lddx * type_size(p.x_type), 16) &&
                   aligned_rows(p.dy, p.lddy * type_size(p.dy_type), 16);
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
