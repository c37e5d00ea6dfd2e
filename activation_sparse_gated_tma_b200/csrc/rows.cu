// Launches of the row kernels (rows.cuh): launch shapes and type dispatch.
#include "rows.cuh"

#include "launch.h"

namespace twell {
namespace {

// Warps per row and rows (groups) per block for rows of D elements held as
// `cpt` chunks of eight per thread: blocks of about eight warps.
struct RowShape {
  int warps, groups;
  int threads() const { return 32 * warps * groups; }
};
RowShape row_shape(int D, int cpt) {
  const int chunks = (D + 7) / 8;
  RowShape r;
  r.warps = (chunks + 32 * cpt - 1) / (32 * cpt);
  if (r.warps < 1) r.warps = 1;
  if (r.warps > kRowThreads / 32) r.warps = kRowThreads / 32;
  r.groups = r.warps >= kMaxGroups ? 1 : kMaxGroups / r.warps;
  return r;
}

// Blocks for M rows: as many as fill the SMs at `threads_per_sm` resident threads.
int row_grid(int M, const RowShape& r, int sms, int threads_per_sm) {
  const int64_t need = (static_cast<int64_t>(M) + r.groups - 1) / r.groups;
  const int per_sm = threads_per_sm / r.threads() > 1 ? threads_per_sm / r.threads() : 1;
  const int64_t most = static_cast<int64_t>(sms) * per_sm;
  return static_cast<int>(need < most ? need : most);
}

bool aligned(const void* p, int64_t ld_bytes, int to) {
  return (reinterpret_cast<uintptr_t>(p) % to) == 0 && ld_bytes % to == 0;
}
int64_t type_bytes(int type) { return type == TWELL_F32 ? 4 : type == TWELL_I8 ? 1 : 2; }

constexpr int kNormThreadsPerSm = 1024;
constexpr int kQuantThreadsPerSm = 2048;

// Chunks of eight per thread: the fewest with which at most kRowThreads threads hold a row.
int row_cpt(int D) { return D > 16 * kRowThreads ? 4 : D > 8 * kRowThreads ? 2 : 1; }

template <class TI, class TO>
cudaError_t norm(const LayerNormParams& p, bool vec, int sms, cudaStream_t s) {
  const int cpt = row_cpt(p.D);
  const RowShape r = row_shape(p.D, cpt);
  const int grid = row_grid(p.M, r, sms, kNormThreadsPerSm);
  auto kern = cpt == 1   ? (vec ? layer_norm_kernel<TI, TO, 1, true> : layer_norm_kernel<TI, TO, 1, false>)
              : cpt == 2 ? (vec ? layer_norm_kernel<TI, TO, 2, true> : layer_norm_kernel<TI, TO, 2, false>)
                         : (vec ? layer_norm_kernel<TI, TO, 4, true> : layer_norm_kernel<TI, TO, 4, false>);
  return launch_pdl(kern, grid, r.threads(), 0, s, p, r.warps);
}

template <class TX, class TDY>
cudaError_t norm_bwd(const LayerNormBwdParams& p, bool vec, int sms, cudaStream_t s) {
  const int cpt = row_cpt(p.D);
  const RowShape r = row_shape(p.D, cpt);
  const int grid = row_grid(p.M, r, sms, kNormThreadsPerSm);
  auto kern = cpt == 1   ? (vec ? layer_norm_bwd_kernel<TX, TDY, 1, true> : layer_norm_bwd_kernel<TX, TDY, 1, false>)
              : cpt == 2 ? (vec ? layer_norm_bwd_kernel<TX, TDY, 2, true> : layer_norm_bwd_kernel<TX, TDY, 2, false>)
                         : (vec ? layer_norm_bwd_kernel<TX, TDY, 4, true> : layer_norm_bwd_kernel<TX, TDY, 4, false>);
  return launch_pdl(kern, grid, r.threads(), 0, s, p, r.warps);
}

template <class TI>
cudaError_t quantize(const QuantizeParams& p, bool vec, int sms, cudaStream_t s) {
  const int cpt = row_cpt(p.K);
  const RowShape r = row_shape(p.K, cpt);
  const int grid = row_grid(p.M, r, sms, kQuantThreadsPerSm);
  auto kern = cpt == 1   ? (vec ? quantize_rows_kernel<TI, 1, true> : quantize_rows_kernel<TI, 1, false>)
              : cpt == 2 ? (vec ? quantize_rows_kernel<TI, 2, true> : quantize_rows_kernel<TI, 2, false>)
                         : (vec ? quantize_rows_kernel<TI, 4, true> : quantize_rows_kernel<TI, 4, false>);
  return launch_pdl(kern, grid, r.threads(), 0, s, p, r.warps);
}

}  // namespace

using bf16 = __nv_bfloat16;

cudaError_t launch_layer_norm(const LayerNormParams& p, int sms, cudaStream_t s) {
  const bool vec = aligned(p.x, p.ldx * type_bytes(p.x_type), 16) &&
                   aligned(p.y, p.ldy * type_bytes(p.y_type), p.y_type == TWELL_I8 ? 8 : 16);
  if (p.y_type == TWELL_I8) {
    if (p.x_type == TWELL_F32) return norm<float, int8_t>(p, vec, sms, s);
    if (p.x_type == TWELL_BF16) return norm<bf16, int8_t>(p, vec, sms, s);
    return norm<__half, int8_t>(p, vec, sms, s);
  }
  if (p.x_type == TWELL_F32) {
    if (p.y_type == TWELL_F32) return norm<float, float>(p, vec, sms, s);
    if (p.y_type == TWELL_BF16) return norm<float, bf16>(p, vec, sms, s);
    return norm<float, __half>(p, vec, sms, s);
  }
  if (p.x_type == TWELL_BF16)
    return p.y_type == TWELL_F32 ? norm<bf16, float>(p, vec, sms, s) : norm<bf16, bf16>(p, vec, sms, s);
  return p.y_type == TWELL_F32 ? norm<__half, float>(p, vec, sms, s) : norm<__half, __half>(p, vec, sms, s);
}

int layer_norm_bwd_parts(int M, int D, int sms) {
  const RowShape r = row_shape(D, row_cpt(D));
  const int64_t groups = static_cast<int64_t>(row_grid(M, r, sms, kNormThreadsPerSm)) * r.groups;
  return static_cast<int>(groups < M ? groups : M);
}

cudaError_t launch_layer_norm_bwd(const LayerNormBwdParams& p, int sms, cudaStream_t s) {
  const bool vec = aligned(p.x, p.ldx * type_bytes(p.x_type), 16) && aligned(p.dx, p.lddx * type_bytes(p.x_type), 16) &&
                   aligned(p.dy, p.lddy * type_bytes(p.dy_type), 16);
  if (p.x_type == TWELL_F32) {
    if (p.dy_type == TWELL_F32) return norm_bwd<float, float>(p, vec, sms, s);
    if (p.dy_type == TWELL_BF16) return norm_bwd<float, bf16>(p, vec, sms, s);
    return norm_bwd<float, __half>(p, vec, sms, s);
  }
  if (p.x_type == TWELL_BF16)
    return p.dy_type == TWELL_F32 ? norm_bwd<bf16, float>(p, vec, sms, s) : norm_bwd<bf16, bf16>(p, vec, sms, s);
  return p.dy_type == TWELL_F32 ? norm_bwd<__half, float>(p, vec, sms, s) : norm_bwd<__half, __half>(p, vec, sms, s);
}

cudaError_t launch_layer_norm_bwd_reduce(const LayerNormBwdParams& p, int parts, cudaStream_t s) {
  return launch_pdl(layer_norm_bwd_reduce_kernel, (2 * p.D + 31) / 32, 32 * kReduceWarps, 0, s,
                    static_cast<const float*>(p.partial), parts, p.D, p.dweight, p.dbias);
}

cudaError_t launch_quantize_rows(const QuantizeParams& p, int sms, cudaStream_t s) {
  const bool vec = aligned(p.x, p.ldx * type_bytes(p.type), 16) && aligned(p.y, p.ldy, 8);
  if (p.type == TWELL_F32) return quantize<float>(p, vec, sms, s);
  if (p.type == TWELL_BF16) return quantize<bf16>(p, vec, sms, s);
  return quantize<__half>(p, vec, sms, s);
}

cudaError_t launch_dequantize_rows(const QuantizeParams& p, int sms, cudaStream_t s) {
  const bool vec = aligned(p.x, p.ldx, 8) && aligned(p.y, p.ldy * type_bytes(p.type), 16);
  const int64_t blocks = (static_cast<int64_t>(p.M) * ((p.K + 7) / 8) + 255) / 256;
  const int grid = static_cast<int>(blocks < 8 * sms ? blocks : 8 * sms);
  if (p.type == TWELL_F32)
    return launch_pdl(vec ? dequantize_rows_kernel<float, true> : dequantize_rows_kernel<float, false>, grid, 256, 0, s, p);
  if (p.type == TWELL_BF16)
    return launch_pdl(vec ? dequantize_rows_kernel<bf16, true> : dequantize_rows_kernel<bf16, false>, grid, 256, 0, s, p);
  return launch_pdl(vec ? dequantize_rows_kernel<__half, true> : dequantize_rows_kernel<__half, false>, grid, 256, 0, s, p);
}

}  // namespace twell
