// Rows to int8 and back: launches and type dispatch (kernels in rows.cuh).
#include "rows_launch.h"

namespace twell {
namespace {

template <class TI>
cudaError_t quantize(const QuantizeParams& p, bool aligned, int sms, cudaStream_t s) {
  if (p.K > kQuantizeMaxRow)
    return launch_pdl(quantize_long_rows_kernel<TI>, p.M < 4 * sms ? p.M : 4 * sms, kRowThreads, 0, s, p);
  const RowShape r = row_shape(p.M, p.K, kQuantizeChunks, kQuantizeFewWarps, sms);
  RowPlan plan{r.warps, 0, static_cast<uint32_t>(p.M)};
  rows_inside(p.x, p.ldx, p.M, p.K, p.type, plan.begin, plan.end);
  void (*kern)(const QuantizeParams, const RowPlan) = nullptr;
#define TW_NC(n) \
  case n:        \
    kern = aligned ? quantize_rows_kernel<TI, n, true> : quantize_rows_kernel<TI, n, false>; \
    break;
  switch (r.chunks) { TW_NC(1) TW_NC(2) TW_NC(3) TW_NC(4) TW_NC(5) TW_NC(6) TW_NC(8) TW_NC(10) }
#undef TW_NC
  return launch_pdl(kern, row_grid(p.M, r, quantize_blocks(r.chunks, sizeof(TI)), sms), r.threads(), 0, s, p, plan);
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantizeParams& p, int sms, cudaStream_t s) {
  const bool vec = p.K % 8 == 0 && chunk_rows(p.x, p.ldx, p.type) && chunk_rows(p.y, p.ldy, TWELL_I8);
  if (p.type == TWELL_F32) return quantize<float>(p, vec, sms, s);
  if (p.type == TWELL_BF16) return quantize<bf16>(p, vec, sms, s);
  return quantize<__half>(p, vec, sms, s);
}

template <class TO>
static cudaError_t dequantize(const QuantizeParams& p, int sms, cudaStream_t s) {
  const bool q_aligned = chunk_rows(p.x, p.ldx, TWELL_I8);
  const bool vec = p.K % 8 == 0 && chunk_rows(p.y, p.ldy, p.type);
  // Threads along a row: the number that leaves the fewest of them idle in the last segment.
  const int chunks = (p.K + 7) / 8;
  int across = 256;
  for (int a = 128; a >= 32; a /= 2)
    if ((chunks + a - 1) / a * a < (chunks + across - 1) / across * across) across = a;
  const int segments = (chunks + across - 1) / across, rows = 4 * (256 / across);
  const int gx = segments < 16 * sms ? segments : 16 * sms;
  const int64_t need = (static_cast<int64_t>(p.M) + rows - 1) / rows, most = 16 * sms / gx;
  const dim3 grid(gx, static_cast<unsigned>(need < most ? need : most));
  auto kern = q_aligned ? (vec ? dequantize_rows_kernel<TO, true, true> : dequantize_rows_kernel<TO, true, false>)
                        : (vec ? dequantize_rows_kernel<TO, false, true> : dequantize_rows_kernel<TO, false, false>);
  return launch_pdl(kern, grid, 256, 0, s, p, across);
}

cudaError_t launch_dequantize_rows(const QuantizeParams& p, int sms, cudaStream_t s) {
  if (p.type == TWELL_F32) return dequantize<float>(p, sms, s);
  if (p.type == TWELL_BF16) return dequantize<bf16>(p, sms, s);
  return dequantize<__half>(p, sms, s);
}

}  // namespace twell
