// Rows to int8 and back: launches and type dispatch (kernels in rows.cuh).
#include "rows_launch.h"

namespace twell {
namespace {

template <class TI>
cudaError_t quantize(const QuantizeParams& p, bool vec, int sms, cudaStream_t s) {
  if (p.K > kQuantizeMaxRow)
    return launch_pdl(quantize_long_rows_kernel<TI>, p.M < 4 * sms ? p.M : 4 * sms, kRowThreads, 0, s, p);
  const RowShape r = row_shape(p.M, p.K, sms);
  uint32_t begin = 0, end = p.M;
  rows_inside(p.x, p.ldx, p.M, p.K, p.type, begin, end);
  void (*kern)(const QuantizeParams, const RowPlan) = nullptr;
#define TW_NG(n) \
  case n:        \
    kern = vec ? quantize_rows_kernel<TI, n, true> : quantize_rows_kernel<TI, n, false>; \
    break;
  switch (r.layers) { TW_NG(1) TW_NG(2) TW_NG(4) TW_NG(8) TW_NG(12) TW_NG(16) TW_NG(20) }
#undef TW_NG
  return launch_rows(kern, p, r, row_slot_bytes(p.K * sizeof(TI)), 0, begin, end, sms, s);
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantizeParams& p, int sms, cudaStream_t s) {
  const bool vec = p.K % 4 == 0 && quads(p.x, p.ldx, p.type) && quads(p.y, p.ldy, TWELL_I8);
  if (p.type == TWELL_F32) return quantize<float>(p, vec, sms, s);
  if (p.type == TWELL_BF16) return quantize<bf16>(p, vec, sms, s);
  return quantize<__half>(p, vec, sms, s);
}

template <class TO>
static cudaError_t dequantize(const QuantizeParams& p, int sms, cudaStream_t s) {
  const bool q_aligned = quads(p.x, p.ldx, TWELL_I8), vec = p.K % 4 == 0 && quads(p.y, p.ldy, p.type);
  int across = 32;
  while (across < 256 && across * 16 < p.K) across *= 2;
  const int high = 256 / across;
  const int64_t need = (static_cast<int64_t>(p.M) + high - 1) / high;
  const int grid = static_cast<int>(need < 8 * sms ? need : 8 * sms);
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
