// Layer norm: launches and type dispatch (kernels in rows.cuh).
#include "rows_launch.h"

namespace twell {
namespace {

template <class TI, class TO>
cudaError_t norm(const LayerNormParams& p, bool vec, int sms, cudaStream_t s) {
  const RowShape r = row_shape(p.M, p.D, sms);
  uint32_t begin = 0, end = p.M;
  rows_inside(p.x, p.ldx, p.M, p.D, p.x_type, begin, end);
  void (*kern)(const LayerNormParams, const RowPlan) = nullptr;
#define TW_NG(n) \
  case n:        \
    kern = vec ? layer_norm_kernel<TI, TO, n, true> : layer_norm_kernel<TI, TO, n, false>; \
    break;
  switch (r.layers) { TW_NG(1) TW_NG(2) TW_NG(4) TW_NG(8) TW_NG(12) TW_NG(16) TW_NG(20) }
#undef TW_NG
  return launch_rows(kern, p, r, row_slot_bytes(p.D * sizeof(TI)),
                     2 * 4 * 4 * r.layers * 32 * r.warps, begin, end, sms, s);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormParams& p, int sms, cudaStream_t s) {
  const bool vec = p.D % 4 == 0 && quads(p.x, p.ldx, p.x_type) && quads(p.y, p.ldy, p.y_type);
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

}  // namespace twell
