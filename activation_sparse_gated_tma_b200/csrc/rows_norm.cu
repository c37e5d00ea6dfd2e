// Layer norm: launches and type dispatch (kernels in rows.cuh).
#include "rows_launch.h"

namespace twell {
namespace {

template <class TI, class TO>
cudaError_t norm(const LayerNormParams& p, bool aligned, int sms, cudaStream_t s) {
  const RowShape r = row_shape(p.M, p.D, aligned ? kNormChunks : norm_chunks_unaligned(p.M, sms), kNormFewWarps, sms);
  RowPlan plan{r.warps, 0, static_cast<uint32_t>(p.M)};
  rows_inside(p.x, p.ldx, p.M, p.D, p.x_type, plan.begin, plan.end);
  void (*kern)(const LayerNormParams, const RowPlan) = nullptr;
#define TW_NC(n) \
  case n:        \
    kern = aligned ? layer_norm_kernel<TI, TO, n, true> : layer_norm_kernel<TI, TO, n, false>; \
    break;
  switch (r.chunks) { TW_NC(1) TW_NC(2) TW_NC(3) TW_NC(4) TW_NC(5) TW_NC(6) TW_NC(8) TW_NC(10) }
#undef TW_NC
  // Weight and bias, 227 KB at most per SM.
  const int each = 2 * 4 * 8 * r.chunks * 32, vectors = each * r.warps;
  int per_sm = norm_blocks(r.chunks);
  while (per_sm > 1 && per_sm * (kRowThreads / r.threads()) * (vectors + 2048) > 220 * 1024) --per_sm;
  if (vectors > 40 * 1024) {  // up to 48 KB with the static part, no attribute is needed
    const cudaError_t e = allow_shared(kern, each * kMaxGroupWarps);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, row_grid(p.M, r, per_sm, sms), r.threads(), vectors, s, p, plan);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormParams& p, int sms, cudaStream_t s) {
  const bool vec = p.D % 8 == 0 && chunk_rows(p.x, p.ldx, p.x_type) && chunk_rows(p.y, p.ldy, p.y_type);
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
