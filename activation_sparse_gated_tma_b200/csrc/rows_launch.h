// Launch shapes of the row kernels.
#pragma once

#include "launch.h"
#include "rows.cuh"

namespace twell {

using bf16 = __nv_bfloat16;

constexpr int64_t kSmShared = 220 * 1024;  // of an SM's 227 KB, for the dynamic shared memory of its blocks
constexpr int64_t kBlockFixed = 3 * 1024;  // of a block besides: static and reserved

inline bool aligned_rows(const void* p, int64_t ld_bytes, int to) {
  return (reinterpret_cast<uintptr_t>(p) % to) == 0 && ld_bytes % to == 0;
}
inline int type_size(int type) { return type == TWELL_F32 ? 4 : type == TWELL_I8 ? 1 : 2; }
// Whether a matrix's rows all start on four elements' common alignment (and,
// for the kernels' aligned form, consist of whole fours).
inline bool quads(const void* p, int64_t ld, int type) { return aligned_rows(p, ld * type_size(type), 4 * type_size(type)); }

// The rows of a matrix whose whole 16-byte pieces lie between its first and
// its last element: all but a few at either end, narrowed into [begin, end).
inline void rows_inside(const void* p, int64_t ld, int M, int D, int type, uint32_t& begin, uint32_t& end) {
  const uint64_t base = reinterpret_cast<uint64_t>(p), step = static_cast<uint64_t>(ld) * type_size(type);
  const uint64_t bytes = static_cast<uint64_t>(D) * type_size(type), last = base + (M - 1) * step + bytes;
  while (begin < end && ((base + begin * step) & ~uint64_t(15)) < base) ++begin;
  while (begin < end && ((base + (end - 1) * step + bytes + 15) & ~uint64_t(15)) > last) --end;
}

// Warps per row, layers per thread, rows (groups) per block, blocks.
struct RowShape {
  int warps, layers, groups, grid, per_sm;
  int threads() const { return 32 * warps * groups; }
};
inline int row_layers(int D, int warps) {
  const int n = (D + 128 * warps - 1) / (128 * warps);
  return n <= 2 ? n : (n + 3) / 4 * 4;
}
// One warp per row as long as its lanes hold it; more while twice as many
// warps would still find the rows too few to give every SM eight warps.
inline RowShape row_shape(int M, int D, int sms) {
  RowShape r;
  r.warps = 1;
  while (r.warps < kMaxGroupWarps && D > 128 * kMaxLayers * r.warps) r.warps *= 2;
  while (2 * r.warps <= kMaxGroupWarps && D > 256 * r.warps && static_cast<int64_t>(M) * 2 * r.warps <= 8 * sms) r.warps *= 2;
  r.layers = row_layers(D, r.warps);
  r.groups = kMaxGroups / r.warps;
  const int64_t each = (static_cast<int64_t>(M) + sms - 1) / sms;  // rows per SM
  if (r.groups > each) r.groups = static_cast<int>(each);
  r.per_sm = row_blocks(r.layers) * kRowThreads / r.threads();
  r.grid = 0;
  return r;
}

// The ring takes the shared memory of the block's share of an SM that its
// vectors leave, in slots of `slot_bytes` for each group, as many as the group
// has rows at most.
template <class P>
cudaError_t launch_rows(void (*kern)(const P, const RowPlan), const P& p, RowShape r, uint32_t slot_bytes,
                        uint32_t vector_bytes, uint32_t begin, uint32_t end, int sms, cudaStream_t s) {
  const int64_t need = (static_cast<int64_t>(p.M) + r.groups - 1) / r.groups;
  int64_t slots = 0;
  for (; r.per_sm >= 1; --r.per_sm) {
    const int64_t most = static_cast<int64_t>(sms) * r.per_sm;
    r.grid = static_cast<int>(need < most ? need : most);
    const int64_t rows = (need + r.grid - 1) / r.grid;  // of a group at most
    slots = (kSmShared / r.per_sm - kBlockFixed - vector_bytes) / (static_cast<int64_t>(slot_bytes) * r.groups);
    if (slots > kMaxSlots) slots = kMaxSlots;
    if (slots > rows) slots = rows;
    if (slots >= 2 || slots == rows) break;
  }
  if (r.per_sm < 1) r.per_sm = 1;
  if (slots < 1) slots = 1;
  const size_t smem = vector_bytes + static_cast<size_t>(slots) * slot_bytes * r.groups;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, r.grid, r.threads(), smem, s, p, RowPlan{r.warps, static_cast<int>(slots), slot_bytes, begin, end});
}

}  // namespace twell
