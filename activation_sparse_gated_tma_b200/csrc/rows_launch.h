// Launch shapes of the row kernels.
#pragma once

#include "launch.h"
#include "rows.cuh"

namespace twell {

using bf16 = __nv_bfloat16;

inline bool aligned_rows(const void* p, int64_t ld_bytes, int to) {
  return (reinterpret_cast<uintptr_t>(p) % to) == 0 && ld_bytes % to == 0;
}
inline int type_size(int type) { return type == TWELL_F32 ? 4 : type == TWELL_I8 ? 1 : 2; }
// Whether a matrix's rows all start on the size of eight elements (32 bytes of fp32, 16, 8 of int8).
inline bool chunk_rows(const void* p, int64_t ld, int type) { return aligned_rows(p, ld * type_size(type), 8 * type_size(type)); }

// The rows of a matrix whose whole pieces (of `piece` bytes) lie between its first and
// its last element: all but a few at either end, narrowed into [begin, end).
inline void rows_inside(const void* p, int64_t ld, int M, int D, int type, uint32_t& begin, uint32_t& end,
                        uint64_t piece = 16) {
  const uint64_t base = reinterpret_cast<uint64_t>(p), step = static_cast<uint64_t>(ld) * type_size(type);
  const uint64_t bytes = static_cast<uint64_t>(D) * type_size(type), last = base + (M - 1) * step + bytes;
  while (begin < end && ((base + begin * step) & ~(piece - 1)) < base) ++begin;
  while (begin < end && ((base + (end - 1) * step + bytes + piece - 1) & ~(piece - 1)) > last) --end;
}

// A kernel's limit of dynamic shared memory: `most` is the most that any call of
// it takes, not what this one does.  The limit belongs to the kernel, and a lower
// one set by another host thread before this one's launch would refuse the launch.
template <class Kernel>
cudaError_t allow_shared(Kernel kern, int most) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

// Warps per row, chunks per thread, rows (groups) per block.
struct RowShape {
  int warps, chunks, groups;
  int threads() const { return 32 * warps * groups; }
};
// The fewest warps per row whose lanes hold it in `most` chunks each; more
// while twice as many warps leave every SM no more than `few` of them. A row's
// warps meet at a barrier, so the norm, with two sums to join, gains from more
// warps up to 8 an SM (bf16 1000 x 2560: 8.3 us; with 32 it took 9.3 where 8 took
// 8.1) and the quantisation, with one maximum, up to 32 (1000 x 2560: 4.3 us
// against 5.7 with 8, and 2.9 since).
inline RowShape row_shape(int M, int D, int most, int few, int sms) {
  RowShape r;
  r.warps = 1;
  while (r.warps < kMaxGroupWarps && D > 256 * most * r.warps) r.warps *= 2;
  while (2 * r.warps <= kMaxGroupWarps && D > 256 * r.warps && static_cast<int64_t>(M) * 2 * r.warps <= few * sms) r.warps *= 2;
  const int n = (D + 256 * r.warps - 1) / (256 * r.warps);
  r.chunks = n <= 6 ? n : (n + 1) / 2 * 2;
  r.groups = kMaxGroups / r.warps;
  const int64_t each = (static_cast<int64_t>(M) + sms - 1) / sms;  // rows per SM
  if (r.groups > each) r.groups = static_cast<int>(each);
  return r;
}
// Blocks: as many as share the SMs at `per_sm` of full size each.
inline int row_grid(int M, const RowShape& r, int per_sm, int sms) {
  const int64_t need = (static_cast<int64_t>(M) + r.groups - 1) / r.groups;
  const int64_t most = static_cast<int64_t>(sms) * (per_sm * kRowThreads / r.threads());
  return static_cast<int>(need < most ? need : most);
}

}  // namespace twell
