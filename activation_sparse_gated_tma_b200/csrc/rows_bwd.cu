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
#pragma unroll 16
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
// own a row (8 is none).
int bwd_chunks(int columns) {
  return columns <= 8 * kBwdThreads ? 1 : columns <= 16 * kBwdThreads ? 2 : columns <= 32 * kBwdThreads ? 4 : 8;
}
// Two rows at a time where one chunk (of rows not read by elements)
// leaves the registers for it.
struct BwdShape {
  int chunks, warps, groups, rows, grid;
};
// Warps whose registers an SM holds: each of its four parts has 16384 for every fourth warp.
constexpr int resident_warps(int registers) { return 4 * (16384 / (32 * registers)); }
BwdShape bwd_shape(int M, int D, BwdRows kind, int classes, int sms) {
  BwdShape r;
  const int columns = kind == kShifted ? D + 7 : D;
  r.chunks = bwd_chunks(columns);
  r.warps = (columns + 256 * r.chunks - 1) / (256 * r.chunks);
  r.rows = r.chunks == 1 && kind != kElements && 2 * r.warps <= resident_warps(bwd_registers(1, 2, kind == kShifted)) ? 2 : 1;
  // As many groups as an SM's registers take, in as few blocks as hold them: each block leaves a partial row.
  const int fit = resident_warps(bwd_registers(r.chunks, r.rows, kind == kShifted)) / r.warps;
  int per_sm = 1;
  r.groups = 1;
  for (int blocks = 1; blocks <= 4; ++blocks) {
    const int groups = fit / blocks < kMaxGroups ? fit / blocks : kMaxGroups;
    if (groups * blocks > r.groups * per_sm) {
      r.groups = groups;
      per_sm = blocks;
    }
  }
  const int64_t each = (static_cast<int64_t>(M) + static_cast<int64_t>(sms) * r.rows - 1) / (static_cast<int64_t>(sms) * r.rows);
  if (r.groups > each) r.groups = static_cast<int>(each);
  const int64_t of_class = (static_cast<int64_t>(M) + classes - 1) / classes;
  const int64_t need = (of_class + r.groups * r.rows - 1) / (r.groups * r.rows);
  const int64_t most = static_cast<int64_t>(sms) * per_sm / classes;
  r.grid = static_cast<int>(need < most ? need : most) * classes;
  return r;
}
// Rows after which the place where a row starts within a chunk repeats.
int shift_classes(int64_t ld) { return ld % 8 == 0 ? 1 : ld % 4 == 0 ? 2 : ld % 2 == 0 ? 4 : 8; }
int shift_of(const void* p, int type) { return static_cast<int>(reinterpret_cast<uint64_t>(p) / type_size(type) % 8); }

template <class TX, class TDY, BwdRows ROWS>
void (*bwd_kernel(int chunks, int rows))(const LayerNormBwdParams, const BwdPlan) {
  constexpr int kRows = ROWS == kElements ? 1 : 2;
  return rows == 2     ? layer_norm_bwd_kernel<TX, TDY, 1, kRows, ROWS>
         : chunks == 1 ? layer_norm_bwd_kernel<TX, TDY, 1, 1, ROWS>
         : chunks == 2 ? layer_norm_bwd_kernel<TX, TDY, 2, 1, ROWS>
                       : layer_norm_bwd_kernel<TX, TDY, 4, 1, ROWS>;
}

template <class TX, class TDY>
cudaError_t norm_bwd(const LayerNormBwdParams& p, bool aligned, int sms, int& parts, cudaStream_t s) {
  const int x0 = shift_of(p.x, p.x_type);
  // (With few rows those at the matrix's ends, read by elements, hold up the others: bf16 16 x 2047 7.0 us, by elements
  // 5.3; 300 x 1535 9.3 and 8.1, 1000 x 1535 11.4 and 13.5.  Where the shift takes a chunk more it does not pay:
  // fp32 8191 x 4093 102 us, by elements 90.)
  const bool shifted = !aligned && p.M > 4 * sms && bwd_chunks(p.D + 7) == bwd_chunks(p.D) &&
                       shift_of(p.dx, p.x_type) == x0 && shift_of(p.dy, p.dy_type) == x0 && p.lddx % 8 == p.ldx % 8 &&
                       p.lddy % 8 == p.ldx % 8;
  const BwdRows kind = aligned ? kAligned : shifted ? kShifted : kElements;
  const int classes = shifted ? shift_classes(p.ldx) : 1;
  const BwdShape r = bwd_shape(p.M, p.D, kind, classes, sms);
  parts = r.grid;
  BwdPlan plan{{r.warps, 0, static_cast<uint32_t>(p.M)}, static_cast<uint32_t>(classes)};
  rows_inside(p.x, p.ldx, p.M, p.D, p.x_type, plan.begin, plan.end, shifted ? 8 * sizeof(TX) : 16);
  rows_inside(p.dy, p.lddy, p.M, p.D, p.dy_type, plan.begin, plan.end, shifted ? 8 * sizeof(TDY) : 16);
  const auto kern = kind == kAligned   ? bwd_kernel<TX, TDY, kAligned>(r.chunks, r.rows)
                    : kind == kShifted ? bwd_kernel<TX, TDY, kShifted>(r.chunks, r.rows)
                                       : bwd_kernel<TX, TDY, kElements>(r.chunks, r.rows);
  const size_t smem = r.groups > 1 ? static_cast<size_t>(r.groups) * 2 * p.D * sizeof(float) : 0;
  if (smem > 40 * 1024) {  // up to 48 KB with the static part, no attribute is needed
    // groups * warps fit an SM, and a row has at most 256 columns a warp and chunk
    const int most = 2 * 256 * r.chunks * resident_warps(bwd_registers(r.chunks, r.rows, kind == kShifted)) * sizeof(float);
    const cudaError_t e = allow_shared(kern, most);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, r.grid, 32 * r.warps * r.groups, smem, s, p, plan);
}

}  // namespace

int layer_norm_bwd_max_parts(int M, int D, int sms) {
  int most = bwd_shape(M, D, kAligned, 1, sms).grid;
  const int elements = bwd_shape(M, D, kElements, 1, sms).grid;
  if (elements > most) most = elements;
  if (bwd_chunks(D + 7) == bwd_chunks(D))
    for (int classes = 1; classes <= 8; classes *= 2) {
      const int shifted = bwd_shape(M, D, kShifted, classes, sms).grid;
      if (shifted > most) most = shifted;
    }
  return most;
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
