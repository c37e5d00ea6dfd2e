// Layer norm's backward pass.  With xh = (x - mu) r and g = dy w:
//   dx = r (g - (sum g + xh sum g xh) / D),   dw = sum_rows dy xh,   db = sum_rows dy.
// dw and db want a thread to keep its columns over many rows, so a row belongs
// to a group of as many warps as it takes (a thread holds NC chunks of eight
// columns), and what a row costs beyond its columns is shared by R rows at a time
// (two where the registers allow): their 2 R sums go through one exchange and one barrier.  x and dy are
// read straight into registers, several rows' worth of bytes in flight per SM.
// Bound by HBM for fp32 rows: 16384 x 2560 takes 85 us (5.9 TB/s; batches of
// rows through a shared-memory ring and two passes over each took 93).  Of
// 16-bit rows (bf16 x, fp32 dy: 70 us) a row's chain of load, exchange and store
// takes as long as its bytes: halving the fp32 instructions (two values each)
// changed nothing.
// Rows are dealt to groups in a fixed way, so the order of every sum depends on
// the sizes alone.  A block adds its groups' dw and db and writes one partial
// row; a second kernel adds those.
#pragma once

#include "rows.cuh"

namespace twell {

constexpr int kBwdWarps = kBwdThreads / 32;

struct BwdShared {
  float part[kMaxGroups][2][kBwdWarps][4];  // per group, exchange buffer, warp: 2 R sums
};

// Sums 2 R values per thread over the group; every thread gets all of them.
// Halving exchange: at each step a lane keeps half of the values and hands the
// other half to its partner, so 2 R values take 2 R + 2 shuffles instead of 10 R.
template <int R>
__device__ __forceinline__ void group_sums(const Group& g, int flip, BwdShared& sh, float (&v)[2 * R]) {
  constexpr int kValues = 2 * R;
  constexpr int kStep = 32 / kValues;  // lanes that end up with the same value
  const int lane = g.t & 31;
#pragma unroll
  for (int n = kValues / 2, o = 16; n >= 1; n /= 2, o /= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float keep = upper ? v[k + n] : v[k], give = upper ? v[k] : v[k + n];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  float s = v[0];
#pragma unroll
  for (int o = kStep / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  // Lane l has value l / kStep of this warp.
  if (g.warps > 1) {
    if (lane % kStep == 0) sh.part[g.id][flip][g.t >> 5][lane / kStep] = s;
    named_bar_sync(1 + g.id, g.nt);
    s = 0.f;
    for (int w = lane % kStep; w < g.warps; w += kStep) s += sh.part[g.id][flip][w][lane / kStep];
#pragma unroll
    for (int o = kStep / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  }
#pragma unroll
  for (int k = 0; k < kValues; ++k) v[k] = __shfl_sync(0xffffffffu, s, k * kStep);
}

// Where a thread's columns lie.
//   kAligned   rows of whole chunks that start on one: chunks t, t + T, ...
//   kShifted   rows of x, dy and dx that all start the same number of elements,
//              0 <= s < 8, behind a chunk's boundary: the chunks from that
//              boundary on, the first and last of a row in part.  s repeats with
//              every `classes` rows (8 for an odd row stride), and a block takes
//              rows of one class only, so its threads keep their columns.
//   kElements  any others: every T-th column, neighbouring lanes on neighbouring ones
// (fp16, 4099 x 2047: shifted 25 us, by elements 32, chunks joined from two pieces 39.)
enum BwdRows { kAligned, kShifted, kElements };
template <BwdRows ROWS>
__device__ __forceinline__ int bwd_column(int t, int nt, int s, int j, int i) {
  return ROWS == kElements ? (8 * j + i) * nt + t : 8 * (t + j * nt) - (ROWS == kShifted ? s : 0) + i;
}
__device__ __forceinline__ bool in_row(int c, int D) { return static_cast<unsigned>(c) < static_cast<unsigned>(D); }
template <class T, BwdRows ROWS>
using BwdLayer = typename std::conditional<ROWS == kElements, Oct, Chunk<T>>::type;
__device__ __forceinline__ Oct unpack8(const Oct& v) { return v; }
// (kShifted: chunks at either end of the row are read whole and cleared later,
// by clear_ends, so that no load waits for another, unless one would reach
// outside the matrix.)
template <class T, int NC, BwdRows ROWS>
__device__ __forceinline__ void load_bwd(const T* row, bool whole, int D, int t, int nt, int s, BwdLayer<T, ROWS> (&v)[NC]) {
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = bwd_column<ROWS>(t, nt, s, j, 0);
    if constexpr (ROWS == kAligned) {
      v[j] = load_chunk<T, true, false>(row, 0, c, D);
    } else if constexpr (ROWS == kShifted) {
      v[j] = {};
      if (whole ? c < D : c >= 0 && c + 8 <= D) {
        v[j] = load_whole(row + c);
      } else if (!whole) {
        union { Chunk<T> c; T e[8]; } u;
        u.c = {};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (in_row(c + i, D)) u.e[i] = row[c + i];
        v[j] = u.c;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j].e[i] = c + i * nt < D ? to_f32(row[c + i * nt]) : 0.f;
    }
  }
}
template <class T>
__device__ __forceinline__ void clear_ends(Chunk<T>& v, int c, int D) {
  union { Chunk<T> c; T e[8]; } u;
  u.c = v;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (!in_row(c + i, D)) u.e[i] = from_f32<T>(0.f);
  v = u.c;
}
template <class T, BwdRows ROWS>
__device__ __forceinline__ void store_bwd(T* row, int D, int t, int nt, int s, int j, const Oct& o) {
  const int c = bwd_column<ROWS>(t, nt, s, j, 0);
  if constexpr (ROWS == kAligned) {
    store_chunk<T, true, false>(row, 0, c, D, pack8<T>(o));
  } else if constexpr (ROWS == kShifted) {
    if (c >= 0 && c + 8 <= D) {
      store_whole(row + c, pack8<T>(o));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (in_row(c + i, D)) row[c + i] = from_f32<T>(o.e[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i * nt < D) row[c + i * nt] = from_f32<T>(o.e[i]);
  }
}

template <class TX, class TDY, int NC, int R, BwdRows ROWS>
__global__ void __maxnreg__(bwd_registers(NC, R, ROWS == kShifted))
    layer_norm_bwd_kernel(const LayerNormBwdParams p, const BwdPlan plan) {
  extern __shared__ __align__(16) float sums[];  // [groups][2][D], only with more than one group
  __shared__ BwdShared sh;
  Group g;
  g.warps = plan.warps;
  g.nt = 32 * plan.warps;
  g.id = static_cast<int>(threadIdx.x) / g.nt;
  g.t = static_cast<int>(threadIdx.x) - g.id * g.nt;
  const int groups = static_cast<int>(blockDim.x) / g.nt;
  int flip = 0;
  griddep_launch_dependents();
  griddep_wait();

  // Rows cls, cls + classes, ...; all with the shift of the first.
  const uint32_t classes = ROWS == kShifted ? plan.classes : 1, cls = ROWS == kShifted ? blockIdx.x % classes : 0;
  const uint32_t rows = cls < p.M ? (p.M - cls + classes - 1) / classes : 0;
  const int s = ROWS == kShifted
                    ? static_cast<int>(reinterpret_cast<uint64_t>(static_cast<const TX*>(p.x) + cls * p.ldx) / sizeof(TX) % 8)
                    : 0;
  Oct w[NC], dw[NC], db[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = bwd_column<ROWS>(g.t, g.nt, s, j, i);
      float e = 0.f;
      if (in_row(c, p.D))
        e = !p.weight                ? 1.f
            : p.w_type == TWELL_F32  ? static_cast<const float*>(p.weight)[c]
            : p.w_type == TWELL_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(p.weight)[c])
                                     : to_f32(static_cast<const __half*>(p.weight)[c]);
      w[j].e[i] = e;
      dw[j].e[i] = db[j].e[i] = 0.f;
    }
  const uint32_t step = gridDim.x / classes * groups * R;
  for (uint32_t at = (blockIdx.x / classes * groups + g.id) * R; at < rows; at += step) {
    auto row_at = [&](uint32_t i) { return cls + classes * (at + i); };
    BwdLayer<TX, ROWS> x[R][NC];
    BwdLayer<TDY, ROWS> dy[R][NC];
    float mean[R], rstd[R], sum[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (at + r < rows) {
        const uint32_t row = row_at(r);
        load_bwd<TX, NC, ROWS>(static_cast<const TX*>(p.x) + row * p.ldx, plan.whole_pieces(row), p.D, g.t, g.nt, s, x[r]);
        load_bwd<TDY, NC, ROWS>(static_cast<const TDY*>(p.dy) + row * p.lddy, plan.whole_pieces(row), p.D, g.t, g.nt, s, dy[r]);
        mean[r] = p.mean[row];
        rstd[r] = p.rstd[row];
      } else {
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          x[r][j] = {};
          dy[r][j] = {};
        }
        mean[r] = rstd[r] = 0.f;
      }
    }
    if (g.t < 2 * R) {
      const uint32_t i = step + (g.t >> 1), row = row_at(i);
      if (at + i < rows && plan.whole_pieces(row)) {
        if (g.t & 1)
          prefetch_row(static_cast<const TDY*>(p.dy) + row * p.lddy, p.D);
        else
          prefetch_row(static_cast<const TX*>(p.x) + row * p.ldx, p.D);
      }
    }
    if constexpr (ROWS == kShifted) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int c = bwd_column<ROWS>(g.t, g.nt, s, j, 0);
        if (c < 0 || c + 8 > p.D) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            clear_ends(x[r][j], c, p.D);
            clear_ends(dy[r][j], c, p.D);
          }
        }
      }
    }
    // Outside the row x and dy are 0, so nothing is added there: 0 times 0 - mean.  (The sum of g xh takes its rstd
    // afterwards.  (0 - mean) rstd may pass the fp32 range where all of the row is far from zero, and 0 times that is
    // NaN; so may the sum before rstd where the squared deviations did and left an rstd of 0.)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float a[2] = {0.f, 0.f}, b[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const Oct xv = unpack8(x[r][j]), dv = unpack8(dy[r][j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float off = xv.e[i] - mean[r], gr = dv.e[i] * w[j].e[i];
          dw[j].e[i] = fmaf(dv.e[i], off * rstd[r], dw[j].e[i]);
          db[j].e[i] += dv.e[i];
          a[i & 1] += gr;
          b[i & 1] = fmaf(gr, off, b[i & 1]);
        }
      }
      sum[2 * r] = a[0] + a[1];
      sum[2 * r + 1] = rstd[r] == 0.f ? 0.f : (b[0] + b[1]) * rstd[r];
    }
    group_sums<R>(g, flip, sh, sum);
    flip ^= 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (at + r >= rows) break;
      // dx = r g - r sum g / D - xh r sum g xh / D
      const float c1 = -rstd[r] * (sum[2 * r] * p.inv_d), c2 = -rstd[r] * (sum[2 * r + 1] * p.inv_d);
      TX* dx = static_cast<TX*>(p.dx) + row_at(r) * p.lddx;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const Oct xv = unpack8(x[r][j]), dv = unpack8(dy[r][j]);
        Oct o;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o.e[i] = fmaf((xv.e[i] - mean[r]) * rstd[r], c2, fmaf(dv.e[i] * w[j].e[i], rstd[r], c1));
        store_bwd<TX, ROWS>(dx, p.D, g.t, g.nt, s, j, o);
      }
    }
  }
  if (!p.partial) return;
  float* out = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
  float* to = groups > 1 ? sums + static_cast<int64_t>(g.id) * 2 * p.D : out;
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = bwd_column<ROWS>(g.t, g.nt, s, j, i);
      if (in_row(c, p.D)) {
        to[c] = dw[j].e[i];
        to[p.D + c] = db[j].e[i];
      }
    }
  if (groups > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.D; c += blockDim.x) {
      float v = sums[c];
      for (int k = 1; k < groups; ++k) v += sums[k * 2 * p.D + c];
      out[c] = v;
    }
  }
}

}  // namespace twell
