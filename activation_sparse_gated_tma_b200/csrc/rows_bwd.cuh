// Layer norm's backward pass.  With xh = (x - mu) r and g = dy w:
//   dx = r (g - (sum g + xh sum g xh) / D),   dw = sum_rows dy xh,   db = sum_rows dy.
// dw and db want a thread to keep its columns over many rows, so a row belongs
// to a group of as many warps as it takes (a thread holds NC chunks of eight
// columns), and what a row costs beyond its columns is shared by R rows at a time
// (two of aligned rows): their 2 R sums go through one exchange and one barrier.  x and dy are
// read straight into registers, several rows' worth of bytes in flight per SM.
// Bound by HBM for fp32 rows: 16384 x 2560 takes 84 us (6.0 TB/s; batches of
// rows through a shared-memory ring and two passes over each took 93).  Of
// 16-bit rows (bf16 x, fp32 dy: 69 us) a row's chain of load, exchange and store
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

// Columns of a thread: eight neighbouring ones of aligned rows; of others every
// T-th, read and written by elements, neighbouring lanes on neighbouring ones.
template <bool ALIGNED>
__device__ __forceinline__ int bwd_column(int t, int nt, int j, int i) {
  return ALIGNED ? 8 * (t + j * nt) + i : (8 * j + i) * nt + t;
}
template <class T, bool ALIGNED>
using BwdLayer = typename std::conditional<ALIGNED, Chunk<T>, Oct>::type;
__device__ __forceinline__ Oct unpack8(const Oct& v) { return v; }
template <class T, int NC, bool ALIGNED>
__device__ __forceinline__ void load_bwd(const T* row, int D, int t, int nt, BwdLayer<T, ALIGNED> (&v)[NC]) {
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    if constexpr (ALIGNED) {
      v[j] = load_chunk<T, true, false>(row, 0, 8 * (t + j * nt), D);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j].e[i] = bwd_column<false>(t, nt, j, i) < D ? to_f32(row[bwd_column<false>(t, nt, j, i)]) : 0.f;
    }
  }
}
template <class T, bool ALIGNED>
__device__ __forceinline__ void store_bwd(T* row, int D, int t, int nt, int j, const Oct& o) {
  if constexpr (ALIGNED) {
    store_chunk<T, true, false>(row, 0, 8 * (t + j * nt), D, pack8<T>(o));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (bwd_column<false>(t, nt, j, i) < D) row[bwd_column<false>(t, nt, j, i)] = from_f32<T>(o.e[i]);
  }
}

template <class TX, class TDY, int NC, int R, bool ALIGNED>
__global__ void __maxnreg__(bwd_registers(NC))
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

  Oct w[NC], dw[NC], db[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = bwd_column<ALIGNED>(g.t, g.nt, j, i);
      float e = 0.f;
      if (c < p.D)
        e = !p.weight                ? 1.f
            : p.w_type == TWELL_F32  ? static_cast<const float*>(p.weight)[c]
            : p.w_type == TWELL_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(p.weight)[c])
                                     : to_f32(static_cast<const __half*>(p.weight)[c]);
      w[j].e[i] = e;
      dw[j].e[i] = db[j].e[i] = 0.f;
    }
  const uint32_t step = gridDim.x * groups * R;
  for (uint32_t row0 = (blockIdx.x * groups + g.id) * R; row0 < p.M; row0 += step) {
    BwdLayer<TX, ALIGNED> x[R][NC];
    BwdLayer<TDY, ALIGNED> dy[R][NC];
    float mean[R], rstd[R], s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row0 + r < p.M) {
        const uint32_t row = row0 + r;
        load_bwd<TX, NC, ALIGNED>(static_cast<const TX*>(p.x) + row * p.ldx, p.D, g.t, g.nt, x[r]);
        load_bwd<TDY, NC, ALIGNED>(static_cast<const TDY*>(p.dy) + row * p.lddy, p.D, g.t, g.nt, dy[r]);
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
      const uint32_t row = row0 + step + (g.t >> 1);
      if (plan.whole_pieces(row)) {
        if (g.t & 1)
          prefetch_row(static_cast<const TDY*>(p.dy) + row * p.lddy, p.D);
        else
          prefetch_row(static_cast<const TX*>(p.x) + row * p.ldx, p.D);
      }
    }
    // Outside the row dy is 0, so x's value there adds nothing.
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float a[2] = {0.f, 0.f}, b[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const Oct xv = unpack8(x[r][j]), dv = unpack8(dy[r][j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = (xv.e[i] - mean[r]) * rstd[r], gr = dv.e[i] * w[j].e[i];
          dw[j].e[i] = fmaf(dv.e[i], xh, dw[j].e[i]);
          db[j].e[i] += dv.e[i];
          a[i & 1] += gr;
          b[i & 1] = fmaf(gr, xh, b[i & 1]);
        }
      }
      s[2 * r] = a[0] + a[1];
      s[2 * r + 1] = b[0] + b[1];
    }
    group_sums<R>(g, flip, sh, s);
    flip ^= 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row0 + r >= p.M) break;
      // dx = r g - r sum g / D - xh r sum g xh / D
      const float c1 = -rstd[r] * (s[2 * r] * p.inv_d), c2 = -rstd[r] * (s[2 * r + 1] * p.inv_d);
      TX* dx = static_cast<TX*>(p.dx) + static_cast<int64_t>(row0 + r) * p.lddx;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const Oct xv = unpack8(x[r][j]), dv = unpack8(dy[r][j]);
        Oct o;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o.e[i] = fmaf((xv.e[i] - mean[r]) * rstd[r], c2, fmaf(dv.e[i] * w[j].e[i], rstd[r], c1));
        store_bwd<TX, ALIGNED>(dx, p.D, g.t, g.nt, j, o);
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
      const int c = bwd_column<ALIGNED>(g.t, g.nt, j, i);
      if (c < p.D) {
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
