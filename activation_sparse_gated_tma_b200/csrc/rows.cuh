// Kernels over rows of activations: layer norm, its backward pass, and the
// quantisation of rows to int8 with one scale each.
//
// All are bound by HBM: each row is read once, kept in the registers of the
// group of `warps_per_row` warps that owns it, and written once.  A thread
// owns the same columns of every row its group takes, so the norm's weight and
// bias (and, backward, their gradients' partial sums) stay in its registers
// while the group walks over rows.
//
// Columns of thread t in a group of T threads, j < CPT, i < 8:
//   VEC   8 (t + j T) + i    16-byte accesses (bases and row strides of 16 bytes)
//   else  (8 j + i) T + t    element accesses, neighbouring threads on neighbouring elements
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/twell.h"
#include "ptx.cuh"
#include "rows.h"

namespace twell {

// ---------------------------------------------------------------- element types
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Eight consecutive elements, 16-byte aligned.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <class T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  union { uint4 u; T e[8]; } c;
  c.u = *reinterpret_cast<const uint4*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f32(c.e[i]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
template <class T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  union { uint4 u; T e[8]; } c;
#pragma unroll
  for (int i = 0; i < 8; ++i) c.e[i] = from_f32<T>(v[i]);
  *reinterpret_cast<uint4*>(p) = c.u;
}

template <bool VEC>
__device__ __forceinline__ int row_column(int t, int T, int j, int i) {
  return VEC ? 8 * (t + j * T) + i : (8 * j + i) * T + t;
}

// This thread's elements of one row; columns from D on read as 0.
template <class T, int CPT, bool VEC>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int D, int t, int nt, float (&v)[CPT][8]) {
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    if (VEC && row_column<VEC>(t, nt, j, 8) <= D) {
      load8(row + row_column<VEC>(t, nt, j, 0), v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = row_column<VEC>(t, nt, j, i);
        v[j][i] = c < D ? to_f32(row[c]) : 0.f;
      }
    }
  }
}
template <class T, int CPT, bool VEC>
__device__ __forceinline__ void store_row(T* __restrict__ row, int D, int t, int nt, const float (&v)[CPT][8]) {
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    if (VEC && row_column<VEC>(t, nt, j, 8) <= D) {
      store8(row + row_column<VEC>(t, nt, j, 0), v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = row_column<VEC>(t, nt, j, i);
        if (c < D) row[c] = from_f32<T>(v[j][i]);
      }
    }
  }
}

// A parameter vector of a type known at run time (read once per thread);
// `fill` where p is NULL, 0 from D on.
template <int CPT, bool VEC>
__device__ __forceinline__ void load_vector(const void* p, int type, float fill, int D, int t, int nt,
                                            float (&v)[CPT][8]) {
#pragma unroll
  for (int j = 0; j < CPT; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = row_column<VEC>(t, nt, j, i);
      float e = fill;
      if (p && c < D)
        e = type == TWELL_F32    ? static_cast<const float*>(p)[c]
            : type == TWELL_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(p)[c])
                                 : to_f32(static_cast<const __half*>(p)[c]);
      v[j][i] = c < D ? e : 0.f;
    }
}

// ---------------------------------------------------------------- group reductions
// A block holds blockDim.x / T groups of T = 32 * warps threads, each on its
// own row with its own named barrier.  Consecutive reductions alternate
// between two shared buffers, so one barrier each is enough: a thread that
// writes a buffer again has passed the barrier of the reduction in between,
// which every thread reaches only after it has read the buffer.
struct Group {
  int warps, t, nt, id;  // warps per row, thread in the group, threads in the group, group in the block
  int flip = 0;
  float2* buf;           // [2][32] of this group
};

struct AddOp {
  __device__ float2 operator()(float2 a, float2 b) const { return make_float2(a.x + b.x, a.y + b.y); }
};
// Maximum of non-negative values by their bits, under which a NaN is above infinity.
struct MaxBitsOp {
  __device__ float2 operator()(float2 a, float2 b) const {
    return make_float2(__uint_as_float(max(__float_as_uint(a.x), __float_as_uint(b.x))), 0.f);
  }
};

// Reduces over the group; every thread gets the result.  The order is fixed.
template <class Op>
__device__ __forceinline__ float2 group_reduce(Group& g, float2 v, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = op(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  if (g.warps == 1) return v;
  float2* b = g.buf + 32 * g.flip;
  g.flip ^= 1;
  const int lane = g.t & 31;
  if (lane == 0) b[g.t >> 5] = v;
  named_bar_sync(1 + g.id, g.nt);
  v = lane < g.warps ? b[lane] : make_float2(0.f, 0.f);  // 0 is neutral for both operations
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = op(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  return v;
}

constexpr int kMaxGroups = 8;
constexpr int kRowThreads = 512;  // of a block at most, hence also of a row

__device__ __forceinline__ Group make_group(int warps, float2* buffers) {
  Group g;
  g.warps = warps;
  g.nt = 32 * warps;
  g.id = static_cast<int>(threadIdx.x) / g.nt;
  g.t = static_cast<int>(threadIdx.x) - g.id * g.nt;
  g.buf = buffers + 64 * g.id;
  return g;
}

// ---------------------------------------------------------------- quantisation
// One row's scale.  q is the integer nearest to 127 x / amax, ties to even,
// exactly: the product with the fp32 reciprocal is within 2e-5 of the quotient
// (|q| <= 127, two roundings of 2^-24), so where it lies further than 4e-5 from
// a half the nearest integer is certain, and else the quotient is taken in 64
// bits.  A row whose largest magnitude is so small that 127 / amax overflows
// takes all its quotients in 64 bits; one with a NaN or an infinity gets scale
// NaN and q = 0, one of zeros scale 0.
struct RowScale {
  float amax, inv, scale;
  bool wide, none;
};
__device__ __forceinline__ RowScale row_scale(float amax) {
  RowScale r;
  r.amax = amax;
  r.none = !(amax > 0.f && amax <= 3.402823466e38f);
  r.inv = 127.f / amax;
  r.wide = r.inv > 3.402823466e38f;
  r.scale = r.none && amax != 0.f ? __uint_as_float(0x7fc00000u) : amax / 127.f;
  return r;
}
__device__ __forceinline__ int quantize1(float x, const RowScale& r) {
  if (r.none) return 0;
  const float t = x * r.inv;
  float n = rintf(t);
  if (r.wide || fabsf(fabsf(t - n) - 0.5f) < 4e-5f)
    n = static_cast<float>(rint(static_cast<double>(x) * 127.0 / static_cast<double>(r.amax)));
  return static_cast<int>(n);
}
// Quantises and stores this thread's elements of a row.
template <int CPT, bool VEC>
__device__ __forceinline__ void store_row_i8(int8_t* __restrict__ row, int D, int t, int nt, const float (&v)[CPT][8],
                                             const RowScale& r) {
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    if (VEC && row_column<VEC>(t, nt, j, 8) <= D) {
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i >> 2] |= (static_cast<uint32_t>(quantize1(v[j][i], r)) & 0xffu) << (8 * (i & 3));
      *reinterpret_cast<uint2*>(row + row_column<VEC>(t, nt, j, 0)) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = row_column<VEC>(t, nt, j, i);
        if (c < D) row[c] = static_cast<int8_t>(quantize1(v[j][i], r));
      }
    }
  }
}
template <int CPT>
__device__ __forceinline__ float row_abs_max(const float (&v)[CPT][8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < CPT; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[j][i]) & 0x7fffffffu);
  return __uint_as_float(m);
}

// ---------------------------------------------------------------- layer norm
// mu = sum x / D, v = sum (x - mu)^2 / D, r = 1 / sqrt(v + eps),
// y = (x - mu) r w + b.  The variance is taken from the deviations (two
// reductions over registers, no second read): sums of squares would cancel for
// rows whose mean is far above their spread.  TO int8_t: y is quantised from
// its fp32 values, with one more reduction for the row's largest magnitude.
template <class TI, class TO, int CPT, bool VEC>
__global__ void __launch_bounds__(kRowThreads) layer_norm_kernel(const LayerNormParams p, int warps) {
  __shared__ float2 buffers[kMaxGroups * 64];
  Group g = make_group(warps, buffers);
  const int groups = static_cast<int>(blockDim.x) / g.nt;
  griddep_launch_dependents();
  griddep_wait();
  float w[CPT][8], b[CPT][8];
  load_vector<CPT, VEC>(p.weight, p.w_type, 1.f, p.D, g.t, g.nt, w);
  load_vector<CPT, VEC>(p.bias, p.w_type, 0.f, p.D, g.t, g.nt, b);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * groups + g.id; row < p.M;
       row += static_cast<int64_t>(gridDim.x) * groups) {
    float v[CPT][8];
    load_row<TI, CPT, VEC>(static_cast<const TI*>(p.x) + row * p.ldx, p.D, g.t, g.nt, v);
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < CPT; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[j][i];
    const float mean = group_reduce(g, make_float2(s, 0.f), AddOp()).x / p.D;
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < CPT; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[j][i] = row_column<VEC>(g.t, g.nt, j, i) < p.D ? v[j][i] - mean : 0.f;
        q += v[j][i] * v[j][i];
      }
    const float var = group_reduce(g, make_float2(q, 0.f), AddOp()).x / p.D;
    const float rstd = 1.f / sqrtf(var + p.eps);
#pragma unroll
    for (int j = 0; j < CPT; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * rstd * w[j][i] + b[j][i];
    if constexpr (sizeof(TO) == 1) {
      const RowScale r = row_scale(group_reduce(g, make_float2(row_abs_max(v), 0.f), MaxBitsOp()).x);
      store_row_i8<CPT, VEC>(static_cast<int8_t*>(p.y) + row * p.ldy, p.D, g.t, g.nt, v, r);
      if (g.t == 0) p.y_scale[row] = r.scale;
    } else {
      store_row<TO, CPT, VEC>(static_cast<TO*>(p.y) + row * p.ldy, p.D, g.t, g.nt, v);
    }
    if (g.t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
  }
}

// ---------------------------------------------------------------- layer norm, backward
// With xh = (x - mu) r and g = dy w:
//   dx = r (g - (sum g + xh sum g xh) / D),   dw = sum_rows dy xh,   db = sum_rows dy.
// A group adds its rows' dw and db in registers (fixed rows per group, so the
// sums' order depends on the sizes alone) and writes one partial row; a second
// kernel adds the partial rows.
template <class TX, class TDY, int CPT, bool VEC>
__global__ void __launch_bounds__(kRowThreads) layer_norm_bwd_kernel(const LayerNormBwdParams p, int warps) {
  __shared__ float2 buffers[kMaxGroups * 64];
  Group g = make_group(warps, buffers);
  const int groups = static_cast<int>(blockDim.x) / g.nt;
  griddep_launch_dependents();
  griddep_wait();
  float w[CPT][8], dw[CPT][8] = {}, db[CPT][8] = {};
  load_vector<CPT, VEC>(p.weight, p.w_type, 1.f, p.D, g.t, g.nt, w);
  const int64_t part = static_cast<int64_t>(blockIdx.x) * groups + g.id;
  for (int64_t row = part; row < p.M; row += static_cast<int64_t>(gridDim.x) * groups) {
    float x[CPT][8], dy[CPT][8];
    load_row<TX, CPT, VEC>(static_cast<const TX*>(p.x) + row * p.ldx, p.D, g.t, g.nt, x);
    load_row<TDY, CPT, VEC>(static_cast<const TDY*>(p.dy) + row * p.lddy, p.D, g.t, g.nt, dy);
    const float mean = p.mean[row], rstd = p.rstd[row];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < CPT; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = row_column<VEC>(g.t, g.nt, j, i) < p.D;
        x[j][i] = in ? (x[j][i] - mean) * rstd : 0.f;
        dw[j][i] += dy[j][i] * x[j][i];
        db[j][i] += dy[j][i];
        dy[j][i] *= w[j][i];
        s.x += dy[j][i];
        s.y += dy[j][i] * x[j][i];
      }
    s = group_reduce(g, s, AddOp());
    s.x /= p.D;
    s.y /= p.D;
#pragma unroll
    for (int j = 0; j < CPT; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = rstd * (dy[j][i] - s.x - x[j][i] * s.y);
    store_row<TX, CPT, VEC>(static_cast<TX*>(p.dx) + row * p.lddx, p.D, g.t, g.nt, x);
  }
  if (p.partial) {
    // Groups beyond the last row hold zeros and write nothing: the host counts min(M, groups) partial rows.
    if (part < p.M) {
      float* out = p.partial + part * 2 * p.D;
#pragma unroll
      for (int j = 0; j < CPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = row_column<VEC>(g.t, g.nt, j, i);
          if (c < p.D) {
            out[c] = dw[j][i];
            out[p.D + c] = db[j][i];
          }
        }
    }
  }
}

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

// ---------------------------------------------------------------- rows to int8 and back
// Rows longer than the group's registers hold are read twice.
template <class TI, int CPT, bool VEC>
__global__ void __launch_bounds__(kRowThreads) quantize_rows_kernel(const QuantizeParams p, int warps) {
  __shared__ float2 buffers[kMaxGroups * 64];
  Group g = make_group(warps, buffers);
  const int groups = static_cast<int>(blockDim.x) / g.nt;
  const int span = g.nt * 8 * CPT;
  griddep_launch_dependents();
  griddep_wait();
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * groups + g.id; row < p.M;
       row += static_cast<int64_t>(gridDim.x) * groups) {
    const TI* x = static_cast<const TI*>(p.x) + row * p.ldx;
    int8_t* y = static_cast<int8_t*>(p.y) + row * p.ldy;
    float v[CPT][8];
    uint32_t m = 0;
    for (int c = 0; c < p.K; c += span) {
      load_row<TI, CPT, VEC>(x + c, p.K - c, g.t, g.nt, v);
      m = max(m, __float_as_uint(row_abs_max(v)));
    }
    const RowScale r = row_scale(group_reduce(g, make_float2(__uint_as_float(m), 0.f), MaxBitsOp()).x);
    for (int c = 0; c < p.K; c += span) {
      if (p.K > span) load_row<TI, CPT, VEC>(x + c, p.K - c, g.t, g.nt, v);
      store_row_i8<CPT, VEC>(y + c, p.K - c, g.t, g.nt, v, r);
    }
    if (g.t == 0) p.scale[row] = r.scale;
  }
}

// x = q s: a thread takes eight columns of a row at a time.
template <class TO, bool VEC>
__global__ void __launch_bounds__(256) dequantize_rows_kernel(const QuantizeParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t chunks = (p.K + 7) / 8;
  const int64_t total = chunks * p.M;
  for (int64_t k = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; k < total;
       k += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = k / chunks;
    const int c = static_cast<int>(k - row * chunks) * 8;
    const int8_t* q = static_cast<const int8_t*>(p.x) + row * p.ldx + c;
    TO* y = static_cast<TO*>(p.y) + row * p.ldy + c;
    const float s = p.scale[row];
    if (VEC && c + 8 <= p.K) {
      union { uint2 u; int8_t e[8]; } in;
      in.u = *reinterpret_cast<const uint2*>(q);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(in.e[i]) * s;
      store8(y, v);
    } else {
      for (int i = 0; i < 8 && c + i < p.K; ++i) y[i] = from_f32<TO>(static_cast<float>(q[i]) * s);
    }
  }
}

}  // namespace twell
