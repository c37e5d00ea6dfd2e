// Kernels over rows of activations: layer norm, its backward pass, and the
// quantisation of rows to int8 with one scale each.
//
// All are bound by HBM: each row is read once and written once.  What competes
// with the copies is the instruction issue (a bf16 row of 2560 leaves an SM
// 290 cycles), so the work per row that does not depend on its length is kept
// small: a row belongs to one warp up to 2560 columns (more for longer rows, or
// while rows are too few for the warps), whose lanes hold it as packed fp32
// pairs; the norm's weight and bias are read from shared memory.
//
// Rows arrive through a ring of shared-memory slots filled by bulk copies (one
// per row, one thread issues them), several rows ahead: the bytes in flight
// cost no registers and do not pause at the reductions.  A bulk copy takes
// whole 16-byte pieces, so a row that starts or ends inside one is fetched
// with its neighbours' bytes and read from its own offset; rows for which that
// would reach outside the matrix (a few at either end) are copied into their
// slots with plain loads.
//
// Columns of thread t in a group of T threads, layer j < NG, i < 4: 4 (t + j T) + i,
// read and written four at a time.  Rows that do not start on four elements'
// common alignment are read from shared memory at their offset and shifted
// together; towards global memory neighbouring lanes exchange what lies across
// an aligned piece, and only a warp's first and last piece go out by elements.
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

// ---------------------------------------------------------------- quads
// Four consecutive elements.
struct Quad {
  float e[4];
};
__device__ __forceinline__ Quad load4(const float* p) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  return Quad{{v.x, v.y, v.z, v.w}};
}
__device__ __forceinline__ float2 unpack2(uint32_t u, __nv_bfloat16) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t u, __half) {
  union { uint32_t u; __half2 h; } c;
  c.u = u;
  return __half22float2(c.h);
}
template <class T>
__device__ __forceinline__ Quad unpack4(uint2 u) {
  const float2 a = unpack2(u.x, T()), b = unpack2(u.y, T());
  return Quad{{a.x, a.y, b.x, b.y}};
}
template <class T>
__device__ __forceinline__ Quad load4(const T* p) {
  return unpack4<T>(*reinterpret_cast<const uint2*>(p));
}
// The same from shared memory at any element; `bytes` is p's distance from the
// common alignment, the same for all lanes.  Reads up to 8 bytes behind the quad.
__device__ __forceinline__ Quad load4_at(const float* p, uint32_t) { return Quad{{p[0], p[1], p[2], p[3]}}; }
template <class T>
__device__ __forceinline__ Quad load4_at(const T* p, uint32_t bytes) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(p) - (bytes & 2));
  const uint32_t s = 8 * (bytes & 2);
  return unpack4<T>(make_uint2(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s)));
}

__device__ __forceinline__ uint4 pack4(Quad q, float) {
  return make_uint4(__float_as_uint(q.e[0]), __float_as_uint(q.e[1]), __float_as_uint(q.e[2]), __float_as_uint(q.e[3]));
}
__device__ __forceinline__ uint2 pack4(Quad q, __nv_bfloat16) {
  union { uint2 u; __nv_bfloat162 e[2]; } c;
  c.e[0] = __floats2bfloat162_rn(q.e[0], q.e[1]);
  c.e[1] = __floats2bfloat162_rn(q.e[2], q.e[3]);
  return c.u;
}
__device__ __forceinline__ uint2 pack4(Quad q, __half) {
  union { uint2 u; __half2 e[2]; } c;
  c.e[0] = __floats2half2_rn(q.e[0], q.e[1]);
  c.e[1] = __floats2half2_rn(q.e[2], q.e[3]);
  return c.u;
}
// What an aligned piece holds when rows start `bytes` behind one: the last
// `bytes` of the quad before (`p`), then the first of this one (`c`).
__device__ __forceinline__ uint32_t join(uint32_t p, uint32_t c, uint32_t bytes) {
  return __funnelshift_l(p, c, 8 * bytes);
}
__device__ __forceinline__ uint2 join(uint2 p, uint2 c, uint32_t bytes) {
  const uint32_t s = 8 * (bytes & 3), w0 = bytes & 4 ? p.x : p.y, w1 = bytes & 4 ? p.y : c.x, w2 = bytes & 4 ? c.x : c.y;
  return make_uint2(__funnelshift_l(w0, w1, s), __funnelshift_l(w1, w2, s));
}
__device__ __forceinline__ uint4 join(uint4 p, uint4 c, uint32_t bytes) {
  // By two words, then by one.
  const bool two = bytes & 8, one = bytes & 4;
  const uint32_t a = two ? p.y : p.w, b = two ? p.z : c.x, d = two ? p.w : c.y, e = two ? c.x : c.z, f = two ? c.y : c.w;
  return make_uint4(one ? a : b, one ? b : d, one ? d : e, one ? e : f);
}
__device__ __forceinline__ uint32_t lane_before(uint32_t v) { return __shfl_up_sync(0xffffffffu, v, 1); }
__device__ __forceinline__ uint2 lane_before(uint2 v) { return make_uint2(lane_before(v.x), lane_before(v.y)); }
__device__ __forceinline__ uint4 lane_before(uint4 v) {
  return make_uint4(lane_before(v.x), lane_before(v.y), lane_before(v.z), lane_before(v.w));
}
template <class T, class P>
__device__ __forceinline__ T element_of(P v, int i) {
  union { P v; T e[4]; } c;
  c.v = v;
  return c.e[i];
}
// A warp's 32 neighbouring quads (this lane's starts at column c of a row of D)
// to global memory; `bytes`: how far the row starts behind an aligned piece.
// FULL: all 32 lie inside the row.  ALIGNED rows start on aligned pieces and
// have whole quads.  The whole warp calls it.
template <class T, bool ALIGNED, bool FULL, class P>
__device__ __forceinline__ void store_warp_quads(T* row, uint32_t bytes, int c, int D, P v) {
  static_assert(sizeof(P) == 4 * sizeof(T), "a quad of T");
  if (ALIGNED) {
    if (FULL || c < D) *reinterpret_cast<P*>(row + c) = v;
    return;
  }
  const int lane = threadIdx.x & 31;
  if (FULL || c - 4 * lane + 128 <= D) {
    const int s = static_cast<int>(bytes / sizeof(T));
    const P piece = join(lane_before(v), v, bytes);
    if (lane > 0 || s == 0) *reinterpret_cast<P*>(row + c - s) = piece;
    if (s > 0 && (lane == 0 || lane == 31)) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((lane == 0) == (i < 4 - s)) row[c + i] = element_of<T>(v, i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < D) row[c + i] = element_of<T>(v, i);
  }
}

// ---------------------------------------------------------------- a thread's part of a row
// A row is held as NG layers, the smallest of 1, 2, 4, 8, 12, 16, 20 that covers
// it, so that many of them are full.
__host__ __device__ constexpr int full_layers(int NG) { return NG > 4 ? NG - 4 : NG / 2; }
template <int NG>
struct RowPart {
  Quad q[NG];
};
__device__ __forceinline__ int row_column(int t, int T, int j) { return 4 * (t + j * T); }

// This thread's elements of one row in shared memory; columns from D on read as 0.
template <class T, int NG, bool ALIGNED>
__device__ __forceinline__ void load_row(const T* row, int D, int t, int nt, RowPart<NG>& r) {
  const uint32_t bytes = ALIGNED ? 0 : smem_u32(row) & (4 * sizeof(T) - 1);
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    const int c = row_column(t, nt, j);
    r.q[j] = Quad{{0.f, 0.f, 0.f, 0.f}};
    if (ALIGNED) {
      if (j < full_layers(NG) || c < D) r.q[j] = load4(row + c);
    } else if (j < full_layers(NG) || c + 4 <= D) {
      r.q[j] = load4_at(row + c, bytes);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < D) r.q[j].e[i] = to_f32(row[c + i]);
    }
  }
}

// A parameter vector of D elements into `padded` floats of shared memory, by
// the whole block; `fill` where p is NULL and from D on.
__device__ __forceinline__ void stage_vector(const void* p, int type, float fill, int D, int padded, float* to) {
  for (int c = threadIdx.x; c < padded; c += blockDim.x) {
    float e = fill;
    if (p && c < D)
      e = type == TWELL_F32    ? static_cast<const float*>(p)[c]
          : type == TWELL_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(p)[c])
                               : to_f32(static_cast<const __half*>(p)[c]);
    to[c] = e;
  }
}

// ---------------------------------------------------------------- groups
// A block holds blockDim.x / T groups of T = 32 W threads, each on its own
// rows with its own named barrier, ring and reduction buffers.
struct Group {
  int warps, t, nt, id;  // warps per row, thread in the group, threads in the group, group in the block
  int flip;
  float* buf;            // [2][8] of this group
};
struct GroupShared {
  float buf[kMaxGroups][2][kMaxGroupWarps];
  uint64_t full[kMaxGroups][kMaxSlots];
};

__device__ __forceinline__ Group make_group(int warps, GroupShared& sh) {
  Group g;
  g.warps = warps;
  g.nt = 32 * warps;
  g.id = static_cast<int>(threadIdx.x) / g.nt;
  g.t = static_cast<int>(threadIdx.x) - g.id * g.nt;
  g.flip = 0;
  g.buf = &sh.buf[g.id][0][0];
  return g;
}
__device__ __forceinline__ void group_sync(const Group& g) {
  if (g.warps == 1)
    __syncwarp();
  else
    named_bar_sync(1 + g.id, g.nt);
}

// Group-wide sum in a fixed order, or maximum of magnitudes (by their bits,
// under which a NaN is above infinity); every thread gets it.  Consecutive reductions
// alternate between two shared buffers, so one barrier each is enough: a thread
// that writes a buffer again has passed the barrier of the reduction in
// between, which every thread reaches only after it has read the buffer.
__device__ __forceinline__ float group_sum(Group& g, float v) {
  v = warp_sum(v);
  if (g.warps == 1) return v;
  float* b = g.buf + kMaxGroupWarps * g.flip;
  g.flip ^= 1;
  if ((g.t & 31) == 0) b[g.t >> 5] = v;
  named_bar_sync(1 + g.id, g.nt);
  v = b[0];
  for (int w = 1; w < g.warps; ++w) v += b[w];
  return v;
}
__device__ __forceinline__ float group_max(Group& g, float magnitude) {
  uint32_t v = __reduce_max_sync(0xffffffffu, __float_as_uint(magnitude));
  if (g.warps == 1) return __uint_as_float(v);
  uint32_t* b = reinterpret_cast<uint32_t*>(g.buf + kMaxGroupWarps * g.flip);
  g.flip ^= 1;
  if ((g.t & 31) == 0) b[g.t >> 5] = v;
  named_bar_sync(1 + g.id, g.nt);
  v = b[0];
  for (int w = 1; w < g.warps; ++w) v = max(v, b[w]);
  return __uint_as_float(v);
}

// ---------------------------------------------------------------- the ring
__device__ __forceinline__ void bulk_load(uint32_t dst, uint64_t src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// The whole 16-byte pieces of a row: where they start and their bytes.
struct RowPieces {
  uint64_t at;
  uint32_t bytes;
};
__device__ __forceinline__ RowPieces row_pieces(uint64_t row, uint32_t row_bytes) {
  RowPieces r;
  r.at = row & ~uint64_t(15);
  r.bytes = ((static_cast<uint32_t>(row) & 15u) + row_bytes + 15u) & ~15u;
  return r;
}
// One thread: one row into a slot, completing on a barrier of its own.
__device__ __forceinline__ void fetch_row(uint64_t row, uint32_t row_bytes, uint32_t slot, uint64_t* bar) {
  const RowPieces r = row_pieces(row, row_bytes);
  mbar_arrive_expect_tx(bar, r.bytes);
  bulk_load(slot, r.at, r.bytes, bar);
}
// A row with plain loads, by `threads` threads (rows whose 16-byte pieces reach outside the matrix).
template <class T>
__device__ __forceinline__ void stage_row(uint64_t row, int D, uint8_t* slot, int t, int threads) {
  const T* x = reinterpret_cast<const T*>(row);
  T* to = reinterpret_cast<T*>(slot + (row & 15));
#pragma unroll 1
  for (int c = t; c < D; c += threads) to[c] = x[c];
}

// A group's walk over its rows first, first + step, ... through its ring: the
// row that follows row r into r's slot is r + slots * step.  Rows outside
// [begin, end) are copied in when their turn comes.
template <class T>
struct RowWalk {
  uint64_t base, ahead;   // the matrix; the next row to fetch
  uint64_t ld_bytes;
  uint32_t row_bytes, next, step;
  uint8_t* ring;
  uint64_t* full;
  int slot;
  uint32_t parity;

  __device__ __forceinline__ bool fetched(uint32_t row, const RowPlan& plan) const {
    return row >= plan.ring_begin && row < plan.ring_end;
  }
  __device__ __forceinline__ void fetch(const RowPlan& plan, int into) {
    if (fetched(next, plan)) fetch_row(ahead, row_bytes, smem_u32(ring + into * plan.slot_bytes), &full[into]);
    next += step;
    ahead += step * ld_bytes;
  }
  // Set-up by the group's first thread; holds the block's barrier and the wait for the kernel before.
  __device__ __forceinline__ void start(const void* p, int64_t ld, int D, const Group& g, const RowPlan& plan,
                                        uint8_t* smem, uint64_t* bars, uint32_t first, uint32_t step_) {
    base = reinterpret_cast<uint64_t>(p);
    ld_bytes = ld * sizeof(T);
    row_bytes = D * static_cast<uint32_t>(sizeof(T));
    step = step_;
    ring = smem + g.id * plan.slots * plan.slot_bytes;
    full = bars;
    slot = 0;
    parity = 0;
    next = first;
    ahead = base + next * ld_bytes;
    if (g.t == 0) {
      for (int s = 0; s < plan.slots; ++s) mbar_init(&full[s], 1);
      fence_barrier_init();
    }
    __syncthreads();
    griddep_launch_dependents();
    griddep_wait();
    if (g.t == 0)
      for (int s = 0; s < plan.slots; ++s) fetch(plan, s);
  }
  // Row `row` into registers; NaN if its copy never arrived.
  template <int NG, bool ALIGNED>
  __device__ __forceinline__ void load(uint32_t row, int D, const Group& g, const RowPlan& plan, RowPart<NG>& v) {
    const uint64_t a = base + row * ld_bytes;
    uint8_t* at = ring + slot * plan.slot_bytes;
    bool ok = true;
    if (fetched(row, plan)) {
      ok = mbar_wait(&full[slot], parity >> slot & 1u, nullptr);
      parity ^= 1u << slot;
    } else {
      stage_row<T>(a, D, at, g.t, g.nt);
      group_sync(g);
    }
    load_row<T, NG, ALIGNED>(reinterpret_cast<const T*>(at + (a & 15)), D, g.t, g.nt, v);
    if (!ok) v.q[0].e[0] = __uint_as_float(0x7fc00000u);
  }
  // After a reduction: every thread of the group has its part of the row, so its slot may be filled again.
  __device__ __forceinline__ void release(const Group& g, const RowPlan& plan) {
    if (g.warps == 1) __syncwarp();
    if (g.t == 0) fetch(plan, slot);
    if (++slot == plan.slots) slot = 0;
  }
};

// ---------------------------------------------------------------- quantisation
// One row's scale.  q is the integer nearest to 127 x / amax, ties to even,
// exactly.  inv = 127 / amax in fp32 is within 2^-24 of the quotient's factor,
// so the true quotient lies between x low and x high, low and high 2^-22 below
// and above inv.  Adding 1.5 * 2^23 rounds both to integers (held in the sum's
// low byte); where they agree that is the answer, else the quotient is taken in
// 64 bits.  A row whose largest magnitude is so small that 127 / amax overflows
// takes all its quotients in 64 bits; one with a NaN or an infinity gets scale
// NaN and q = 0, one of zeros scale 0.
struct RowScale {
  float amax, low, high, scale;
};
__device__ __forceinline__ RowScale row_scale(float amax) {
  RowScale r;
  r.amax = amax;
  const float inv = 127.f / amax;
  const bool finite = amax <= 3.402823466e38f;  // a NaN is not
  r.low = inv * (1.f - 0x1p-22f);
  r.high = inv * (1.f + 0x1p-22f);
  if (r.high > 3.402823466e38f) r.low = 0.f;  // low and high never agree: every quotient in 64 bits
  if (!finite || amax == 0.f) r.low = r.high = 0.f;
  r.scale = finite ? amax / 127.f : __uint_as_float(0x7fc00000u);
  return r;
}
// Four values to four bytes; sets bits of `differ` where the 64-bit quotient is needed.
__device__ __forceinline__ uint32_t pack_low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t quantize4(Quad v, const RowScale& r, uint32_t& differ) {
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[i] = __float_as_uint(fmaf(v.e[i], r.low, 12582912.f));
    differ |= q[i] ^ __float_as_uint(fmaf(v.e[i], r.high, 12582912.f));
  }
  return pack_low_bytes(q[0], q[1], q[2], q[3]);
}
static __device__ __noinline__ uint32_t quantize4_wide(Quad v, float amax) {
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = static_cast<uint32_t>(static_cast<int>(rint(static_cast<double>(v.e[i]) * 127.0 / static_cast<double>(amax))));
  return pack_low_bytes(q[0], q[1], q[2], q[3]);
}
// This thread's elements of a row in int8.
template <int NG>
__device__ __forceinline__ void quantize_row(const RowPart<NG>& v, const RowScale& r, uint32_t (&q)[NG]) {
  uint32_t differ = 0;
#pragma unroll
  for (int j = 0; j < NG; ++j) q[j] = quantize4(v.q[j], r, differ);
  if (r.high == 0.f) {  // zeros, or a NaN or an infinity in the row
#pragma unroll
    for (int j = 0; j < NG; ++j) q[j] = 0;
  } else if (differ) {
#pragma unroll
    for (int j = 0; j < NG; ++j) q[j] = quantize4_wide(v.q[j], r.amax);
  }
}
template <int NG, bool ALIGNED>
__device__ __forceinline__ void store_row_i8(int8_t* row, int D, int t, int nt, const uint32_t (&q)[NG]) {
  const uint32_t bytes = static_cast<uint32_t>(reinterpret_cast<uint64_t>(row)) & 3;
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    if (j < full_layers(NG))
      store_warp_quads<int8_t, ALIGNED, true>(row, bytes, row_column(t, nt, j), D, q[j]);
    else
      store_warp_quads<int8_t, ALIGNED, false>(row, bytes, row_column(t, nt, j), D, q[j]);
  }
}
// The larger magnitude; a NaN stays one.
__device__ __forceinline__ float max_abs(float m, float v) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(m), "f"(fabsf(v)));
  return d;
}
template <int NG>
__device__ __forceinline__ float row_abs_max(const RowPart<NG>& r) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < NG; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max_abs(m, r.q[j].e[i]);
  return m;
}

// ---------------------------------------------------------------- layer norm
// mu = sum x / D, v = sum (x - mu)^2 / D, r = 1 / sqrt(v + eps),
// y = (x - mu) r w + b.  The variance is taken from the deviations (two
// reductions over registers, no second read): sums of squares would cancel for
// rows whose mean is far above their spread.  TO int8_t: y is quantised from
// its fp32 values, with one more reduction for the row's largest magnitude.
template <class TI, class TO, int NG, bool ALIGNED>
__global__ void __launch_bounds__(kRowThreads, row_blocks(NG)) layer_norm_kernel(const LayerNormParams p, const RowPlan plan) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ GroupShared sh;
  Group g = make_group(plan.warps, sh);
  const uint32_t groups = blockDim.x / g.nt, first = blockIdx.x * groups + g.id, step = gridDim.x * groups;
  const int padded = 4 * NG * g.nt;  // whole layers, read without a check
  float* w = reinterpret_cast<float*>(smem);
  float* b = w + padded;
  RowWalk<TI> walk;
  walk.start(p.x, p.ldx, p.D, g, plan, smem + 8 * padded, sh.full[g.id], first, step);
  stage_vector(p.weight, p.w_type, p.weight ? 0.f : 1.f, p.D, padded, w);
  stage_vector(p.bias, p.w_type, 0.f, p.D, padded, b);
  __syncthreads();
  for (uint32_t row = first; row < p.M; row += step) {
    RowPart<NG> v;
    walk.template load<NG, ALIGNED>(row, p.D, g, plan, v);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NG; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += v.q[j].e[i];
    const float mean = group_sum(g, (s[0] + s[1]) + (s[2] + s[3])) * p.inv_d;
    walk.release(g, plan);
    float q[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const int c = row_column(g.t, g.nt, j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v.q[j].e[i] -= mean;
        if (j < full_layers(NG) || c + (ALIGNED ? 0 : i) < p.D) q[i] = fmaf(v.q[j].e[i], v.q[j].e[i], q[i]);
      }
    }
    const float rstd = rsqrtf(group_sum(g, (q[0] + q[1]) + (q[2] + q[3])) * p.inv_d + p.eps);
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const Quad qw = load4(w + row_column(g.t, g.nt, j)), qb = load4(b + row_column(g.t, g.nt, j));
#pragma unroll
      for (int i = 0; i < 4; ++i) v.q[j].e[i] = fmaf(v.q[j].e[i] * rstd, qw.e[i], qb.e[i]);
      if constexpr (sizeof(TO) > 1) {
        TO* y = static_cast<TO*>(p.y) + row * p.ldy;
        const uint32_t bytes = static_cast<uint32_t>(reinterpret_cast<uint64_t>(y)) & (4 * sizeof(TO) - 1);
        const int c = row_column(g.t, g.nt, j);
        if (j < full_layers(NG))
          store_warp_quads<TO, ALIGNED, true>(y, bytes, c, p.D, pack4(v.q[j], TO()));
        else
          store_warp_quads<TO, ALIGNED, false>(y, bytes, c, p.D, pack4(v.q[j], TO()));
      }
    }
    if constexpr (sizeof(TO) == 1) {
      const RowScale r = row_scale(group_max(g, row_abs_max(v)));
      uint32_t q8[NG];
      quantize_row(v, r, q8);
      store_row_i8<NG, ALIGNED>(static_cast<int8_t*>(p.y) + row * p.ldy, p.D, g.t, g.nt, q8);
      if (g.t == 0) p.y_scale[row] = r.scale;
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
// dw and db want a thread to keep its columns over many rows, the two sums over
// a row want few threads per row.  So a block takes batches of `rows` rows
// through the ring (x and dy) and goes over each batch twice, in shared memory:
// first a few warps per row form its sums, then every thread takes its own
// columns of all the rows, adds to its dw and db in registers and writes dx.
// Batches are dealt to blocks in a fixed way, so the order of every sum depends
// on the sizes alone.  Each block writes one partial row of dw and db; a second
// kernel adds those.
template <class TX, class TDY, int NL, bool ALIGNED>
__global__ void __launch_bounds__(kBwdThreads, NL == 2 ? 2 : 1)
    layer_norm_bwd_kernel(const LayerNormBwdParams p, const BatchPlan plan) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kMaxSlots];
  __shared__ float2 sums[kMaxBatch][kBwdThreads / 32];  // per row and warp of the row
  __shared__ float2 stats[kMaxBatch];                   // mean, rstd
  const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, warp = t >> 5, warps = nt >> 5;
  const int padded = 4 * NL * nt;
  float* w = reinterpret_cast<float*>(smem);
  uint8_t* ring = smem + 4 * padded;
  const uint32_t x_bytes = p.D * static_cast<uint32_t>(sizeof(TX)), dy_bytes = p.D * static_cast<uint32_t>(sizeof(TDY));
  const uint32_t x_slot = row_slot_bytes(x_bytes), row_slot = x_slot + row_slot_bytes(dy_bytes);
  const uint32_t batch_bytes = plan.rows * row_slot;
  const int per_row = max(1, warps / plan.rows);  // warps of a row in the first pass
  const uint64_t x_base = reinterpret_cast<uint64_t>(p.x), x_ld = p.ldx * sizeof(TX);
  const uint64_t dy_base = reinterpret_cast<uint64_t>(p.dy), dy_ld = p.lddy * sizeof(TDY);

  // Lane r of warp 0 fetches row r of a batch; a row outside the ring's range only arrives.
  auto fetch = [&](uint32_t batch, int slot) {
    if (batch >= plan.batches || lane >= plan.rows) return;
    const uint32_t row = batch * plan.rows + lane;
    if (row < plan.ring_begin || row >= plan.ring_end) {
      mbar_arrive(&full[slot]);
      return;
    }
    const RowPieces a = row_pieces(x_base + row * x_ld, x_bytes), b = row_pieces(dy_base + row * dy_ld, dy_bytes);
    const uint32_t at = smem_u32(ring) + slot * batch_bytes + lane * row_slot;
    mbar_arrive_expect_tx(&full[slot], a.bytes + b.bytes);
    bulk_load(at, a.at, a.bytes, &full[slot]);
    bulk_load(at + x_slot, b.at, b.bytes, &full[slot]);
  };
  if (t == 0) {
    for (int s = 0; s < plan.slots; ++s) mbar_init(&full[s], plan.rows);
    fence_barrier_init();
  }
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();
  if (warp == 0)
    for (int s = 0; s < plan.slots; ++s) fetch(blockIdx.x + s * gridDim.x, s);
  stage_vector(p.weight, p.w_type, p.weight ? 0.f : 1.f, p.D, padded, w);

  Quad dw[NL], db[NL];
#pragma unroll
  for (int j = 0; j < NL; ++j) dw[j] = db[j] = Quad{{0.f, 0.f, 0.f, 0.f}};
  const int first_row = warp / per_row, my_part = warp - first_row * per_row, high = warps / per_row;
  int slot = 0;
  uint32_t parity = 0;
  // Thread r has row r's mean and rstd, one batch ahead.
  float2 ahead = make_float2(0.f, 0.f);
  if (t < plan.rows && blockIdx.x * plan.rows + t < p.M)
    ahead = make_float2(p.mean[blockIdx.x * plan.rows + t], p.rstd[blockIdx.x * plan.rows + t]);
  for (uint32_t batch = blockIdx.x; batch < plan.batches; batch += gridDim.x) {
    const uint32_t row0 = batch * plan.rows;
    const int rows = min(static_cast<uint32_t>(plan.rows), p.M - row0);
    uint8_t* at = ring + slot * batch_bytes;
    const bool ok = mbar_wait(&full[slot], parity, nullptr);
    if (row0 < plan.ring_begin || row0 + rows > plan.ring_end) {
      for (int r = 0; r < rows; ++r)
        if (row0 + r < plan.ring_begin || row0 + r >= plan.ring_end) {
          stage_row<TX>(x_base + (row0 + r) * x_ld, p.D, at + r * row_slot, t, nt);
          stage_row<TDY>(dy_base + (row0 + r) * dy_ld, p.D, at + r * row_slot + x_slot, t, nt);
        }
    }
    if (t < plan.rows) stats[t] = ahead;
    __syncthreads();  // also: staged rows and, the first time, the weight
    if (t < plan.rows && batch + gridDim.x < plan.batches) {
      const uint32_t row = (batch + gridDim.x) * plan.rows + t;
      if (row < p.M) ahead = make_float2(p.mean[row], p.rstd[row]);
    }
    for (int my_row = first_row; my_row < rows; my_row += high) {
      const float2 st = stats[my_row];
      const TX* x = reinterpret_cast<const TX*>(at + my_row * row_slot + ((x_base + (row0 + my_row) * x_ld) & 15));
      const TDY* dy = reinterpret_cast<const TDY*>(at + my_row * row_slot + x_slot + ((dy_base + (row0 + my_row) * dy_ld) & 15));
      float s1[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t xo = smem_u32(x) & (4 * sizeof(TX) - 1), dyo = smem_u32(dy) & (4 * sizeof(TDY) - 1);
      const int across = 128 * per_row;
#pragma unroll 4
      for (int c = 4 * (my_part * 32 + lane); c + 4 <= p.D; c += across) {
        const Quad qx = ALIGNED ? load4(x + c) : load4_at(x + c, xo), qd = ALIGNED ? load4(dy + c) : load4_at(dy + c, dyo);
        const Quad qw = load4(w + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float gr = qd.e[i] * qw.e[i];
          s1[i] += gr;
          s2[i] = fmaf(gr, (qx.e[i] - st.x) * st.y, s2[i]);
        }
      }
      const int tail = (p.D & ~3) + lane;
      if (my_part == 0 && tail < p.D) {
        const float gr = to_f32(dy[tail]) * w[tail];
        s1[0] += gr;
        s2[0] += gr * ((to_f32(x[tail]) - st.x) * st.y);
      }
      float2 s = make_float2(warp_sum((s1[0] + s1[1]) + (s1[2] + s1[3])), warp_sum((s2[0] + s2[1]) + (s2[2] + s2[3])));
      if (!ok) s.x = __uint_as_float(0x7fc00000u);
      if (lane == 0) sums[my_row][my_part] = s;
    }
    __syncthreads();
    for (int r = 0; r < rows; ++r) {
      const float2 m = stats[r];
      float2 s = sums[r][0];
      for (int k = 1; k < per_row; ++k) {
        s.x += sums[r][k].x;
        s.y += sums[r][k].y;
      }
      // dx = r g - r sum g / D - xh r sum g xh / D
      const float c1 = -m.y * (s.x * p.inv_d), c2 = -m.y * (s.y * p.inv_d);
      const TX* x = reinterpret_cast<const TX*>(at + r * row_slot + ((x_base + (row0 + r) * x_ld) & 15));
      const TDY* dy = reinterpret_cast<const TDY*>(at + r * row_slot + x_slot + ((dy_base + (row0 + r) * dy_ld) & 15));
      const uint32_t xo = smem_u32(x) & (4 * sizeof(TX) - 1), dyo = smem_u32(dy) & (4 * sizeof(TDY) - 1);
      TX* dx = static_cast<TX*>(p.dx) + static_cast<int64_t>(row0 + r) * p.lddx;
      const uint32_t dxo = static_cast<uint32_t>(reinterpret_cast<uint64_t>(dx)) & (4 * sizeof(TX) - 1);
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const int c = row_column(t, nt, j);
        Quad qx{{0.f, 0.f, 0.f, 0.f}}, qd = qx, out;
        if (c + 4 <= p.D) {
          qx = ALIGNED ? load4(x + c) : load4_at(x + c, xo);
          qd = ALIGNED ? load4(dy + c) : load4_at(dy + c, dyo);
        } else if (!ALIGNED) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i < p.D) {
              qx.e[i] = to_f32(x[c + i]);
              qd.e[i] = to_f32(dy[c + i]);
            }
        }
        const Quad qw = load4(w + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float xh = (qx.e[i] - m.x) * m.y;
          dw[j].e[i] = fmaf(qd.e[i], xh, dw[j].e[i]);
          db[j].e[i] += qd.e[i];
          out.e[i] = fmaf(xh, c2, fmaf(qd.e[i] * qw.e[i], m.y, c1));
        }
        store_warp_quads<TX, ALIGNED, false>(dx, dxo, c, p.D, pack4(out, TX()));
      }
    }
    __syncthreads();  // the batch's slot may be filled again
    if (warp == 0) fetch(batch + plan.slots * gridDim.x, slot);
    if (++slot == plan.slots) {
      slot = 0;
      parity ^= 1u;
    }
  }
  if (p.partial) {
    float* out = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
#pragma unroll
    for (int j = 0; j < NL; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = row_column(t, nt, j) + i;
        if (c < p.D) {
          out[c] = dw[j].e[i];
          out[p.D + c] = db[j].e[i];
        }
      }
  }
}

// ---------------------------------------------------------------- rows to int8 and back
template <class TI, int NG, bool ALIGNED>
__global__ void __launch_bounds__(kRowThreads, row_blocks(NG)) quantize_rows_kernel(const QuantizeParams p, const RowPlan plan) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ GroupShared sh;
  Group g = make_group(plan.warps, sh);
  const uint32_t groups = blockDim.x / g.nt, first = blockIdx.x * groups + g.id, step = gridDim.x * groups;
  RowWalk<TI> walk;
  walk.start(p.x, p.ldx, p.K, g, plan, smem, sh.full[g.id], first, step);
  for (uint32_t row = first; row < p.M; row += step) {
    RowPart<NG> v;
    walk.template load<NG, ALIGNED>(row, p.K, g, plan, v);
    const RowScale r = row_scale(group_max(g, row_abs_max(v)));
    walk.release(g, plan);
    uint32_t q8[NG];
    quantize_row(v, r, q8);
    store_row_i8<NG, ALIGNED>(static_cast<int8_t*>(p.y) + row * p.ldy, p.K, g.t, g.nt, q8);
    if (g.t == 0) p.scale[row] = r.scale;
  }
}

// Rows longer than a block's registers hold: a block per row, read twice by
// elements (the second time from L2), whatever the alignment.
template <class TI>
__global__ void __launch_bounds__(kRowThreads) quantize_long_rows_kernel(const QuantizeParams p) {
  __shared__ GroupShared sh;
  Group g = make_group(kRowThreads / 32, sh);
  griddep_launch_dependents();
  griddep_wait();
  for (uint32_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const TI* x = static_cast<const TI*>(p.x) + row * p.ldx;
    int8_t* y = static_cast<int8_t*>(p.y) + row * p.ldy;
    float m = 0.f;
#pragma unroll 16
    for (int c = g.t; c < p.K; c += kRowThreads) m = max_abs(m, to_f32(x[c]));
    const RowScale r = row_scale(group_max(g, m));
#pragma unroll 2
    for (int c = g.t; c < p.K; c += 4 * kRowThreads) {
      Quad v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v.e[i] = c + i * kRowThreads < p.K ? to_f32(x[c + i * kRowThreads]) : 0.f;
      uint32_t differ = 0, q = quantize4(v, r, differ);
      if (r.high == 0.f)
        q = 0;
      else if (differ)
        q = quantize4_wide(v, r.amax);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i * kRowThreads < p.K) y[c + i * kRowThreads] = static_cast<int8_t>(q >> (8 * i));
    }
    if (g.t == 0) p.scale[row] = r.scale;
  }
}

// x = q s.  Blocks of `across` threads along a row, four columns each at a
// time, by 256 / across rows.  A byte becomes fp32 without a conversion: with
// its sign bit flipped it is the last byte of 2^23 + q + 128.
__device__ __forceinline__ Quad dequantize4(uint32_t word, float s) {
  const uint32_t u = word ^ 0x80808080u;
  Quad v;
  v.e[0] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440));
  v.e[1] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441));
  v.e[2] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442));
  v.e[3] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443));
#pragma unroll
  for (int i = 0; i < 4; ++i) v.e[i] = (v.e[i] - 8388736.f) * s;  // 2^23 + 128
  return v;
}
// Q_ALIGNED: q's rows start on four bytes.
template <class TO, bool Q_ALIGNED, bool ALIGNED>
__global__ void __launch_bounds__(256) dequantize_rows_kernel(const QuantizeParams p, int across) {
  griddep_launch_dependents();
  griddep_wait();
  const int tx = static_cast<int>(threadIdx.x) % across, ty = static_cast<int>(threadIdx.x) / across;
  const int high = 256 / across;
  constexpr int kAhead = 4;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * high + ty; row < p.M; row += static_cast<int64_t>(gridDim.x) * high) {
    const int8_t* q = static_cast<const int8_t*>(p.x) + row * p.ldx;
    TO* y = static_cast<TO*>(p.y) + row * p.ldy;
    const uint32_t bytes = static_cast<uint32_t>(reinterpret_cast<uint64_t>(y)) & (4 * sizeof(TO) - 1);
    const float s = p.scale[row];
    // Whole warps take part in every step, up to the row's last column.
    for (int c0 = 0; c0 < p.K; c0 += across * 4 * kAhead) {
      uint32_t word[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int c = c0 + 4 * (tx + k * across);
        word[k] = 0;
        if (Q_ALIGNED && c + 4 <= p.K) {
          word[k] = *reinterpret_cast<const uint32_t*>(q + c);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i < p.K) word[k] |= (static_cast<uint32_t>(q[c + i]) & 0xffu) << (8 * i);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        store_warp_quads<TO, ALIGNED, false>(y, bytes, c0 + 4 * (tx + k * across), p.K, pack4(dequantize4(word[k], s), TO()));
    }
  }
}

}  // namespace twell
