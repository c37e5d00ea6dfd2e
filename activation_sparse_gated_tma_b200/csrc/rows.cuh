// Kernels over rows of activations: layer norm and the quantisation of rows to
// int8 with one scale each.
//
// All are bound by HBM: each row is read once, kept in registers and written
// once.  What competes with the copies is instruction issue (at 6.5 TB/s an SM
// has 450 cycles for a bf16 row of 2560), so the work per row that does not
// depend on its length is kept small: a row belongs to as few warps as hold it
// (one up to 2560 columns for the norm), more only while rows are too few for
// the warps; 16-byte loads and stores, and 16 to 32 warps per SM, are all the
// memory parallelism it takes.  Measured at 16384 x 2560: norm bf16 to bf16 32 us
// (5.2 TB/s; five warps per row 68, rows through a shared-memory ring of bulk
// copies 36), fp32 to bf16 45 us (5.6 TB/s), bf16 to int8 40 us; at 8192 x 5632,
// bf16 to int8 rows 24 us (5.7 TB/s) and back 25.
//
// Columns of thread t in a group of T threads, layer j < NC, i < 8: 8 (t + j T) + i.
// Rows that do not start on 16 bytes are read in aligned pieces, which
// neighbouring lanes join, and written the same way; only what lies outside
// the whole pieces at the ends of a warp's stretch goes by elements.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

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

__device__ __forceinline__ float2 unpack2(uint32_t u, __nv_bfloat16) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t u, __half) {
  union { uint32_t u; __half2 h; } c;
  c.u = u;
  return __half22float2(c.h);
}

// ---------------------------------------------------------------- chunks of eight elements
struct Oct {
  float e[8];
};
// Eight elements as 16-byte pieces (8-byte ones of int8).
template <class T>
struct Chunk {
  using Piece = uint4;
  static constexpr int kPieces = sizeof(T) == 4 ? 2 : 1;
  static constexpr int kElements = 16 / sizeof(T);  // of a piece
  Piece p[kPieces];
};
template <>
struct Chunk<int8_t> {
  using Piece = uint2;
  static constexpr int kPieces = 1;
  static constexpr int kElements = 8;
  Piece p[1];
};
__device__ __forceinline__ Oct unpack8(const Chunk<float>& c) {
  return Oct{{__uint_as_float(c.p[0].x), __uint_as_float(c.p[0].y), __uint_as_float(c.p[0].z), __uint_as_float(c.p[0].w),
              __uint_as_float(c.p[1].x), __uint_as_float(c.p[1].y), __uint_as_float(c.p[1].z), __uint_as_float(c.p[1].w)}};
}
template <class T>
__device__ __forceinline__ Oct unpack8(const Chunk<T>& c) {
  const float2 a = unpack2(c.p[0].x, T()), b = unpack2(c.p[0].y, T()), d = unpack2(c.p[0].z, T()), f = unpack2(c.p[0].w, T());
  return Oct{{a.x, a.y, b.x, b.y, d.x, d.y, f.x, f.y}};
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  union { uint32_t u; __nv_bfloat162 h; } c;
  c.h = __floats2bfloat162_rn(a, b);
  return c.u;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  union { uint32_t u; __half2 h; } c;
  c.h = __floats2half2_rn(a, b);
  return c.u;
}
template <class T>
__device__ __forceinline__ Chunk<T> pack8(const Oct& v) {
  Chunk<T> c;
  if constexpr (sizeof(T) == 4) {
    c.p[0] = make_uint4(__float_as_uint(v.e[0]), __float_as_uint(v.e[1]), __float_as_uint(v.e[2]), __float_as_uint(v.e[3]));
    c.p[1] = make_uint4(__float_as_uint(v.e[4]), __float_as_uint(v.e[5]), __float_as_uint(v.e[6]), __float_as_uint(v.e[7]));
  } else {
    c.p[0] = make_uint4(pack2(v.e[0], v.e[1], T()), pack2(v.e[2], v.e[3], T()), pack2(v.e[4], v.e[5], T()),
                        pack2(v.e[6], v.e[7], T()));
  }
  return c;
}
template <class T>
__device__ __forceinline__ T chunk_element(const Chunk<T>& c, int i) {
  union { Chunk<T> c; T e[8]; } u;
  u.c = c;
  return u.e[i];
}

// The 16 (8) bytes that start `s` bytes into lo; s below a piece's size, the same for all lanes.
__device__ __forceinline__ uint4 bytes_from(uint4 lo, uint4 hi, uint32_t s) {
  const bool two = s & 8, one = s & 4;
  const uint32_t a0 = two ? lo.z : lo.x, a1 = two ? lo.w : lo.y, a2 = two ? hi.x : lo.z, a3 = two ? hi.y : lo.w,
                 a4 = two ? hi.z : hi.x, a5 = two ? hi.w : hi.y;
  const uint32_t b0 = one ? a1 : a0, b1 = one ? a2 : a1, b2 = one ? a3 : a2, b3 = one ? a4 : a3, b4 = one ? a5 : a4;
  const uint32_t bits = 8 * (s & 3);
  return make_uint4(__funnelshift_r(b0, b1, bits), __funnelshift_r(b1, b2, bits), __funnelshift_r(b2, b3, bits),
                    __funnelshift_r(b3, b4, bits));
}
__device__ __forceinline__ uint2 bytes_from(uint2 lo, uint2 hi, uint32_t s) {
  const uint32_t a = s & 4 ? lo.y : lo.x, b = s & 4 ? hi.x : lo.y, c = s & 4 ? hi.y : hi.x, bits = 8 * (s & 3);
  return make_uint2(__funnelshift_r(a, b, bits), __funnelshift_r(b, c, bits));
}
__device__ __forceinline__ uint4 from_lane(uint4 v, int lane) {
  return make_uint4(__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.y, lane),
                    __shfl_sync(0xffffffffu, v.z, lane), __shfl_sync(0xffffffffu, v.w, lane));
}
__device__ __forceinline__ uint2 from_lane(uint2 v, int lane) {
  return make_uint2(__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.y, lane));
}
template <class T>
__device__ __forceinline__ uint32_t bytes_past(const T* row) {
  return static_cast<uint32_t>(reinterpret_cast<uint64_t>(row)) & (sizeof(typename Chunk<T>::Piece) - 1);
}

// A whole chunk in one access: 16 bytes of 16-bit elements, 32 of fp32 (backward
// fp32 16384 x 2560: 84 us, as two of 16 88).
__device__ __forceinline__ Chunk<float> load_whole(const float* p) {
  Chunk<float> v;
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v.p[0].x), "=r"(v.p[0].y), "=r"(v.p[0].z), "=r"(v.p[0].w), "=r"(v.p[1].x), "=r"(v.p[1].y),
                 "=r"(v.p[1].z), "=r"(v.p[1].w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void store_whole(float* p, const Chunk<float>& v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.p[0].x), "r"(v.p[0].y),
               "r"(v.p[0].z), "r"(v.p[0].w), "r"(v.p[1].x), "r"(v.p[1].y), "r"(v.p[1].z), "r"(v.p[1].w)
               : "memory");
}
template <class T>
__device__ __forceinline__ Chunk<T> load_whole(const T* p) {
  Chunk<T> v;
  v.p[0] = *reinterpret_cast<const typename Chunk<T>::Piece*>(p);
  return v;
}
template <class T>
__device__ __forceinline__ void store_whole(T* p, const Chunk<T>& v) {
  *reinterpret_cast<typename Chunk<T>::Piece*>(p) = v.p[0];
}

// This lane's chunk, at column c, of a row of D elements in global memory;
// columns from D on are 0.  FULL: no lane of the warp reaches D.  ALIGNED rows
// start on whole chunks' sizes and have whole chunks.  Else the row starts `past` bytes
// behind a piece, and pieces that hold bytes of the row are read whole (rows
// for which one would reach outside the matrix are not read this way).
template <class T, bool ALIGNED, bool FULL>
__device__ __forceinline__ Chunk<T> load_chunk(const T* row, uint32_t past, int c, int D) {
  using C = Chunk<T>;
  using Piece = typename C::Piece;
  C v = {};
  if (ALIGNED) {
    if (FULL || c < D) v = load_whole(row + c);
    return v;
  }
  const int lane = threadIdx.x & 31;
  const int skip = static_cast<int>(past / sizeof(T));
  const Piece* at = reinterpret_cast<const Piece*>(reinterpret_cast<const uint8_t*>(row + c) - past);
#pragma unroll
  for (int i = 0; i < C::kPieces; ++i)
    if (FULL || c + i * C::kElements - skip < D) v.p[i] = at[i];
  if (past) {
    // The piece behind this lane's: the next lane's first, or one more load.
    Piece next = from_lane(v.p[0], lane + 1);
    if (lane == 31) {
      next = Piece{};
      if (c + 8 - skip < D) next = at[C::kPieces];
    }
#pragma unroll
    for (int i = 0; i < C::kPieces; ++i) v.p[i] = bytes_from(v.p[i], i + 1 < C::kPieces ? v.p[i + 1] : next, past);
  }
  if (!FULL && c + 8 > D) {
    union { C c; T e[8]; } u;
    u.c = v;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i >= D) u.e[i] = from_f32<T>(0.f);
    v = u.c;
  }
  return v;
}
// The same by elements.
template <class T>
__device__ __forceinline__ Chunk<T> load_elements(const T* row, int c, int D) {
  union { Chunk<T> c; T e[8]; } u;
  u.c = {};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < D) u.e[i] = row[c + i];
  return u.c;
}

// A warp's 32 neighbouring chunks (this lane's at column c) to a row of global
// memory; the whole warp calls it.  Terms as above.
template <class T, bool ALIGNED, bool FULL>
__device__ __forceinline__ void store_chunk(T* row, uint32_t past, int c, int D, const Chunk<T>& v) {
  using C = Chunk<T>;
  using Piece = typename C::Piece;
  if (ALIGNED) {
    if (FULL || c < D) store_whole(row + c, v);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int first = c - 8 * lane, n = FULL ? 256 : min(256, D - first);  // the warp's stretch
  if (n <= 0) return;
  const int s = static_cast<int>(past / sizeof(T));
  const Piece before = from_lane(v.p[C::kPieces - 1], lane - 1);
  // Piece g of the stretch holds its elements [kElements g - s, kElements (g + 1) - s).
#pragma unroll
  for (int i = 0; i < C::kPieces; ++i) {
    const int e0 = 8 * lane + i * C::kElements - s;
    if (e0 >= 0 && e0 + C::kElements <= n) {
      const Piece lo = i == 0 ? before : v.p[i > 0 ? i - 1 : 0];
      *reinterpret_cast<Piece*>(row + first + e0) =
          past ? bytes_from(lo, v.p[i], static_cast<uint32_t>(sizeof(Piece)) - past) : v.p[i];
    }
  }
  const int head = s ? C::kElements - s : 0;                        // elements before the first whole piece
  const int tail = (n + s) / C::kElements * C::kElements - s;       // from here on, behind the last
  if (8 * lane < head || 8 * lane + 8 > tail) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = 8 * lane + i;
      if ((e < head || e >= tail) && e < n) row[c + i] = chunk_element(v, i);
    }
  }
}

// ---------------------------------------------------------------- a thread's part of a row
// NC chunks, the smallest of 1, 2, 3, 4, 5, 6, 8, 10 that covers the row, so
// that many of the layers are full.
__host__ __device__ constexpr int full_layers(int NC) { return NC > 6 ? NC - 2 : NC - 1; }
template <class T, int NC>
struct RowPart {
  Chunk<T> c[NC];
};
template <class T, int NC, bool ALIGNED>
__device__ __forceinline__ void load_row(const T* row, bool whole_pieces, int D, int t, int nt, RowPart<T, NC>& r) {
  if (ALIGNED || whole_pieces) {
    const uint32_t past = bytes_past(row);
#pragma unroll
    for (int j = 0; j < NC; ++j)
      r.c[j] = j < full_layers(NC) ? load_chunk<T, ALIGNED, true>(row, past, 8 * (t + j * nt), D)
                                   : load_chunk<T, ALIGNED, false>(row, past, 8 * (t + j * nt), D);
  } else {
#pragma unroll
    for (int j = 0; j < NC; ++j) r.c[j] = load_elements(row, 8 * (t + j * nt), D);
  }
}
template <class T, int NC, bool ALIGNED>
__device__ __forceinline__ void store_layer(T* row, uint32_t past, int D, int t, int nt, int j, const Chunk<T>& v) {
  if (j < full_layers(NC))
    store_chunk<T, ALIGNED, true>(row, past, 8 * (t + j * nt), D, v);
  else
    store_chunk<T, ALIGNED, false>(row, past, 8 * (t + j * nt), D, v);
}

// Asks for a row in L2, one thread for the whole row, ahead of its loads (rows
// whose aligned pieces lie inside the matrix only): the loads then wait for L2
// instead of DRAM, at no cost in registers.
template <class T>
__device__ __forceinline__ void prefetch_row(const T* row, int D) {
  const uint64_t a = reinterpret_cast<uint64_t>(row), at = a & ~uint64_t(15);
  const uint32_t bytes = (static_cast<uint32_t>(a - at) + D * static_cast<uint32_t>(sizeof(T)) + 15u) & ~15u;
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
}

// A parameter vector of D elements into `padded` floats of shared memory, by
// the whole block, several loads in flight; `fill` where p is NULL, 0 from D
// on.  nt > 0: each layer of 8 nt columns with the first halves of its chunks
// before the second ones.  (Not inlined: the kernels have no registers to spare.)
template <class T>
__device__ __forceinline__ void stage_typed(const T* p, float fill, int D, int padded, float* to, int nt) {
  constexpr int kAhead = 8;
  for (int c0 = threadIdx.x; c0 < padded; c0 += kAhead * blockDim.x) {
    float e[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int c = c0 + k * blockDim.x;
      e[k] = c >= D ? 0.f : p ? to_f32(p[c]) : fill;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      int c = c0 + k * blockDim.x;
      if (c >= padded) break;
      if (nt > 0) {
        const int layer = c / (8 * nt), in = c - layer * 8 * nt;
        c = layer * 8 * nt + ((in >> 2) & 1) * 4 * nt + (in >> 3) * 4 + (in & 3);
      }
      to[c] = e[k];
    }
  }
}
static __device__ __noinline__ void stage_vector(const void* p, int type, float fill, int D, int padded, float* to, int nt) {
  if (type == TWELL_F32)
    stage_typed(static_cast<const float*>(p), fill, D, padded, to, nt);
  else if (type == TWELL_BF16)
    stage_typed(static_cast<const __nv_bfloat16*>(p), fill, D, padded, to, nt);
  else
    stage_typed(static_cast<const __half*>(p), fill, D, padded, to, nt);
}

// ---------------------------------------------------------------- groups
// A block holds blockDim.x / T groups of T = 32 W threads, each on its own
// rows with its own named barrier and reduction buffers.
struct Group {
  int warps, t, nt, id;  // warps per row, thread in the group, threads in the group, group in the block
  int flip;
  float* buf;            // [2][8] of this group
};
struct GroupShared {
  float buf[kMaxGroups][2][kMaxGroupWarps];
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

// Group-wide sum in a fixed order, or maximum of magnitudes (by their bits,
// under which a NaN is above infinity); every thread gets it.  Consecutive
// reductions alternate between two shared buffers, so one barrier each is
// enough: a thread that writes a buffer again has passed the barrier of the
// reduction in between, which every thread reaches only after it has read the buffer.
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

// ---------------------------------------------------------------- quantisation
// One row's scale.  q is the integer nearest to 127 x / amax, ties to even,
// exactly, found by adding 1.5 * 2^23, which rounds to an integer held in the
// sum's low byte.
// fp32 values: 127 / amax in fp32 is within 2^-24 of the quotient's factor, so
// the true quotient lies between x low and x high, low and high 2^-22 below and
// above it.  Where both round to the same integer that is the answer, else the
// sign of 254 x - (2 q + 1) amax decides between q and q + 1.
// 16-bit values (NARROW): ties are frequent (x = amax / 2 is one), but what is
// none is far from one.  254 x - (2 q + 1) amax is a multiple of x's last bit and
// x has 11 bits at most, so a quotient next to a tie is off by at least
// 1 / (254 * 2047) of it: 16 units of its last fp32 place.  The factor
// (127 + 2^-15) / amax puts x's product (2.016 -+ 0.5) m -+ 0.5 units, 1 <= m < 2,
// above the true quotient (0.5 m the factor's rounding, 0.5 the product's), and
// clearing the last three bits takes a tie back to itself and all others to their side of it.
// Rows near either end of the exponents' range are scaled by 2^100 or 2^-100
// first.  A row with a NaN or an infinity gets scale NaN and q = 0, one of zeros scale 0.
struct RowScale {
  float amax, low, high, scale, up;
  bool none;
};
template <bool NARROW>
__device__ __forceinline__ RowScale row_scale(float amax) {
  RowScale r;
  const bool finite = amax <= 3.402823466e38f;  // a NaN is not
  r.scale = finite ? amax / 127.f : __uint_as_float(0x7fc00000u);
  r.none = !finite || amax == 0.f;
  r.up = amax < 0x1p-100f ? 0x1p100f : amax > 0x1p100f ? 0x1p-100f : 1.f;
  r.amax = amax * r.up;
  if (NARROW) {
    r.low = r.high = (127.f + 0x1p-15f) / r.amax;
  } else {
    const float inv = 127.f / r.amax;
    r.low = inv * (1.f - 0x1p-22f);
    r.high = inv * (1.f + 0x1p-22f);
  }
  return r;
}
__device__ __forceinline__ uint32_t pack_low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// t = 254 x - (2 q + 1) amax from the products' roundings and what those leave
// (Dekker's two-product by fused multiply-add): near a tie the two products are
// neighbours, so their difference is exact, and a non-zero t is at least 2^-33 of them.
__device__ __forceinline__ uint32_t nearest(float x, uint32_t a, uint32_t b, float amax) {
  const int q = min(static_cast<int>(a), static_cast<int>(b)) - 0x4b400000;
  const float k = static_cast<float>(2 * q + 1);
  const float px = 254.f * x, pa = k * amax;
  const float t = (px - pa) + (fmaf(254.f, x, -px) - fmaf(k, amax, -pa));
  return static_cast<uint32_t>(q + (a != b && (t > 0.f || (t == 0.f && (q & 1))) ? 1 : 0));
}
// Eight values to eight bytes.
template <bool NARROW>
__device__ __forceinline__ uint2 quantize8(Oct v, const RowScale& r) {
  if (r.none) return make_uint2(0, 0);
  if (r.up != 1.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v.e[i] *= r.up;
  }
  uint32_t q[8];
  if constexpr (NARROW) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      q[i] = __float_as_uint(__uint_as_float(__float_as_uint(v.e[i] * r.low) & ~7u) + 12582912.f);
  } else {
    uint32_t h[8], differ = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = __float_as_uint(fmaf(v.e[i], r.low, 12582912.f));
      h[i] = __float_as_uint(fmaf(v.e[i], r.high, 12582912.f));
      differ |= q[i] ^ h[i];
    }
    if (differ) {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = nearest(v.e[i], q[i], h[i], r.amax);
    }
  }
  return make_uint2(pack_low_bytes(q[0], q[1], q[2], q[3]), pack_low_bytes(q[4], q[5], q[6], q[7]));
}
// The larger magnitude; a NaN stays one.
__device__ __forceinline__ float max_abs(float m, float v) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(m), "f"(fabsf(v)));
  return d;
}
__device__ __forceinline__ float max_abs(float m, const Oct& v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_abs(m, v.e[i]);
  return m;
}
// Over the chunks of a row; 16-bit elements two at a time as they are packed.
template <class T, int NC>
__device__ __forceinline__ float max_abs(RowPart<T, NC>& r) {
  if constexpr (sizeof(T) == 4) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) m = max_abs(m, unpack8(r.c[j]));
    return m;
  } else {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    union { uint32_t u; T2 v; } m, e;
    m.u = 0;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const uint32_t w[4] = {r.c[j].p[0].x, r.c[j].p[0].y, r.c[j].p[0].z, r.c[j].p[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e.u = w[i] & 0x7fff7fffu;
        m.v = __hmax2_nan(m.v, e.v);
      }
    }
    const float2 f = unpack2(m.u, T());
    return max_abs(f.x, f.y);
  }
}
// This thread's elements of a row, layer j's given by get(j), to int8 and into the row.
template <int NC, bool ALIGNED, bool NARROW, class Get>
__device__ __forceinline__ void store_row_i8(int8_t* row, int D, int t, int nt, const RowScale& r, Get get) {
  const uint32_t past = bytes_past(row);
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    Chunk<int8_t> q;
    q.p[0] = quantize8<NARROW>(get(j), r);
    store_layer<int8_t, NC, ALIGNED>(row, past, D, t, nt, j, q);
  }
}

// ---------------------------------------------------------------- layer norm
// mu = sum x / D, v = sum (x - mu)^2 / D, r = 1 / sqrt(v + eps),
// y = (x - mu) r w + b.  The variance is taken from the deviations (two
// reductions over registers, no second read): sums of squares would cancel for
// rows whose mean is far above their spread (as x r - mu r would, where x - mu is
// exact); of such rows the mean is corrected by the deviations' own.  TO int8_t:
// y is quantised from its fp32 values, with one more reduction for the row's
// largest magnitude.
// The weight and the bias are staged in shared memory once per block (from
// global memory every row's reads cost 4 us at bf16 16384 x 2560), each layer's first and
// second halves of chunks apart, so that the lanes' 16-byte reads meet
// different banks.
template <class TI, class TO, int NC, bool ALIGNED>
__global__ void __launch_bounds__(kRowThreads, norm_blocks(NC))
    layer_norm_kernel(const LayerNormParams p, const RowPlan plan) {
  extern __shared__ __align__(16) float vectors[];
  __shared__ GroupShared sh;
  Group g = make_group(plan.warps, sh);
  const uint32_t groups = blockDim.x / g.nt, step = gridDim.x * groups;
  const int padded = 8 * NC * g.nt;  // whole layers, read without a check
  griddep_launch_dependents();
  griddep_wait();
  // The first row on its way while the vectors are staged.
  if (g.t == 0 && plan.whole_pieces(blockIdx.x * groups + g.id))
    prefetch_row(static_cast<const TI*>(p.x) + (blockIdx.x * groups + g.id) * p.ldx, p.D);
  stage_vector(p.weight, p.w_type, 1.f, p.D, padded, vectors, g.nt);
  stage_vector(p.bias, p.w_type, 0.f, p.D, padded, vectors + padded, g.nt);
  __syncthreads();
  for (uint32_t row = blockIdx.x * groups + g.id; row < p.M; row += step) {
    Oct v[NC];
    {
      RowPart<TI, NC> raw;
      load_row<TI, NC, ALIGNED>(static_cast<const TI*>(p.x) + row * p.ldx, plan.whole_pieces(row), p.D, g.t, g.nt, raw);
      // (Rows of many chunks keep enough loads in flight by themselves: bf16 16384 x 2560 took 3 us more with it.)
      if ((!ALIGNED || NC <= 2) && g.t == 0 && plan.whole_pieces(row + step))
        prefetch_row(static_cast<const TI*>(p.x) + (row + step) * p.ldx, p.D);
#pragma unroll
      for (int j = 0; j < NC; ++j) v[j] = unpack8(raw.c[j]);
    }
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i & 3] = fmaf(v[j].e[i], 0x1p-15f, s[i & 3]);
    // (Of at most 2^14 elements at 2^-15 the sum stays within the range.  Rounding may still take the mean of rows of
    // the largest value out of it.)
    float mean = group_sum(g, (s[0] + s[1]) + (s[2] + s[3])) * (p.inv_d * 0x1p15f);
    if (fabsf(mean) > 3.402823466e38f) mean = copysignf(3.402823466e38f, mean);
    auto take_off = [&](float d) {
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j].e[i] -= d;
    };
    // Sum over the row of f(deviation) added up in turn (behind the row they are 0 - mean).
    auto sum_of = [&](auto f) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int c = 8 * (g.t + j * g.nt);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (j < full_layers(NC) || c + (ALIGNED ? 0 : i) < p.D) s[i & 3] = f(s[i & 3], v[j].e[i]);
      }
      return group_sum(g, (s[0] + s[1]) + (s[2] + s[3]));
    };
    auto plus_square = [](float s, float d) { return fmaf(d, d, s); };
    take_off(mean);
    float rstd = rsqrtf(sum_of(plus_square) * p.inv_d + p.eps);
    // This mean is off by a few 2^-24 of itself: where it is far above the spread, by much of a deviation (or so much
    // that the squares pass the range and leave no rstd).  The deviations' own mean, off by as little of itself, takes
    // that off again.  The whole group does or does not.  (fp32 to bf16 16384 x 2560 takes 42 us whether all rows do or
    // none; the check itself costs bf16 65536 x 256 18.8 us for 17.9, 8192 x 4096 32.1 for 30.7, 16384 x 2560 nothing.)
    if (fabsf(mean) * rstd > 4.f || rstd == 0.f) {
      const float off = sum_of([](float s, float d) { return s + d; }) / static_cast<float>(p.D);
      mean += off;
      take_off(off);
      rstd = rsqrtf(sum_of(plus_square) * p.inv_d + p.eps);
    }
    auto result = [&](int j) {
      const float* w = vectors + 8 * j * g.nt + 4 * g.t;
      const float4 wa = *reinterpret_cast<const float4*>(w), wb = *reinterpret_cast<const float4*>(w + 4 * g.nt);
      const float4 ba = *reinterpret_cast<const float4*>(w + padded), bb = *reinterpret_cast<const float4*>(w + padded + 4 * g.nt);
      const float wv[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
      const float bv[8] = {ba.x, ba.y, ba.z, ba.w, bb.x, bb.y, bb.z, bb.w};
      Oct o;
#pragma unroll
      for (int i = 0; i < 8; ++i) o.e[i] = fmaf(v[j].e[i] * rstd, wv[i], bv[i]);
      return o;
    };
    TO* y = static_cast<TO*>(p.y) + row * p.ldy;
    if constexpr (sizeof(TO) == 1) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        v[j] = result(j);
        const int c = 8 * (g.t + j * g.nt);
        // Behind the row (0 - mean) rstd may pass the fp32 range, which the weight of 0 there makes a NaN.
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (j < full_layers(NC) || c + (ALIGNED ? 0 : i) < p.D) m = max_abs(m, v[j].e[i]);
      }
      const RowScale r = row_scale<false>(group_max(g, m));
      store_row_i8<NC, ALIGNED, false>(y, p.D, g.t, g.nt, r, [&](int j) { return v[j]; });
      if (g.t == 0) p.y_scale[row] = r.scale;
    } else {
      const uint32_t past = bytes_past(y);
#pragma unroll
      for (int j = 0; j < NC; ++j) store_layer<TO, NC, ALIGNED>(y, past, p.D, g.t, g.nt, j, pack8<TO>(result(j)));
    }
    if (g.t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
  }
}

// ---------------------------------------------------------------- rows to int8 and back
// The row stays packed in registers (few enough for 32 warps per SM of 16-bit rows up to six chunks) and is unpacked twice.
template <class TI, int NC, bool ALIGNED>
__global__ void __launch_bounds__(kRowThreads, quantize_blocks(NC, sizeof(TI)))
    quantize_rows_kernel(const QuantizeParams p, const RowPlan plan) {
  __shared__ GroupShared sh;
  Group g = make_group(plan.warps, sh);
  const uint32_t groups = blockDim.x / g.nt, step = gridDim.x * groups;
  griddep_launch_dependents();
  griddep_wait();
  for (uint32_t row = blockIdx.x * groups + g.id; row < p.M; row += step) {
    RowPart<TI, NC> v;
    load_row<TI, NC, ALIGNED>(static_cast<const TI*>(p.x) + row * p.ldx, plan.whole_pieces(row), p.K, g.t, g.nt, v);
    if ((!ALIGNED || NC <= 2) && g.t == 0 && plan.whole_pieces(row + step))
      prefetch_row(static_cast<const TI*>(p.x) + (row + step) * p.ldx, p.K);
    const RowScale r = row_scale<sizeof(TI) == 2>(group_max(g, max_abs(v)));
    store_row_i8<NC, ALIGNED, sizeof(TI) == 2>(static_cast<int8_t*>(p.y) + row * p.ldy, p.K, g.t, g.nt, r,
                              [&](int j) { return unpack8(v.c[j]); });
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
    const RowScale r = row_scale<sizeof(TI) == 2>(group_max(g, m));
    for (int c = g.t; c < p.K; c += 8 * kRowThreads) {
      Oct v;
#pragma unroll
      for (int i = 0; i < 8; ++i) v.e[i] = c + i * kRowThreads < p.K ? to_f32(x[c + i * kRowThreads]) : 0.f;
      Chunk<int8_t> q;
      q.p[0] = quantize8<sizeof(TI) == 2>(v, r);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i * kRowThreads < p.K) y[c + i * kRowThreads] = chunk_element(q, i);
    }
    if (g.t == 0) p.scale[row] = r.scale;
  }
}

// x = q s.  A block takes a segment of `across` chunks of 4 * 256 / across rows,
// a thread the same chunk of four of them, so that its loads are in flight
// together whatever the row's length (with neighbouring chunks of one row
// instead, rows of 256 took 19 us for 65536 and rows of 2560 30 us for 16384).
// A byte becomes fp32 without a conversion: with its sign bit flipped it is
// the last byte of 2^23 + q + 128.
__device__ __forceinline__ Oct dequantize8(uint2 word, float s) {
  const uint32_t u[2] = {word.x ^ 0x80808080u, word.y ^ 0x80808080u};
  Oct v;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v.e[i] = (__uint_as_float(__byte_perm(u[i >> 2], 0x4b000000u, 0x7440 + (i & 3))) - 8388736.f) * s;  // 2^23 + 128
  return v;
}
// Q_ALIGNED: q's rows start on eight bytes.
template <class TO, bool Q_ALIGNED, bool ALIGNED>
__global__ void __launch_bounds__(256) dequantize_rows_kernel(const QuantizeParams p, int across) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kRows = 4;
  const int tx = static_cast<int>(threadIdx.x) % across, ty = static_cast<int>(threadIdx.x) / across;
  const int high = 256 / across;
  const int64_t step_x = high * p.ldx, step_y = high * p.ldy;
  const int segments = (p.K + 8 * across - 1) / (8 * across);
  for (int segment = blockIdx.x; segment < segments; segment += gridDim.x) {
    const int c = (segment * across + tx) * 8;
    for (int64_t row0 = static_cast<int64_t>(blockIdx.y) * (kRows * high) + ty; row0 < p.M;
         row0 += static_cast<int64_t>(gridDim.y) * (kRows * high)) {  // then every high-th
      const int rows = static_cast<int>(min(static_cast<int64_t>(kRows), (p.M - row0 + high - 1) / high));
      const int8_t* q = static_cast<const int8_t*>(p.x) + row0 * p.ldx;
      TO* y = static_cast<TO*>(p.y) + row0 * p.ldy;
      Chunk<int8_t> in[kRows];
      float s[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r >= rows) break;
        s[r] = p.scale[row0 + r * high];
        if (Q_ALIGNED && c + 8 <= p.K)
          in[r].p[0] = *reinterpret_cast<const uint2*>(q + c);
        else
          in[r] = load_elements(q, c, p.K);
        q += step_x;
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r >= rows) break;
        store_chunk<TO, ALIGNED, false>(y, bytes_past(y), c, p.K, pack8<TO>(dequantize8(in[r].p[0], s[r])));
        y += step_y;
      }
    }
  }
}

}  // namespace twell
