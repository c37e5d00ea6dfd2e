// Layer norm's backward pass (kernels).
//
// With xh = (x - mu) r and g = dy w:
//   dx = r (g - (sum g + xh sum g xh) / D),   dw = sum_rows dy xh,   db = sum_rows dy.
// dw and db want a thread to keep its columns over many rows, the two sums over
// a row want few threads per row.  So a block takes batches of `rows` rows
// through a ring of shared-memory slots (bulk copies, one per row and input,
// several batches ahead) and goes over each batch twice, in shared memory:
// first one or a few warps per row form its sums, then every thread takes its
// own columns of all the rows, adds to its dw and db in registers and writes
// dx.  Bound by HBM for fp32 rows, by instruction issue for 16-bit ones.
// Batches are dealt to blocks in a fixed way, so the order of every sum depends
// on the sizes alone.  Each block writes one partial row of dw and db; a second
// kernel adds those.
#pragma once

#include "rows.cuh"

namespace twell {

// ---------------------------------------------------------------- quads
// Four consecutive elements.
struct Quad {
  float e[4];
};
__device__ __forceinline__ Quad load4(const float* p) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  return Quad{{v.x, v.y, v.z, v.w}};
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

template <class T>
__device__ __forceinline__ Quad load_quad(const T* p, uint32_t past, bool aligned) {
  return aligned ? load4(p) : load4_at(p, past);
}

// ALIGNED: the rows of x, dy and dx start on 16 bytes and have whole quads.
template <class TX, class TDY, int NL, bool ALIGNED>
__global__ void __launch_bounds__(kBwdThreads, NL == 2 ? 2 : 1)
    layer_norm_bwd_kernel(const LayerNormBwdParams p, const BatchPlan plan) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kMaxSlots];
  __shared__ float2 sums[kMaxBatch][kBwdThreads / 32];  // per row and warp of the row
  __shared__ float2 stats[kMaxBatch];                   // mean, rstd
  __shared__ float4 factors[kMaxBatch];                 // mu, r, -r sum g / D, -r sum g xh / D
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
  stage_vector(p.weight, p.w_type, 1.f, p.D, padded, w, [](int c) { return c; });

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
    for (int r = first_row; r < rows; r += high) {
      const float2 st = stats[r];
      // Where the rows start in their slots (0 when ALIGNED).
      const uint32_t xo = ALIGNED ? 0 : static_cast<uint32_t>(x_base + (row0 + r) * x_ld) & 15;
      const uint32_t dyo = ALIGNED ? 0 : static_cast<uint32_t>(dy_base + (row0 + r) * dy_ld) & 15;
      const TX* x = reinterpret_cast<const TX*>(at + r * row_slot + xo);
      const TDY* dy = reinterpret_cast<const TDY*>(at + r * row_slot + x_slot + dyo);
      float s1[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
      const int across = 128 * per_row;
#pragma unroll 4
      for (int c = 4 * (my_part * 32 + lane); c + 4 <= p.D; c += across) {
        const Quad qx = load_quad(x + c, xo, ALIGNED), qd = load_quad(dy + c, dyo, ALIGNED), qw = load4(w + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float gr = qd.e[i] * qw.e[i];
          s1[i] += gr;
          s2[i] = fmaf(gr, (qx.e[i] - st.x) * st.y, s2[i]);
        }
      }
      if (!ALIGNED) {
        const int tail = (p.D & ~3) + lane;
        if (my_part == 0 && tail < p.D) {
          const float gr = to_f32(dy[tail]) * w[tail];
          s1[0] += gr;
          s2[0] += gr * ((to_f32(x[tail]) - st.x) * st.y);
        }
      }
      float2 s = make_float2(warp_sum((s1[0] + s1[1]) + (s1[2] + s1[3])), warp_sum((s2[0] + s2[1]) + (s2[2] + s2[3])));
      if (!ok) s.x = __uint_as_float(0x7fc00000u);
      if (lane == 0) {
        if (per_row == 1)
          factors[r] = make_float4(st.x, st.y, -st.y * (s.x * p.inv_d), -st.y * (s.y * p.inv_d));
        else
          sums[r][my_part] = s;
      }
    }
    __syncthreads();
    if (per_row > 1) {
      if (t < rows) {
        const float2 st = stats[t];
        float2 s = sums[t][0];
        for (int k = 1; k < per_row; ++k) {
          s.x += sums[t][k].x;
          s.y += sums[t][k].y;
        }
        factors[t] = make_float4(st.x, st.y, -st.y * (s.x * p.inv_d), -st.y * (s.y * p.inv_d));
      }
      __syncthreads();
    }
    // dx = r g - r sum g / D - xh r sum g xh / D
    {
      Quad qw[NL];
#pragma unroll
      for (int j = 0; j < NL; ++j) qw[j] = load4(w + 4 * (t + j * nt));
      const uint8_t* xr = at;
      TX* dx = static_cast<TX*>(p.dx) + static_cast<int64_t>(row0) * p.lddx;
#pragma unroll 1
      for (int r = 0; r < rows; ++r, xr += row_slot, dx += p.lddx) {
        const float4 f = factors[r];
        const uint32_t xo = ALIGNED ? 0 : static_cast<uint32_t>(x_base + (row0 + r) * x_ld) & 15;
        const uint32_t dyo = ALIGNED ? 0 : static_cast<uint32_t>(dy_base + (row0 + r) * dy_ld) & 15;
        const uint32_t dxo = ALIGNED ? 0 : static_cast<uint32_t>(reinterpret_cast<uint64_t>(dx)) & (4 * sizeof(TX) - 1);
        const TX* x = reinterpret_cast<const TX*>(xr + xo);
        const TDY* dy = reinterpret_cast<const TDY*>(xr + x_slot + dyo);
#pragma unroll
        for (int j = 0; j < NL; ++j) {
          const int c = 4 * (t + j * nt);
          Quad qx{{0.f, 0.f, 0.f, 0.f}}, qd = qx, out;
          if (c + 4 <= p.D) {
            qx = load_quad(x + c, xo, ALIGNED);
            qd = load_quad(dy + c, dyo, ALIGNED);
          } else if (!ALIGNED) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c + i < p.D) {
                qx.e[i] = to_f32(x[c + i]);
                qd.e[i] = to_f32(dy[c + i]);
              }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float xh = (qx.e[i] - f.x) * f.y;
            dw[j].e[i] = fmaf(qd.e[i], xh, dw[j].e[i]);
            db[j].e[i] += qd.e[i];
            out.e[i] = fmaf(xh, f.w, fmaf(qd.e[i] * qw[j].e[i], f.y, f.z));
          }
          store_warp_quads<TX, ALIGNED, false>(dx, dxo, c, p.D, pack4(out, TX()));
        }
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
        const int c = 4 * (t + j * nt) + i;
        if (c < p.D) {
          out[c] = dw[j].e[i];
          out[p.D + c] = db[j].e[i];
        }
      }
  }
}

}  // namespace twell
