// 8-bit integer products on the tensor cores (tcgen05 kind::i8): int8 rows of
// tokens against int8 rows of weights, one fp32 scale per token and per weight
// row (channel), the sum exact in 32-bit integers.
//
//   y[m][n] = (float(sum_k x[m][k] w[n][k]) * x_scale[m]) * w_scale[n]   (+ bias[n])
//
// Weights sit on the tile's 128-row side (TMEM lanes = channels), tokens on its
// N side (TMEM columns), so a batch of a few tokens takes a tile of 16 columns
// instead of a mostly empty one of 128 rows, and an epilogue warp stores 32
// neighbouring channels of one token at a time.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/twell.h"
#include "int8_gemm.h"
#include "ptx.cuh"

namespace twell {

__device__ __forceinline__ void store_y(void* y, int type, int64_t at, float v) {
  if (type == TWELL_F32)
    static_cast<float*>(y)[at] = v;
  else if (type == TWELL_BF16)
    static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(y)[at] = __float2half_rn(v);
}

// u * ReLU(g); a NaN in g (a token or channel without a scale) stays one.
__device__ __forceinline__ float gated_value(float g, float u) { return g <= 0.f ? 0.f : g * u; }

// ---------------------------------------------------------------------------
// One tile per CTA (128 channels x BT tokens, two accumulators when GATED); a
// cluster of CTAs shares a tile's reduction, each taking a contiguous range of
// its 128-wide k blocks, so that few tiles still occupy every SM.  The partial
// sums are integers: adding them through the cluster's shared memory gives the
// same result in any order.
//   warp 0  TMA producer, warp 1  TMEM + MMA issuer, warps 2-5  epilogue
// At most two CTAs fit an SM (shared memory), with at most 256 TMEM columns
// each, so an allocation never waits for a CTA that waits for this cluster.
template <int BT, bool GATED>
struct Int8SplitSmem {
  static constexpr int kWBytes = kI8ChannelTile * kI8BK;
  static constexpr int kXBytes = BT * kI8BK;
  static constexpr int kStageBytes = kWBytes * (GATED ? 2 : 1) + kXBytes;
  static constexpr int kAccCols = BT * (GATED ? 2 : 1);
  static constexpr int kTmemCols = kAccCols <= 32 ? 32 : kAccCols <= 64 ? 64 : kAccCols <= 128 ? 128 : 256;
  // Partial sums of a shared reduction; the gated tile of 128 tokens has no room for them and is not split.
  static constexpr bool kSplittable = !(GATED && BT == 128);
  static constexpr int kPartialBytes = kSplittable ? kAccCols * kI8ChannelTile * 4 : 0;
  static constexpr int kBudget = 108 * 1024;
  static constexpr int kStages = kBudget / kStageBytes < 6 ? kBudget / kStageBytes : 6;
  static constexpr int kRing = kStages * kStageBytes > kPartialBytes ? kStages * kStageBytes : kPartialBytes;
  static constexpr int kCtrl = (2 * kStages + 1) * 8 + 16 + 4 * BT;
  // At least 78 KB, so that no third CTA fits.
  static constexpr int kTotal = 1024 + kRing + kCtrl > 78 * 1024 ? 1024 + kRing + kCtrl : 78 * 1024;
  static_assert(kStages >= 2 && kTotal <= 113 * 1024, "two CTAs must fit an SM");
};

template <int BT, bool GATED>
__global__ void __launch_bounds__(192) int8_split_kernel(const __grid_constant__ CUtensorMap tm_x,
                                                         const __grid_constant__ CUtensorMap tm_w,
                                                         const __grid_constant__ CUtensorMap tm_w2,
                                                         const Int8GemmParams p, int splits) {
  using L = Int8SplitSmem<BT, GATED>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kRing);
  uint64_t* empty = full + L::kStages;
  uint64_t* tfull = empty + L::kStages;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(tfull + 1);
  int* failed = reinterpret_cast<int*>(tmem_holder + 1);
  float* xs = reinterpret_cast<float*>(tmem_holder + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    *failed = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  griddep_launch_dependents();
  griddep_wait();

  const int split = static_cast<int>(blockIdx.x) % splits;
  const int tile = static_cast<int>(blockIdx.x) / splits;
  const int channel_tiles = (p.N + kI8ChannelTile - 1) / kI8ChannelTile;
  const int n0 = tile % channel_tiles * kI8ChannelTile;
  const int m0 = tile / channel_tiles * BT;
  const int total_kb = (p.K + kI8BK - 1) / kI8BK;
  const int per = (total_kb + splits - 1) / splits;
  const int kb0 = split * per;
  const int kb1 = min(total_kb, kb0 + per);  // the host leaves no split empty

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, nullptr)) break;
        uint8_t* st = smem + stage * L::kStageBytes;
        mbar_arrive_expect_tx(&full[stage], L::kStageBytes);
        tma_load_2d(&tm_w, &full[stage], st, kb * kI8BK, n0);
        if (GATED) tma_load_2d(&tm_w2, &full[stage], st + L::kWBytes, kb * kI8BK, n0);
        tma_load_2d(&tm_x, &full[stage], st + L::kStageBytes - L::kXBytes, kb * kI8BK, m0);
        if (++stage == L::kStages) { stage = 0; phase ^= 1u; }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_i8_s32(kI8ChannelTile, BT);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&full[stage], phase, nullptr)) { ok = false; break; }
        tc_fence_after();
        const uint32_t w = smem_u32(smem + stage * L::kStageBytes);
        const uint32_t x = w + L::kStageBytes - L::kXBytes;
#pragma unroll
        for (int k = 0; k < kI8BK / 32; ++k) {
          const uint32_t accum = (kb > kb0 || k > 0) ? 1u : 0u;
          const uint64_t xd = smem_desc_sw128(x + k * 32, 16, 1024);
          umma_i8(tmem_base, smem_desc_sw128(w + k * 32, 16, 1024), xd, idesc, accum);
          if (GATED) umma_i8(tmem_base + BT, smem_desc_sw128(w + L::kWBytes + k * 32, 16, 1024), xd, idesc, accum);
        }
        umma_commit(&empty[stage]);
        if (++stage == L::kStages) { stage = 0; phase ^= 1u; }
      }
      if (ok) umma_commit(tfull);
    }
  } else {
    const int q = warp & 3;              // TMEM lane quadrant of this warp
    const int row = q * 32 + lane;       // channel in the tile
    const int e = threadIdx.x - 64;
    const int n = n0 + row;
    for (int i = e; i < BT; i += 128) xs[i] = m0 + i < p.M ? p.x_scale[m0 + i] : 0.f;
    const float ws = n < p.N ? p.w_scale[n] : 0.f;
    const float ws2 = GATED && n < p.N ? p.w2_scale[n] : 0.f;
    const float bias = !GATED && p.bias && n < p.N ? p.bias[n] : 0.f;
    named_bar_sync(1, 128);
    if (!mbar_wait(tfull, 0, nullptr)) *failed = 1;
    __syncwarp();
    tc_fence_after();
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    constexpr int kStep = 16;
    if (L::kSplittable && splits > 1) {
      // Every MMA has read the ring: it takes the partial sums, [column][channel].
      int* part = reinterpret_cast<int*>(smem);
#pragma unroll 1
      for (int c = 0; c < L::kAccCols; c += kStep) {
        uint32_t r[kStep];
        tmem_ld_32x32_x16(taddr + c, r);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < kStep; ++j) part[(c + j) * kI8ChannelTile + row] = static_cast<int>(r[j]);
      }
    } else {
      const bool bad = *failed != 0;
#pragma unroll 1
      for (int c = 0; c < BT; c += kStep) {
        uint32_t r[kStep], r2[kStep];
        tmem_ld_32x32_x16(taddr + c, r);
        if (GATED) tmem_ld_32x32_x16(taddr + BT + c, r2);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < kStep; ++j) {
          const int m = m0 + c + j;
          float v = static_cast<float>(static_cast<int>(r[j])) * xs[c + j] * ws;
          if (GATED)
            v = gated_value(v, static_cast<float>(static_cast<int>(r2[j])) * xs[c + j] * ws2);
          else
            v += bias;
          if (bad) v = __uint_as_float(0x7fc00000u);
          if (m < p.M && n < p.N) store_y(p.y, p.y_type, m * p.ldy + n, v);
        }
      }
    }
    tc_fence_before();
    if (splits > 1) {
      // The other half of the exchange, after the cluster's barrier below.
      cluster_sync();
      const int* part = reinterpret_cast<const int*>(smem);
      bool bad = false;
      for (int s = 0; s < splits; ++s) bad |= ld_cluster_s32(mapa_shared(failed, s)) != 0;
      for (int c = split; c < BT; c += splits) {
        const int m = m0 + c;
        if (m >= p.M) break;
        int a = 0, a2 = 0;
        for (int s = 0; s < splits; ++s) {
          a += ld_cluster_s32(mapa_shared(part + c * kI8ChannelTile + row, s));
          if (GATED) a2 += ld_cluster_s32(mapa_shared(part + (BT + c) * kI8ChannelTile + row, s));
        }
        float v = static_cast<float>(a) * xs[c] * ws;
        if (GATED)
          v = gated_value(v, static_cast<float>(a2) * xs[c] * ws2);
        else
          v += bias;
        if (bad) v = __uint_as_float(0x7fc00000u);
        if (n < p.N) store_y(p.y, p.y_type, m * p.ldy + n, v);
      }
    }
  }
  if (splits > 1) {
    __syncwarp();
    if (warp < 2) cluster_sync();  // partial sums written
    cluster_sync();                // and read: shared memory may go
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, L::kTmemCols);
}

}  // namespace twell
