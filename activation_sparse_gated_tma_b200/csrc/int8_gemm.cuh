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

#include <type_traits>

#include "../../include/twell.h"
#include "int8_gemm.h"
#include "ptx.cuh"

namespace twell {

template <class TY>
__device__ __forceinline__ TY to_y(float v) {
  if constexpr (std::is_same<TY, float>::value)
    return v;
  else if constexpr (std::is_same<TY, __nv_bfloat16>::value)
    return __float2bfloat16_rn(v);
  else
    return __float2half_rn(v);
}
// Four values to consecutive elements; `whole`: all four are inside and the address is aligned.
template <class TY>
__device__ __forceinline__ void store4_y(TY* y, const float (&v)[4], int inside, bool whole) {
  union { uint2 u; TY e[4]; float4 f; } c;
#pragma unroll
  for (int i = 0; i < 4; ++i) c.e[i] = to_y<TY>(v[i]);
  if (whole) {
    if constexpr (sizeof(TY) == 4)
      *reinterpret_cast<float4*>(y) = c.f;
    else
      *reinterpret_cast<uint2*>(y) = c.u;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < inside) y[i] = c.e[i];
  }
}

// u * ReLU(g); a NaN in g or u (a token or channel without a scale) stays one.
__device__ __forceinline__ float gated_value(float g, float u) { return (g <= 0.f ? 0.f : g) * u; }

// Waits (again with a limit) for the last `issued` of a ring's loads to land: no
// CTA leaves with copies into it under way, not even after a wait that gave up.
// (stage, phase) is the place after the last one.
template <int STAGES>
__device__ __forceinline__ void wait_loads(uint64_t* full, int issued, int stage, uint32_t phase) {
  for (int k = issued < STAGES ? issued : STAGES; k > 0; --k) {
    const int s = stage - k;
    if (!mbar_wait(&full[s < 0 ? s + STAGES : s], s < 0 ? phase ^ 1u : phase, nullptr)) break;
  }
}

// Every wait is bounded.  A role whose wait gives up stops for good: the MMA
// issuer once its MMAs in flight are done, the producer once its loads have
// landed, and an epilogue warp writes NaN from then on (its later waits could
// find an older phase of a barrier that nothing completes any more).

// ---------------------------------------------------------------------------
// One tile per CTA (128 channels x BT tokens, two accumulators when GATED); a
// cluster of CTAs shares a tile's reduction, each taking a contiguous range of
// its 128-wide k blocks, so that few tiles still occupy every SM.  The partial
// sums are integers: adding them through the cluster's shared memory gives the
// same result in any order.
//   warp 0  TMA producer, warp 1  TMEM + MMA issuer, warps 2-5  epilogue
// At most two CTAs fit an SM (shared memory), with at most 256 TMEM columns
// each, so an allocation never waits for a CTA that waits for this cluster.
// Bound by the weights' bytes and the start: 16 x 2048 x 8192 takes 5.4 us (17 MB, 3.1 TB/s).
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

template <int BT, bool GATED, class TY>
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
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++issued) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, nullptr, p.wait_limit_ns)) break;
        uint8_t* st = smem + stage * L::kStageBytes;
        mbar_arrive_expect_tx(&full[stage], L::kStageBytes);
        tma_load_2d(&tm_w, &full[stage], st, kb * kI8BK, n0);
        if (GATED) tma_load_2d(&tm_w2, &full[stage], st + L::kWBytes, kb * kI8BK, n0);
        tma_load_2d(&tm_x, &full[stage], st + L::kStageBytes - L::kXBytes, kb * kI8BK, m0);
        if (++stage == L::kStages) { stage = 0; phase ^= 1u; }
      }
      wait_loads<L::kStages>(full, issued, stage, phase);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_i8_s32(kI8ChannelTile, BT);
      int stage = 0, last = -1;
      uint32_t phase = 0, last_phase = 0;
      bool ok = !p.lost;
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        if (!mbar_wait(&full[stage], phase, nullptr, p.wait_limit_ns)) { ok = false; break; }
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
        last = stage;
        last_phase = phase;
        if (++stage == L::kStages) { stage = 0; phase ^= 1u; }
      }
      if (ok)
        umma_commit(tfull);
      else if (last >= 0)
        mbar_wait(&empty[last], last_phase, nullptr);
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
    if (!mbar_wait(tfull, 0, nullptr, p.wait_limit_ns)) *failed = 1;
    __syncwarp();
    tc_fence_after();
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    constexpr int kStep = 16;
    if (L::kSplittable && splits > 1) {
      // Every MMA has read the ring: it takes the partial sums, [column][channel].
      int* part = reinterpret_cast<int*>(smem) + row;
#pragma unroll 1
      for (int c = 0; c < L::kAccCols; c += kStep) {
        uint32_t r[kStep];
        tmem_ld_32x32_x16(taddr + c, r);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < kStep; ++j) part[(c + j) * kI8ChannelTile] = static_cast<int>(r[j]);
      }
    } else {
      const bool bad = *failed != 0;
      TY* out = static_cast<TY*>(p.y) + m0 * p.ldy + n;
#pragma unroll 1
      for (int c = 0; c < BT && m0 + c < p.M; c += kStep) {
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
          if (m < p.M && n < p.N) *out = to_y<TY>(v);
          out += p.ldy;
        }
      }
    }
    tc_fence_before();
    if (splits > 1) {
      // Every CTA of the cluster finishes its share of the tile's tokens: a warp
      // takes a token at a time, a lane four neighbouring channels of it.
      cluster_sync();
      bool bad = false;
      for (int s = 0; s < splits; ++s) bad |= ld_cluster_s32(mapa_shared(failed, s)) != 0;
      const int n4 = n0 + 4 * lane;
      float w4[4], u4[4], b4[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w4[k] = n4 + k < p.N ? p.w_scale[n4 + k] : 0.f;
        u4[k] = GATED && n4 + k < p.N ? p.w2_scale[n4 + k] : 0.f;
        b4[k] = !GATED && p.bias && n4 + k < p.N ? p.bias[n4 + k] : 0.f;
      }
      const bool aligned = (reinterpret_cast<uintptr_t>(p.y) & (4 * sizeof(TY) - 1)) == 0 && (p.ldy & 3) == 0;
      const int* part = reinterpret_cast<const int*>(smem) + 4 * lane;
      constexpr int kAtOnce = 4;  // peers' sums in flight
      for (int c = split + splits * (warp - 2); c < BT && m0 + c < p.M; c += 4 * splits) {
        int a[4] = {0, 0, 0, 0}, a2[4] = {0, 0, 0, 0};
        for (int s0 = 0; s0 < splits; s0 += kAtOnce) {
          int4 t[kAtOnce], t2[kAtOnce];
#pragma unroll
          for (int s = 0; s < kAtOnce; ++s)
            if (s0 + s < splits) {
              const uint32_t from = mapa_shared(part + c * kI8ChannelTile, s0 + s);
              t[s] = ld_cluster_s32x4(from);
              if (GATED) t2[s] = ld_cluster_s32x4(from + BT * kI8ChannelTile * 4);
            }
#pragma unroll
          for (int s = 0; s < kAtOnce; ++s)
            if (s0 + s < splits) {
              a[0] += t[s].x; a[1] += t[s].y; a[2] += t[s].z; a[3] += t[s].w;
              if (GATED) { a2[0] += t2[s].x; a2[1] += t2[s].y; a2[2] += t2[s].z; a2[3] += t2[s].w; }
            }
        }
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[k] = static_cast<float>(a[k]) * xs[c] * w4[k];
          if (GATED)
            v[k] = gated_value(v[k], static_cast<float>(a2[k]) * xs[c] * u4[k]);
          else
            v[k] += b4[k];
          if (bad) v[k] = __uint_as_float(0x7fc00000u);
        }
        store4_y(static_cast<TY*>(p.y) + (m0 + c) * p.ldy + n4, v, p.N - n4, aligned && n4 + 4 <= p.N);
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

// ---------------------------------------------------------------------------
// Large products: persistent clusters of two CTAs on 256 x 256 tiles
// (cta_group::2, each CTA loads half of either operand and keeps 128 rows of
// the accumulator), accumulators double-buffered in TMEM so that the epilogue
// of a tile runs under the MMAs of the next.
//   plain  A = 256 channels, B = 256 tokens: lanes are channels, and a warp
//          stores 32 neighbouring channels of a token
//   gated  A = 256 tokens, B = the gate's and the up weights of the same 128
//          hidden units, one CTA loading each: a thread finds g and u of its
//          token in its own TMEM lane, 128 columns apart
// Bound by the tensor pipe: a 256 x 256 x 32 step takes 128 cycles and reads 64
// bytes of shared memory per cycle and SM, half of what one-CTA 128 x 128 tiles do.
// Gated, 16384 x 2560 x 10240: 562 us, 3.06 PFLOP/s, 0.94 of twice the measured
// bf16 rate (one CTA a tile took 765 us); plain 305 us up, 275 us down (0.86, 0.95).
struct Int8PairSmem {
  static constexpr int kStages = 6;
  static constexpr int kHalf = 128 * kI8BK;           // 128 rows of one operand
  static constexpr int kStageBytes = 2 * kHalf;
  static constexpr int kScales = 2 * 256 * 4;         // column scales of two tiles
  static constexpr int kTotal = 1024 + kStages * kStageBytes + (2 * kStages + 4) * 8 + 16 + kScales;
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
};

template <bool GATED, class TY>
__global__ void __launch_bounds__(Int8PairSmem::kThreads, 1)
    int8_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b0,
                     const __grid_constant__ CUtensorMap tm_b1, const Int8GemmParams p) {
  using L = Int8PairSmem;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kStages * L::kStageBytes);
  uint64_t* empty = full + L::kStages;
  uint64_t* tfull = empty + L::kStages;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(tempty + 2);
  float* scales = reinterpret_cast<float*>(tmem_holder + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);   // used in the leader: its producer's expect_tx + both CTAs' bytes
      mbar_init(&empty[s], 1);  // both CTAs: the leader's commit
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);                       // both CTAs: the leader's commit
      mbar_init(&tempty[a], 2 * 32 * L::kEpiWarps);  // used in the leader: both CTAs' epilogue threads
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers exist before any arrival reaches them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  griddep_launch_dependents();
  griddep_wait();

  const int tok_tiles = (p.M + 255) / 256;
  constexpr int kUnits = GATED ? 128 : 256;  // channels (hidden units) of a tile
  const int ch_tiles = (p.N + kUnits - 1) / kUnits;
  const int tiles = tok_tiles * ch_tiles;
  const int total_kb = (p.K + kI8BK - 1) / kI8BK;
  const int cluster = static_cast<int>(blockIdx.x >> 1), clusters = static_cast<int>(gridDim.x >> 1);
  // Tiles walk kGroup token blocks per sweep over the channels.
  constexpr int kGroup = 8;
  auto coords = [&](int tile, int& tok, int& ch) {
    const int per = kGroup * ch_tiles, grp = tile / per, first = grp * kGroup;
    const int size = min(kGroup, tok_tiles - first), r = tile - grp * per;
    tok = first + r % size;
    ch = r / size;
  };

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      const void* tm_b = GATED && !leader ? &tm_b1 : &tm_b0;
      for (int tile = cluster; tile < tiles && ok; tile += clusters) {
        int tok, ch;
        coords(tile, tok, ch);
        const int a0 = (GATED ? tok : ch) * 256 + static_cast<int>(rank) * 128;
        const int b0 = GATED ? ch * 128 : tok * 256 + static_cast<int>(rank) * 128;
        for (int kb = 0; kb < total_kb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, nullptr, p.wait_limit_ns)) { ok = false; break; }
          if (issued < L::kStages) ++issued;
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * L::kStageBytes);
          const uint32_t bar = mapa_shared(&full[stage], 0);
          uint8_t* st = smem + stage * L::kStageBytes;
          tma_load_2d_pair(&tm_a, bar, st, kb * kI8BK, a0);
          tma_load_2d_pair(tm_b, bar, st + L::kHalf, kb * kI8BK, b0);
          if (++stage == L::kStages) { stage = 0; phase ^= 1u; }
        }
      }
      if (leader) wait_loads<L::kStages>(full, issued, stage, phase);  // both CTAs' loads: neither leaves before the other
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      constexpr uint32_t idesc = idesc_i8_s32(256, 256);
      int stage = 0, last = -1;
      uint32_t phase = 0, last_phase = 0;
      int it = 0;
      bool ok = true;
      for (int tile = cluster; tile < tiles && ok; tile += clusters, ++it) {
        const int acc = it & 1;
        if ((p.lost && it > 0) || !mbar_wait(&tempty[acc], ((it >> 1) & 1) ^ 1u, nullptr, p.wait_limit_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + acc * 256;
        for (int kb = 0; kb < total_kb; ++kb) {
          if (!mbar_wait(&full[stage], phase, nullptr, p.wait_limit_ns)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a = smem_u32(smem + stage * L::kStageBytes), b = a + L::kHalf;
#pragma unroll
          for (int k = 0; k < kI8BK / 32; ++k)
            umma_i8_pair(d, smem_desc_sw128(a + k * 32, 16, 1024), smem_desc_sw128(b + k * 32, 16, 1024), idesc,
                         (kb > 0 || k > 0) ? 1u : 0u);
          umma_commit_pair(&empty[stage]);
          last = stage;
          last_phase = phase;
          if (++stage == L::kStages) { stage = 0; phase ^= 1u; }
        }
        if (ok) umma_commit_pair(&tfull[acc]);
      }
      if (!ok && last >= 0) mbar_wait(&empty[last], last_phase, nullptr);
    }
  } else {
    const int q = warp & 3, part = (warp - 2) >> 2, e = threadIdx.x - 64;
    const uint32_t tempty_leader[2] = {mapa_shared(&tempty[0], 0), mapa_shared(&tempty[1], 0)};
    TY* const y = static_cast<TY*>(p.y);
    bool ok = true;
    int it = 0;
    for (int tile = cluster; tile < tiles; tile += clusters, ++it) {
      int tok, ch;
      coords(tile, tok, ch);
      const int acc = it & 1;
      // Scales of the tile's columns (a buffer per accumulator: the other one may still be read).
      float* cs = scales + acc * 256;
      {
        const int c = GATED ? ch * 128 + (e & 127) : tok * 256 + e;
        const float* from = GATED ? (e < 128 ? p.w_scale : p.w2_scale) : p.x_scale;
        cs[e] = c < (GATED ? p.N : p.M) ? from[c] : 0.f;
      }
      const int r = (GATED ? tok : ch) * 256 + static_cast<int>(rank) * 128 + q * 32 + lane;  // token or channel of the lane
      const bool in = r < (GATED ? p.M : p.N);
      const float rs = in ? (GATED ? p.x_scale : p.w_scale)[r] : 0.f;
      const float bias = !GATED && p.bias && in ? p.bias[r] : 0.f;
      named_bar_sync(1, 32 * L::kEpiWarps);
      ok = __all_sync(0xffffffffu, ok && mbar_wait(&tfull[acc], (it >> 1) & 1, nullptr, p.wait_limit_ns));
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * 256;
      if (GATED) {
        const int h0 = ch * 128 + part * 64;
        TY* out = y + static_cast<int64_t>(r) * p.ldy + h0;
        const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll 1
        for (int c = 0; c < 64; c += 16) {
          uint32_t g[16], u[16];
          tmem_ld_32x32_x16(taddr + part * 64 + c, g);
          tmem_ld_32x32_x16(taddr + 128 + part * 64 + c, u);
          tmem_wait_ld();
          const float* gs = cs + part * 64 + c;
          if (in) {
            union { TY e[16]; uint4 u[sizeof(TY)]; } v;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float h = gated_value(static_cast<float>(static_cast<int>(g[j])) * rs * gs[j],
                                    static_cast<float>(static_cast<int>(u[j])) * rs * gs[128 + j]);
              if (!ok) h = __uint_as_float(0x7fc00000u);
              v.e[j] = to_y<TY>(h);
            }
            const int left = p.N - (h0 + c);
            if (aligned && left >= 16) {
#pragma unroll
              for (int k = 0; k < static_cast<int>(sizeof(TY)); ++k) reinterpret_cast<uint4*>(out + c)[k] = v.u[k];
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (j < left) out[c + j] = v.e[j];
            }
          }
        }
      } else {
        const int m0 = tok * 256 + part * 128;
        TY* out = y + static_cast<int64_t>(m0) * p.ldy + r;
#pragma unroll 1
        for (int c = 0; c < 128 && m0 + c < p.M; c += 32) {
          uint32_t a[32];
          tmem_ld_32x32(taddr + part * 128 + c, a);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float v = static_cast<float>(static_cast<int>(a[j])) * cs[part * 128 + c + j] * rs + bias;
            if (!ok) v = __uint_as_float(0x7fc00000u);
            if (in && m0 + c + j < p.M) {
              out[0] = to_y<TY>(v);
            }
            out += p.ldy;
          }
        }
      }
      tc_fence_before();
      if (ok) mbar_arrive_cluster(tempty_leader[acc]);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while its peer may still reach its shared memory
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

}  // namespace twell
