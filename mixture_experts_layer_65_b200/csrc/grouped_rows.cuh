// grouped_rows.cuh -- mm and dgrad of grouped_mm.cuh on the tensor cores (bf16 operands), weights on
// the MMA's M dimension: y^T = W_e x_e^T and dx^T = W_e^T dy_e^T, tiles of 256 output columns x up
// to `tile_rows` rows of an expert.
//
// Ragged rows are what decides the orientation.  On the N dimension an expert's last tile takes
// its rows rounded up to 32, on the M dimension it would take them rounded up to 256 (measured
// both ways: 63 experts of about 910 rows, 896 x 1280, dgrad 133.8 against 119.7 us; 64 of about
// 1536 rows, 2816 x 2048, 851 against 837 us); and with few rows per expert a tile is one pass over
// 256 rows of W_e with little else to load, so the weights stream (64 experts of 6 rows,
// 2816 x 2048: 148.8 against 117.5 us, 6.3 TB/s).
//
// Persistent clusters of two CTAs, tcgen05.mma with cta_group::2 (M = 256), roles as in
// gemm_tc.cuh.  The accumulator is the output transposed (a TMEM lane per output column): each
// epilogue warp turns 32 x 32 blocks through shared memory and stores 64 bytes per row (stores of
// 2 or 4 bytes a lane straight from registers: the same time).
//
// Bound by the tensor cores, and by the power they draw, with many rows per expert (64 experts of
// 1536 rows, 2816 x 2048: 0.80 ms, 1.43 PFLOP/s, tensor pipe 88% active; 0.98 ms once a loop meets
// the power cap; short contractions pay the change of tiles and the clusters' uneven share of ragged
// tiles: 63 of 910 rows, 896 x 1280, 118 us, 80%), by HBM with few (64 of 6 rows: 117 us, 6.3 TB/s of
// weights).
#pragma once

#include "grouped_tc.cuh"

namespace moe {

constexpr int kGrMaxStages = 5;
constexpr uint32_t kGrABytes = kGemmKPS * kGemmABytes;   // this CTA's 128 output columns of W
constexpr uint32_t kGrWBox = kGemmKPS * kGemmBK * 128;   // W of dgrad: 64 columns, a stage's rows
constexpr uint32_t kGrTurnBytes = 32 * 64;            // one epilogue warp's 32 x 32 block
constexpr uint32_t kGrRingBytes = 196608;

// Rows per tile.  Up to 32 rows an expert on average, 64: the stages are smaller and five of them
// fit instead of three, so more weights are in flight (64 experts of 24 rows: 120.4 against
// 126.3 us); above, 256, since every tile reads W_e again (of 96 rows: 137 against 180 us).
__host__ __device__ constexpr int gr_tile_rows(int64_t rows, int G) { return rows <= 32 * (int64_t)G ? 64 : 256; }

// A stage: two k-blocks of W and of `tile_rows` / 2 rows.
__host__ __device__ constexpr uint32_t gr_stage_bytes(int tile_rows) {
  return kGrABytes + (uint32_t)kGemmKPS * (uint32_t)(tile_rows / 2) * 128u;
}
__host__ __device__ constexpr int gr_stages(int tile_rows) {
  return kGrRingBytes / gr_stage_bytes(tile_rows) > (uint32_t)kGrMaxStages
             ? kGrMaxStages
             : (int)(kGrRingBytes / gr_stage_bytes(tile_rows));
}
// k-blocks of one accumulator chain.  The tensor cores truncate when they add to an accumulator: a
// chain of c values of one sign ends up to 6e-9 c below their sum (measured: 6e-3 of it at 2^20
// values, where bf16's own half step is 4e-3).  Up to 16,384 values that is a fortieth of the half
// step and one chain; longer contractions are cut, and the epilogue warps add the pieces in
// registers, rounding to nearest.
constexpr int kGrChain = 256;

constexpr size_t kGrSmemBytes = 1024 + kGrRingBytes + 1024 + kGpEpiWarps * kGrTurnBytes;

struct GroupedRowsArgs {
  const int32_t* counts;
  int G, rows, N, K;     // of the layer: W is [G, N, K]
  __nv_bfloat16* out;
  int tile_rows;         // gr_tile_rows
};

// mm: W's rows are the output columns (K-major); dgrad: W's columns are (MN-major).  LONG: the
// contraction has more than kGrChain k-blocks.
template <int OP, bool LONG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGpThreads, 1)
grouped_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    GroupedRowsArgs a) {
  constexpr bool kAMn = OP == kGroupedDgrad;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  __shared__ GroupTable tab;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int RT = a.tile_rows;
  const uint32_t stage_bytes = gr_stage_bytes(RT);
  const int S = gr_stages(RT);
  uint8_t* ctl = base + kGrRingBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctl);   // used in the leader
  uint64_t* empty = full + kGrMaxStages;                // both CTAs
  uint64_t* acc_full = empty + kGrMaxStages;            // both CTAs
  uint64_t* acc_empty = acc_full + 2;                   // used in the leader
  uint64_t* drain = acc_empty + 2;                      // both CTAs
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* turn_base = ctl + 1024;
  int* err = &g_grouped_err;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
  const uint32_t tmem_cols = 2u * (uint32_t)RT;   // two accumulators

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&acc_full[s]), 1);
      mbar_init(smem_u32(&acc_empty[s]), 2 * kGpEpiWarps);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), tmem_cols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  const int out_cols = OP == kGroupedMM ? a.N : a.K;
  const int nt = (out_cols + kPairBM - 1) / kPairBM;
  const int kbn = ((OP == kGroupedMM ? a.K : a.N) + kGemmBK - 1) / kGemmBK;
  group_table(tab, a.counts, a.G, a.rows, RT, nt);
  const int total = tab.tile0[a.G];

  // tile -> expert g, column tile n, first row and rows
  struct Tile {
    int g, n, row, rows;
  };
  auto tile_of = [&](int tile, int& g) {
    while (tile >= tab.tile0[g + 1]) ++g;
    const int local = tile - tab.tile0[g], m = local / nt;
    Tile t;
    t.g = g;
    t.n = local - m * nt;
    t.row = tab.row0[g] + m * RT;
    const int left = tab.row0[g + 1] - t.row;
    t.rows = left < RT ? left : RT;
    return t;
  };
  auto mma_n = [&](const Tile& t) { return (t.rows + 31) & ~31; };   // each CTA holds half of the rows

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0, g = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t row_bytes = (uint32_t)(RT / 2) * 128u;   // one k-block of this CTA's rows
      for (int tile = cid; tile < total && ok; tile += ncl) {
        const Tile t = tile_of(tile, g);
        const int c0 = t.n * kPairBM + (int)rank * 128;
        const int r0 = t.row + (int)rank * (mma_n(t) / 2);
        for (int kb0 = 0; kb0 < kbn; kb0 += kGemmKPS) {
          ok = mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, err, kErrWaitProducer);
          if (!ok) break;
          const uint32_t sa = smem_u32(base + (size_t)stage * stage_bytes);
          const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
          const int nk = kbn - kb0 < kGemmKPS ? kbn - kb0 : kGemmKPS;
          if (leader)   // both CTAs' bytes
            mbar_arrive_expect_tx(smem_u32(&full[stage]),
                                  2u * ((kAMn ? kGrABytes : (uint32_t)nk * kGemmABytes) + (uint32_t)nk * row_bytes));
          if (kAMn) {   // rows behind the contraction's end arrive as zeros
            tma_load_3d_pair(sa, &tmW, fb, c0, kb0 * kGemmBK, t.g);
            tma_load_3d_pair(sa + kGrWBox, &tmW, fb, c0 + 64, kb0 * kGemmBK, t.g);
          }
          for (int j = 0; j < nk; ++j) {
            const int q = (kb0 + j) * kGemmBK;
            if (!kAMn) tma_load_3d_pair(sa + j * kGemmABytes, &tmW, fb, q, c0, t.g);
            tma_load_2d_pair(sa + kGrABytes + j * row_bytes, &tmX, fb, q, r0);
          }
          if (++stage == S) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {   // gave up: let the copies in flight land before the CTA's memory is handed on
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
      } else {   // every stage released: no copy of this CTA is in flight
        for (int s = 0; s < S; ++s) {
          if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, err, kErrWaitDrain)) break;
          if (++stage == S) { stage = 0; phase ^= 1u; }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0 && leader) {
      int stage = 0, g = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t row_bytes = (uint32_t)(RT / 2) * 128u;
      const int chain = LONG ? kGrChain : kbn;
      for (int tile = cid; tile < total && ok; tile += ncl) {
        const Tile t = tile_of(tile, g);
        const uint32_t idesc = idesc_bf16_f32(kPairBM, mma_n(t)) | (kAMn ? kIdescAMn : 0u);
        for (int kc = 0; kc < kbn && ok; kc += chain, ++it) {
          const int kend = kbn - kc < chain ? kbn : kc + chain;
          const int acc = it & 1;
          ok = mbar_wait(smem_u32(&acc_empty[acc]), ((it >> 1) & 1) ^ 1u, abort_flag, err, kErrWaitMma);
          if (!ok) break;
          tc_fence_after();
          const uint32_t dt = tmem_base + static_cast<uint32_t>(acc * RT);
          for (int kb0 = kc; kb0 < kend; kb0 += kGemmKPS) {
            ok = mbar_wait(smem_u32(&full[stage]), phase, abort_flag, err, kErrWaitMma);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sa = smem_u32(base + (size_t)stage * stage_bytes);
            const int nk = kend - kb0 < kGemmKPS ? kend - kb0 : kGemmKPS;
            for (int j = 0; j < nk; ++j) {
              const uint64_t ad = kAMn ? sdesc_mn_sw128(sa + j * (kGemmBK * 128u), kGrWBox)
                                       : sdesc_k_sw128(sa + j * kGemmABytes);
              const uint64_t bd = sdesc_k_sw128(sa + kGrABytes + j * row_bytes);
#pragma unroll
              for (int k = 0; k < 4; ++k)   // 16 contraction values a step
                tc_mma_f16_pair(dt, ad + (kAMn ? 128u : 2u) * k, bd + 2u * k, idesc, ((kb0 - kc) | j | k) != 0);
            }
            tc_commit_pair_mc(smem_u32(&empty[stage]), 0x3);
            if (++stage == S) { stage = 0; phase ^= 1u; }
          }
          if (ok) tc_commit_pair_mc(smem_u32(&acc_full[acc]), 0x3);
        }
      }
      tc_commit_pair_mc(smem_u32(drain), 0x3);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3;                 // TMEM lane quadrant: 32 output columns
    const int half = (warp - 2) >> 2;       // even or odd blocks of 32 rows
    uint8_t* turn = turn_base + (warp - 2) * kGrTurnBytes;
    int g = 0, it = 0;
    for (int tile = cid; tile < total; tile += ncl) {
      const Tile t = tile_of(tile, g);
      const int col0 = t.n * kPairBM + (int)rank * 128 + q * 32;   // this warp's output columns
      const int col = col0 + (lane & 3) * 8;                       // this lane's when it stores
      uint32_t tq;
      auto ready = [&] {   // the next accumulator is full
        int ok = 1;
        if (lane == 0) ok = mbar_wait(smem_u32(&acc_full[it & 1]), (it >> 1) & 1, abort_flag, err, kErrWaitEpilogue);
        if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
        tc_fence_after();
        tq = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>((it & 1) * RT);
        return true;
      };
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed_cluster(mapa_shared(smem_u32(&acc_empty[it & 1]), 0));
        ++it;
      };
      auto store = [&](int rb, const uint32_t (&v)[32]) {   // 32 rows of this warp's columns
#pragma unroll
        for (int i = 0; i < 32; ++i)   // row i, column lane
          *reinterpret_cast<__nv_bfloat16*>(turn + i * 64 + lane * 2) = __float2bfloat16_rn(__uint_as_float(v[i]));
        __syncwarp();
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = *reinterpret_cast<const uint4*>(turn + (8 * i + (lane >> 2)) * 64 + (lane & 3) * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = rb + 8 * i + (lane >> 2);
          if (r < t.rows && col < out_cols)   // (out_cols is a multiple of 8)
            *reinterpret_cast<uint4*>(a.out + (size_t)(t.row + r) * out_cols + col) = w[i];
        }
      };
      if constexpr (LONG) {
        uint32_t s[4][32] = {};
        int ok = 1;
        for (int kc = 0; kc < kbn; kc += kGrChain) {
          ok = ready();
          if (!ok) break;
          const int blocks = RT / 64;   // of this warp: one or four (rows behind the tile's are not stored)
          if (kc == 0) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (x < blocks) tmem_ld32(tq + static_cast<uint32_t>(half * 32 + 64 * x), s[x]);
#pragma unroll
            for (int x = 0; x < 4; ++x) tmem_ld_wait(s[x]);
          } else {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (x < blocks) {
                uint32_t v[32];
                tmem_ld32(tq + static_cast<uint32_t>(half * 32 + 64 * x), v);
                tmem_ld_wait(v);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  s[x][i] = __float_as_uint(__fadd_rn(__uint_as_float(s[x][i]), __uint_as_float(v[i])));
              }
          }
          release();
        }
        if (!ok) break;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (half * 32 + 64 * x < t.rows && col0 < out_cols) {
            __syncwarp();
            store(half * 32 + 64 * x, s[x]);
          }
      } else {
        if (!ready()) break;
#pragma unroll 1
        for (int rb = half * 32; rb < t.rows && col0 < out_cols; rb += 64) {
          uint32_t v[32];
          __syncwarp();
          tmem_ld32(tq + static_cast<uint32_t>(rb), v);
          tmem_ld_wait(v);
          store(rb, v);
        }
        release();
      }
    }
  }

  // teardown: all MMAs of the pair have completed before TMEM is released in either CTA
  if (warp == 1 && lane == 0) mbar_wait(smem_u32(drain), 0, abort_flag, err, kErrWaitDrain);
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, tmem_cols);
  }
}

}  // namespace moe
