// grouped_tc.cuh -- mm and dgrad of grouped_mm.cuh on the tensor cores (bf16 operands).
//
// grouped_pair_kernel: persistent clusters of two CTAs, 256 x 256 output tiles, tcgen05.mma
// with cta_group::2 (M = 256), the roles and the ring of gemm_tc.cuh.  The operands are read
// where they lie, without transposed copies: an operand whose contraction index is contiguous
// arrives as a K-major tile, one whose output index is contiguous (W of dgrad; dy and x of
// wgrad) as an MN-major tile -- boxes of 64 output columns x 128 contraction rows, 128-byte
// swizzled, which the MMA reads through the descriptor's strides.
//
// An expert's last row tile reads on into the next expert's rows; those accumulator rows are
// computed and not stored.
#pragma once

#include "gemm_tc.cuh"
#include "grouped_mm.cuh"

namespace moe {

// Error word of the grouped kernels on this device (moe_grouped_device_status).
static __device__ int g_grouped_err;

constexpr int kGpEpiWarps = 8;
constexpr int kGpThreads = 64 + 32 * kGpEpiWarps;
// One MN-major box: the contraction rows of a whole stage (two k-blocks), 128 bytes each.  One
// load per 64 columns and stage instead of one per k-block: the loads' issue, not their bytes,
// held the MMA back (weight gradients of 6144 rows an expert: 990 -> 1324 TFLOP/s without them).
constexpr int kGpBoxRows = kGemmKPS * kGemmBK;
constexpr uint32_t kGpBox = kGpBoxRows * 128;

struct GroupedPairArgs {
  const int32_t* counts;
  int G, rows, N, K;     // of the layer: W is [G, N, K]
  void* out;
  int accumulate;        // wgrad: add to out
  int wide;              // output rows are 32-byte aligned: 32-byte stores
};

// MN-major tile of 64-element blocks, each a box of rows of 128 bytes (128-byte swizzle): leading
// offset = distance of two blocks (64 output columns: a box), stride offset = 8 contraction
// rows.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t box) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(box >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}
constexpr uint32_t kIdescAMn = 1u << 15, kIdescBMn = 1u << 16;   // A / B is MN-major

// mbar_wait whose acquire covers the writes of the peer CTA's threads.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                                  int* err, int code) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if ((it & 255u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        record_error(err, code);
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// Arrive on a barrier that hands no memory over (a tensor-memory accumulator that has been
// read into registers, a slot whose value has been used).  A releasing arrive would first wait
// for the thread's earlier global stores.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_relaxed_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

struct GpTile {
  int g, m, n;      // expert, 256-row block, 256-column block of the output
  int row0, grows;  // the expert's rows
  int kb;           // k-blocks
};

template <int OP>
__device__ __forceinline__ GpTile gp_tile(const GroupTable& t, const GroupedPairArgs& a, int nt, int tile, int& g) {
  while (tile >= t.tile0[g + 1]) ++g;
  GpTile c;
  c.g = g;
  const int local = tile - t.tile0[g];
  c.m = local / nt;
  c.n = local - c.m * nt;
  c.row0 = t.row0[g];
  c.grows = t.row0[g + 1] - c.row0;
  c.kb = ((OP == kGroupedMM ? a.K : a.N) + kGemmBK - 1) / kGemmBK;
  return c;
}

template <int OP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGpThreads, 1)
grouped_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    GroupedPairArgs a) {
  constexpr bool kBMn = OP == kGroupedDgrad;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  __shared__ GroupTable tab;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* ctl = base + (size_t)kGemmStages * kGemmStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctl);   // used in the leader
  uint64_t* empty = full + kGemmStages;                 // both CTAs
  uint64_t* acc_full = empty + kGemmStages;             // both CTAs
  uint64_t* acc_empty = acc_full + 2;                   // used in the leader
  uint64_t* drain = acc_empty + 2;                      // both CTAs
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* err = &g_grouped_err;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kGemmStages; ++s) {
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
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kGemmTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  const int out_cols = OP == kGroupedMM ? a.N : a.K;
  const int nt = (out_cols + kGemmBN - 1) / kGemmBN;
  group_table(tab, a.counts, a.G, a.rows, kPairBM, nt);
  const int total = tab.tile0[a.G];

  // columns of a tile, as the MMA's N: a multiple of 32 (each CTA holds half of B's rows)
  auto tile_cols = [&](int n) {
    const int left = out_cols - n * kGemmBN;
    return left >= kGemmBN ? kGemmBN : (left + 31) & ~31;
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0, g = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = cid; tile < total && ok; tile += ncl) {
        const GpTile c = gp_tile<OP>(tab, a, nt, tile, g);
        // this CTA's 128 rows of A (output rows) and half of B's rows (output columns)
        const int a0 = c.row0 + c.m * kPairBM + (int)rank * 128;
        const int b0 = c.n * kGemmBN + (int)rank * (tile_cols(c.n) / 2);
        for (int kb0 = 0; kb0 < c.kb; kb0 += kGemmKPS) {
          ok = mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, err, kErrWaitProducer);
          if (!ok) break;
          const uint32_t sa = smem_u32(base + (size_t)stage * kGemmStageBytes);
          const int nk = c.kb - kb0 < kGemmKPS ? c.kb - kb0 : kGemmKPS;
          const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
          if (leader)   // both CTAs' bytes
            mbar_arrive_expect_tx(smem_u32(&full[stage]),
                                  2u * ((uint32_t)nk * kGemmABytes + (kBMn ? 2u * kGpBox : (uint32_t)nk * kGemmBBytes)));
          for (int j = 0; j < nk; ++j) {
            const int q = (kb0 + j) * kGemmBK;   // contraction index
            tma_load_2d_pair(sa + j * kGemmABytes, &tmA, fb, q, a0);
            if (!kBMn) tma_load_3d_pair(sa + kGemmBOff + j * kGemmBBytes, &tmB, fb, q, b0, c.g);
          }
          if (kBMn) {   // rows behind the contraction's end arrive as zeros
            tma_load_3d_pair(sa + kGemmBOff, &tmB, fb, b0, kb0 * kGemmBK, c.g);
            tma_load_3d_pair(sa + kGemmBOff + kGpBox, &tmB, fb, b0 + 64, kb0 * kGemmBK, c.g);
          }
          if (++stage == kGemmStages) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {   // gave up: let the copies in flight land before the CTA's memory is handed on
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
      } else {   // every stage released: no copy of this CTA is in flight
        for (int s = 0; s < kGemmStages; ++s) {
          if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, err, kErrWaitDrain)) break;
          if (++stage == kGemmStages) { stage = 0; phase ^= 1u; }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0 && leader) {
      int stage = 0, g = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = cid; tile < total && ok; tile += ncl, ++it) {
        const GpTile c = gp_tile<OP>(tab, a, nt, tile, g);
        const uint32_t idesc = idesc_bf16_f32(kPairBM, tile_cols(c.n)) | (kBMn ? kIdescBMn : 0u);
        const int acc = it & 1;
        const uint32_t acc_par = (it >> 1) & 1;
        ok = mbar_wait(smem_u32(&acc_empty[acc]), acc_par ^ 1u, abort_flag, err, kErrWaitMma);
        if (!ok) break;
        tc_fence_after();
        const uint32_t dt = tmem_base + static_cast<uint32_t>(acc * kGemmBN);
        for (int kb0 = 0; kb0 < c.kb; kb0 += kGemmKPS) {
          ok = mbar_wait(smem_u32(&full[stage]), phase, abort_flag, err, kErrWaitMma);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sa = smem_u32(base + (size_t)stage * kGemmStageBytes);
          const int nk = c.kb - kb0 < kGemmKPS ? c.kb - kb0 : kGemmKPS;
          for (int j = 0; j < nk; ++j) {
            const uint64_t ad = sdesc_k_sw128(sa + j * kGemmABytes);
            const uint64_t bd = kBMn ? sdesc_mn_sw128(sa + kGemmBOff + j * (kGemmBK * 128u), kGpBox)
                                     : sdesc_k_sw128(sa + kGemmBOff + j * kGemmBBytes);
            // 16 contraction values a step: 32 bytes along a K-major row, 16 rows of 128 bytes
            // of an MN-major box
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_f16_pair(dt, ad + 2u * k, bd + (kBMn ? 128u : 2u) * k, idesc, (kb0 | j | k) != 0);
          }
          tc_commit_pair_mc(smem_u32(&empty[stage]), 0x3);
          if (++stage == kGemmStages) { stage = 0; phase ^= 1u; }
        }
        if (ok) tc_commit_pair_mc(smem_u32(&acc_full[acc]), 0x3);
      }
      tc_commit_pair_mc(smem_u32(drain), 0x3);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3;                 // TMEM lane quadrant
    const int half = (warp - 2) >> 2;       // which half of the tile's columns
    const int rr = q * 32 + lane;
    int g = 0, it = 0;
    for (int tile = cid; tile < total; tile += ncl, ++it) {
      const GpTile c = gp_tile<OP>(tab, a, nt, tile, g);
      const int acc = it & 1;
      const uint32_t acc_par = (it >> 1) & 1;
      int ok = 1;
      if (lane == 0) ok = mbar_wait(smem_u32(&acc_full[acc]), acc_par, abort_flag, err, kErrWaitEpilogue);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      tc_fence_after();
      const uint32_t trow =
          tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * kGemmBN);
      const int mrow = c.m * kPairBM + (int)rank * 128 + rr;   // row of the expert
      const bool row_ok = mrow < c.grows;
      const size_t orow = (size_t)c.row0 + mrow;
      // this thread's half row, rounded, in registers: the accumulator is free before the
      // stores (whose completion a release behind them would wait for)
      const int col0 = c.n * kGemmBN + half * (kGemmBN / 2);
      uint32_t pk[4][16];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (col0 + 32 * x >= out_cols) break;
        uint32_t v[32];
        tmem_ld32(trow + static_cast<uint32_t>(half * (kGemmBN / 2) + 32 * x), v);
        tmem_ld_wait(v);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          pk[x][i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed_cluster(mapa_shared(smem_u32(&acc_empty[acc]), 0));
      if (!row_ok) continue;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + orow * out_cols + col0;
      const int left = out_cols - col0;   // a multiple of 8
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        if (16 * x >= left) break;
        const uint32_t* p = &pk[x >> 1][(x & 1) * 8];
        const uint4 lo = make_uint4(p[0], p[1], p[2], p[3]), hi = make_uint4(p[4], p[5], p[6], p[7]);
        if (a.wide) {
          st_global_v8(o + 16 * x, lo, hi);
        } else {
          *reinterpret_cast<uint4*>(o + 16 * x) = lo;
          if (16 * x + 8 < left) *reinterpret_cast<uint4*>(o + 16 * x + 8) = hi;
        }
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
    tmem_dealloc_pair(tmem_base, kGemmTmemCols);
  }
}

}  // namespace moe
