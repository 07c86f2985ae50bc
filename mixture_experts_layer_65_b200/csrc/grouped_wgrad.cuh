// grouped_wgrad.cuh -- the weight gradients of grouped_mm.cuh on the tensor cores (bf16 operands,
// fp32 result): dW_e = dy_e^T x_e, a product whose contraction runs over the expert's rows.
//
// Clusters of two CTAs, 256 x 256 tiles of dW_e^T, tcgen05.mma with cta_group::2.  x and dy are read
// where they lie: their contiguous index is an output index, so both operands are MN-major
// tiles (boxes of 64 columns x 128 rows, one stage of the ring).  The transpose puts dW's
// contiguous index on the accumulator's lanes: an epilogue warp's store of one accumulator
// column is a whole 128-byte line, straight from registers (with dW's rows on the lanes, stores of
// 32 bytes from 32 rows took 2.6 times as long, and TMA stores through shared memory took 32 KB
// of the ring); and dW's rows, the experts' widths, which are less often multiples of 256 than
// the model's, are on the MMA's N, whose last tile takes any multiple of 32.
//
// Precision: the tensor cores truncate when they add to an accumulator, which over n steps of
// 16 rows leaves a bias of about 2.2e-8 n of the value (measured: 7.4e-6 of dW's norm when an
// expert had 10,800 rows in one chain).  So a chain is cut after kGwChunk stages of 128
// rows: the epilogue warps add the pieces in registers with round-to-nearest while the MMA
// fills the other accumulator.
//
// Ragged rows: a tile's last stage runs ceil(t / 16) of its eight MMA steps for t rows, and the
// rows behind t in the last step are zeroed in both operands (0 x NaN would be NaN) by a
// warp of each CTA before the MMA: that stage's loads complete on a barrier of the CTA, and
// the leader's zeroing warp, told by the peer's, arrives on the "full" barrier instead of the
// producer.  (A second arrival, by the peer's producer, on every stage's "full" barrier held
// the kernel to 1195 TFLOP/s instead of 1412 with 65,536 rows in one expert: its release at
// cluster scope waits for the thread's earlier work.)
//
// Balance: a tile's time goes with its expert's rows, which may differ a hundredfold.  The
// grid has one cluster per tile, experts with most rows first; a running cluster takes the
// next unstarted one over (clusterlaunchcontrol), so no cluster is left with a long tile at
// the end, and which cluster computes a tile does not change its value.  A warp of each CTA does
// nothing but ask (the leader's), read the answer and hand the tile on, worked out: in the
// producer that took 2,400 cycles a tile, which the ring could not cover.
//
// Bound by the tensor cores with long sums (64 experts of 6144 rows, 1408 x 2048: 1.84 ms, 1.23
// PFLOP/s).  With short ones (1 row: 143 us; 160 rows: 152) by the stores' way out of the SM: a
// line takes 3 cycles there, and every barrier, load and MMA instruction of the other warps
// queues with them; stores that stay in L2 take as long, so it is not HBM (738 MB: 112 us).  In
// between (768 rows: 297 us, 0.95 PFLOP/s; 254 without the stores) both count.  Readers that
// look up four words instead of a tile number saved 15 us of the 1-row case; stores through
// shared memory and TMA boxes of 8 rows take 220 us there.
#pragma once

#include "grouped_tc.cuh"

namespace moe {

// A stage: 128 rows (eight MMA steps), two boxes of 64 columns each of x and dy.
constexpr int kGwRows = 128;
constexpr int kGwStages = 3;
constexpr uint32_t kGwBox = kGwRows * 128;
constexpr uint32_t kGwStageBytes = 4 * kGwBox;
constexpr int kGwChunk = 3;                                // stages per accumulator chain
constexpr int kGwThreads = 64 + 32 * (kGpEpiWarps + 2);    // + the zeroing and the scheduling warp
constexpr int kGwSlots = 4;                                // answers, and tiles handed on
constexpr int kGwAhead = 2;                                // requests made ahead
constexpr size_t kGwSmemBytes = 1024 + kGwStages * kGwStageBytes + 1024;
static_assert(kPairBM == 256 && kGemmBN == 256, "wgrad_parts counts tiles of 256 x 256");
static_assert(kGwBox % 1024 == 0 && kGwRows % 16 == 0, "swizzle atoms, MMA steps");

struct GroupedWgradArgs {
  const int32_t* counts;
  float* out;            // [splits, G, N, K]
  int G, rows, N, K;
  int accumulate;        // add to dW
  int splits;            // parts of the rows, each with its own [G, N, K]
};

// The experts' first rows, and the experts in order of falling row counts.
struct WgradTable {
  int32_t row0[kGroupedMaxGroups + 1];
  int32_t order[kGroupedMaxGroups];
};

// Take over the next cluster of the grid that has not started: its answer (16 bytes) arrives
// at the same offset of both CTAs' shared memory, counted on the barrier at the same offset.
__device__ __forceinline__ void clc_try_cancel(uint32_t answer, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
      ".multicast::cluster::all.b128 [%0], [%1];" ::"r"(answer),
      "r"(bar)
      : "memory");
}
// The first CTA of the cluster taken over, or -1 when none was left.
__device__ __forceinline__ int clc_answer(uint32_t answer) {
  uint32_t x, ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %1, 1, 0, p;\n\t"
      "mov.u32 %0, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n\t}\n"
      : "=r"(x), "=r"(ok)
      : "r"(answer)
      : "memory");
  return ok ? static_cast<int>(x) : -1;
}

// A scheduling warp's way through the grid: `ahead` requests open at a time until one is refused,
// every tile granted handed on, -1 behind the last.  A refusal does not mean that the requests made
// after it are refused too (a waiting kernel of higher priority is a reason to refuse, and may
// be gone by then): the open ones' answers are tiles like the others, whose clusters will not
// start any more.  No request follows an observed refusal (the instruction forbids it); clusters still
// unstarted then start by themselves.  ask(), answer(tile) and hand(tile) return false when a wait
// ran out.
template <class Ask, class Answer, class Hand>
__host__ __device__ __forceinline__ bool take_tiles_over(int ahead, Ask&& ask, Answer&& answer, Hand&& hand) {
  int open = 0;
  bool refused = false;
  for (; open < ahead; ++open)
    if (!ask()) return false;
  while (open > 0) {
    int tile = -1;
    if (!answer(tile)) return false;
    --open;
    if (tile < 0) {
      refused = true;
      continue;
    }
    if (!refused) {
      if (!ask()) return false;
      ++open;
    }
    if (!hand(tile)) return false;
  }
  return hand(-1);
}

// Arrive on the peer's barrier without ordering anything (it guards only what the barrier
// itself counts).
__device__ __forceinline__ void mbar_arrive_expect_tx_peer(uint32_t cluster_addr, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_addr),
               "r"(bytes)
               : "memory");
}

static __global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGwThreads, 1)
grouped_wgrad_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmDy,
                     GroupedWgradArgs a) {
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  __shared__ WgradTable tab;
  __shared__ __align__(16) uint8_t answers[kGwSlots][16];
  __shared__ int4 tiles[kGwSlots];   // part times G plus expert, 256-blocks, rows of x and dy
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* ctl = base + (size_t)kGwStages * kGwStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctl);   // used in the leader
  uint64_t* empty = full + kGwStages;                 // both CTAs
  uint64_t* acc_full = empty + kGwStages;             // both CTAs
  uint64_t* acc_empty = acc_full + 2;                   // used in the leader
  uint64_t* drain = acc_empty + 2;                      // both CTAs
  uint64_t* tail = drain + 1;                           // both CTAs: loads of a tail stage
  uint64_t* peer_tail = tail + kGwStages;             // used in the leader: the peer's zeros
  uint64_t* next_full = peer_tail + kGwStages;        // both CTAs: an answer has arrived
  uint64_t* next_empty = next_full + kGwSlots;          // used in the leader: the peer has read it
  uint64_t* tile_full = next_empty + kGwSlots;          // both CTAs: tiles[] filled, and read by all
  uint64_t* tile_empty = tile_full + kGwSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tile_empty + kGwSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* err = &g_grouped_err;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kGwStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);    // the leader's producer, or its zeroing warp
      mbar_init(smem_u32(&peer_tail[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
      mbar_init(smem_u32(&tail[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&acc_full[s]), 1);
      mbar_init(smem_u32(&acc_empty[s]), 2 * kGpEpiWarps);
    }
    for (int s = 0; s < kGwSlots; ++s) {
      mbar_init(smem_u32(&next_full[s]), 1);
      mbar_init(smem_u32(&next_empty[s]), 1);
      mbar_init(smem_u32(&tile_full[s]), 1);
      // the producer, the zeroing warp, the epilogue warps and, in the leader, the MMA issuer
      mbar_init(smem_u32(&tile_empty[s]), 2 + kGpEpiWarps + (leader ? 1 : 0));
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmDy);
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
  const int nt = (a.N + kGemmBN - 1) / kGemmBN;                    // tiles along a gradient's rows
  const int per_group = nt * ((a.K + kPairBM - 1) / kPairBM);
  group_rows(tab.row0, a.counts, a.G, a.rows);
  for (int g = threadIdx.x; g < a.G; g += kGwThreads) {
    const int n = tab.row0[g + 1] - tab.row0[g];
    int before = 0;
    for (int h = 0; h < a.G; ++h) {
      const int m = tab.row0[h + 1] - tab.row0[h];
      before += m > n || (m == n && h < g);
    }
    tab.order[before] = g;
  }
  __syncthreads();

  struct Tile {
    int z, m, n;      // part times G plus expert (< 0: no tile); 256-column block, 256-row block of dW
    int row0, grows;  // the expert's rows of this part
    int kb;           // stages
  };
  // a tile in four words, as the scheduling warp hands it on: a reader has one load to wait for
  auto describe = [&](int tile) {
    if (tile < 0) return make_int4(-1, 0, 0, 0);
    const int o = tile / (per_group * a.splits);
    int local = tile - o * (per_group * a.splits);
    const int part = local / per_group, g = tab.order[o];
    local -= part * per_group;
    const int m = local / nt;
    int row0 = tab.row0[g], rows = tab.row0[g + 1] - row0;
    split_rows(row0, rows, a.splits, part);
    return make_int4(part * a.G + g, m << 16 | (local - m * nt), row0, rows);   // (blocks: below 2^12)
  };
  auto tile_of = [&](const int4& t) {
    return Tile{t.x, t.y >> 16, t.y & 0xffff, t.z, t.w, (t.w + kGwRows - 1) / kGwRows};
  };
  auto tile_cols = [&](int n) {   // the MMA's N: a multiple of 32
    const int left = a.N - n * kGemmBN;
    return left >= kGemmBN ? kGemmBN : (left + 31) & ~31;
  };
  auto tail_rows = [&](const Tile& c) { return c.grows - (c.kb - 1) * kGwRows; };   // of the last stage
  struct Slot {
    int i = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
      if (++i == kGwSlots) { i = 0; phase ^= 1u; }
    }
  };
  // The tile the scheduling warp hands on, to one thread of each reader or to a warp; x < 0: none
  // left, or a wait ran out.
  auto next_tile = [&](Slot& sl) {
    if (!mbar_wait(smem_u32(&tile_full[sl.i]), sl.phase, abort_flag, err, kErrWaitProducer))
      return make_int4(-1, 0, 0, 0);
    const int4 t = tiles[sl.i];
    if (t.x >= -1) mbar_arrive_relaxed(smem_u32(&tile_empty[sl.i]));   // (always: the value has arrived)
    sl.next();
    return t;
  };
  auto warp_tile = [&](Slot& sl) {
    int4 t = make_int4(0, 0, 0, 0);
    if (lane == 0) t = next_tile(sl);
    t.x = __shfl_sync(0xffffffffu, t.x, 0);
    t.y = __shfl_sync(0xffffffffu, t.y, 0);
    t.z = __shfl_sync(0xffffffffu, t.z, 0);
    t.w = __shfl_sync(0xffffffffu, t.w, 0);
    return t;
  };

  const int4 first = describe(blockIdx.x >> 1);
  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      Slot sl;
      for (int4 tile = first; tile.x >= 0 && ok;) {
        const Tile c = tile_of(tile);
        const int a0 = c.m * kPairBM + (int)rank * 128;
        const int b0 = c.n * kGemmBN + (int)rank * (tile_cols(c.n) / 2);
        for (int kb = 0; kb < c.kb; ++kb) {
          ok = mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, err, kErrWaitProducer);
          if (!ok) break;
          const uint32_t sa = smem_u32(base + (size_t)stage * kGwStageBytes);
          const bool fix = kb == c.kb - 1 && (tail_rows(c) & 15) != 0;
          const uint32_t fb =
              fix ? mapa_shared(smem_u32(&tail[stage]), rank) : mapa_shared(smem_u32(&full[stage]), 0);
          if (fix) mbar_arrive_expect_tx(smem_u32(&tail[stage]), kGwStageBytes);
          else if (leader) mbar_arrive_expect_tx(smem_u32(&full[stage]), 2u * kGwStageBytes);
          const int row = c.row0 + kb * kGwRows;
          tma_load_2d_pair(sa, &tmX, fb, a0, row);
          tma_load_2d_pair(sa + kGwBox, &tmX, fb, a0 + 64, row);
          tma_load_2d_pair(sa + 2 * kGwBox, &tmDy, fb, b0, row);
          tma_load_2d_pair(sa + 2 * kGwBox + kGwBox, &tmDy, fb, b0 + 64, row);
          if (++stage == kGwStages) { stage = 0; phase ^= 1u; }
        }
        if (ok) tile = next_tile(sl);
      }
      if (!ok) {   // gave up: let the copies in flight land before the CTA's memory is handed on
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
      } else {   // every stage released: no copy of this CTA is in flight
        for (int s = 0; s < kGwStages; ++s) {
          if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, err, kErrWaitDrain)) break;
          if (++stage == kGwStages) { stage = 0; phase ^= 1u; }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0 && leader) {
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      Slot sl;
      for (int4 tile = first; tile.x >= 0 && ok;) {
        const Tile c = tile_of(tile);
        const uint32_t idesc = idesc_bf16_f32(kPairBM, tile_cols(c.n)) | kIdescAMn | kIdescBMn;
        for (int kc = 0; kc < c.kb && ok; kc += kGwChunk, ++it) {
          const int kend = c.kb - kc < kGwChunk ? c.kb : kc + kGwChunk;
          const int acc = it & 1;
          ok = mbar_wait(smem_u32(&acc_empty[acc]), ((it >> 1) & 1) ^ 1u, abort_flag, err, kErrWaitMma);
          if (!ok) break;
          tc_fence_after();
          const uint32_t dt = tmem_base + static_cast<uint32_t>(acc * kGemmBN);
          for (int kb = kc; kb < kend; ++kb) {
            ok = mbar_wait(smem_u32(&full[stage]), phase, abort_flag, err, kErrWaitMma);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sa = smem_u32(base + (size_t)stage * kGwStageBytes);
            const uint64_t ad = sdesc_mn_sw128(sa, kGwBox), bd = sdesc_mn_sw128(sa + 2 * kGwBox, kGwBox);
            const int steps = kb == c.kb - 1 ? (tail_rows(c) + 15) >> 4 : kGwRows / 16;
#pragma unroll
            for (int k = 0; k < kGwRows / 16; ++k)   // 16 rows of 128 bytes a step
              if (k < steps) tc_mma_f16_pair(dt, ad + 128u * k, bd + 128u * k, idesc, (kb != kc) | k);
            tc_commit_pair_mc(smem_u32(&empty[stage]), 0x3);
            if (++stage == kGwStages) { stage = 0; phase ^= 1u; }
          }
          if (ok) tc_commit_pair_mc(smem_u32(&acc_full[acc]), 0x3);
        }
        if (ok) tile = next_tile(sl);
      }
      tc_commit_pair_mc(smem_u32(drain), 0x3);
    }
    __syncwarp();
  } else if (warp == 2 + kGpEpiWarps) {
    // ------------------------------------------------------------------ zeroing of tail rows
    int stage = 0;
    uint32_t tail_phase = 0;   // a bit per stage
    Slot sl;
    for (int4 tile = first; tile.x >= 0;) {
      const Tile c = tile_of(tile);
      const int last = (stage + c.kb + kGwStages - 1) % kGwStages;
      stage = (stage + c.kb) % kGwStages;
      const int t = tail_rows(c);
      if (c.kb > 0 && (t & 15) != 0) {
        int ok = 1;
        if (lane == 0) ok = mbar_wait(smem_u32(&tail[last]), tail_phase >> last & 1u, abort_flag, err, kErrWaitDrain);
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        __syncwarp();
        // rows [t, 16 ceil(t / 16)) of the stage's four boxes, 128 bytes a row (the swizzle
        // permutes 16-byte chunks within a row)
        uint8_t* sp = base + (size_t)last * kGwStageBytes;
        const int nz = ((t + 15) & ~15) - t;
        for (int i = lane; i < nz * 32; i += 32)
          *reinterpret_cast<uint4*>(sp + ((i >> 3) & 3) * kGwBox + (t + (i >> 5)) * 128 + (i & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_shared();   // the zeros, before the tensor cores read the stage
        __syncwarp();
        if (lane == 0) {
          if (!leader) {
            mbar_arrive_cluster(mapa_shared(smem_u32(&peer_tail[last]), 0));
          } else {
            ok = mbar_wait_cluster(smem_u32(&peer_tail[last]), tail_phase >> last & 1u, abort_flag, err, kErrWaitDrain);
            if (ok) mbar_arrive(smem_u32(&full[last]));
          }
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        tail_phase ^= 1u << last;
      }
      tile = warp_tile(sl);
    }
  } else if (warp == 3 + kGpEpiWarps) {
    // ------------------------------------------------------------------ tiles to take over
    if (lane == 0) {
      Slot ask, got, out;
      auto request = [&] {   // (the leader's) ask for one more tile
        if (!leader) return true;
        if (!mbar_wait_cluster(smem_u32(&next_empty[ask.i]), ask.phase ^ 1u, abort_flag, err, kErrWaitProducer))
          return false;
        mbar_arrive_expect_tx(smem_u32(&next_full[ask.i]), 16);
        mbar_arrive_expect_tx_peer(mapa_shared(smem_u32(&next_full[ask.i]), 1), 16);
        clc_try_cancel(smem_u32(answers[ask.i]), smem_u32(&next_full[ask.i]));
        ask.next();
        return true;
      };
      auto answer = [&](int& tile) {
        if (!mbar_wait_cluster(smem_u32(&next_full[got.i]), got.phase, abort_flag, err, kErrWaitProducer))
          return false;
        const int cta = clc_answer(smem_u32(answers[got.i]));
        fence_proxy_async_shared();   // read before the next answer is written
        if (!leader) mbar_arrive_cluster(mapa_shared(smem_u32(&next_empty[got.i]), 0));
        got.next();
        tile = cta < 0 ? -1 : cta >> 1;
        return true;
      };
      auto hand = [&](int tile) {
        const int4 t = describe(tile);
        if (!mbar_wait(smem_u32(&tile_empty[out.i]), out.phase ^ 1u, abort_flag, err, kErrWaitProducer)) return false;
        tiles[out.i] = t;
        mbar_arrive(smem_u32(&tile_full[out.i]));
        out.next();
        return true;
      };
      const bool ok = take_tiles_over(kGwAhead, request, answer, hand);
      if (!ok) {   // gave up: let the answers in flight land
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3;                 // TMEM lane quadrant
    const int half = (warp - 2) >> 2;       // which half of the tile's columns
    int it = 0;
    Slot sl;
    for (int4 tile = first; tile.x >= 0;) {
      const Tile c = tile_of(tile);
      // this thread's column of dW, 128 of its rows; an expert without rows leaves zeros
      uint32_t s[4][32];
      if (c.kb == 0) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int i = 0; i < 32; ++i) s[x][i] = 0u;
      }
      int ok = 1;
      for (int kc = 0; kc < c.kb; kc += kGwChunk, ++it) {
        const int acc = it & 1;
        if (lane == 0) ok = mbar_wait(smem_u32(&acc_full[acc]), (it >> 1) & 1, abort_flag, err, kErrWaitEpilogue);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        tc_fence_after();
        const uint32_t trow = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                              static_cast<uint32_t>(acc * kGemmBN + half * (kGemmBN / 2));
        if (kc == 0) {
#pragma unroll
          for (int x = 0; x < 4; ++x) tmem_ld32(trow + 32u * x, s[x]);
#pragma unroll
          for (int x = 0; x < 4; ++x) tmem_ld_wait(s[x]);
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t v[32];
            tmem_ld32(trow + 32u * x, v);
            tmem_ld_wait(v);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              s[x][i] = __float_as_uint(__fadd_rn(__uint_as_float(s[x][i]), __uint_as_float(v[i])));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed_cluster(mapa_shared(smem_u32(&acc_empty[acc]), 0));
      }
      if (!ok) break;
      const int col = c.m * kPairBM + (int)rank * 128 + q * 32 + lane;
      const int n0 = c.n * kGemmBN + half * (kGemmBN / 2);
      if (col < a.K && !(c.kb == 0 && a.accumulate)) {
        float* o = a.out + ((size_t)c.z * a.N + n0) * a.K + col;
        const int left = a.N - n0;
#pragma unroll
        for (int i = 0; i < kGemmBN / 2; ++i) {
          if (i % 8 == 0 && i >= left) break;   // (N is a multiple of 8)
          const float v = __uint_as_float(s[i >> 5][i & 31]);
          if (a.accumulate) atomicAdd(o, v);    // one addition per element: no order to it
          else *o = v;
          o += a.K;
        }
      }
      tile = warp_tile(sl);
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
