// grouped_warp.cuh -- the products of grouped_mm.cuh for bf16 operands that TMA cannot take (a width
// that is no multiple of 8, a buffer off a 16-byte boundary): warp-level tensor-core products
// (mma.sync), operands loaded element by element.
//
// BM x BN tiles, a warp WM x WN of it, 32 contraction values a step through two buffers in
// shared memory (the next step's elements are on their way in registers while this one is
// computed).  An operand whose contraction index is contiguous lies as [output][contraction],
// one whose output index is as [contraction][output], read with ldmatrix and ldmatrix.trans
// (16-byte chunks swizzled, or rows padded by 16 bytes, so that the reads do not meet in a bank).
// wgrad adds up its accumulators in registers every kGwpChunk steps (see grouped_wgrad.cuh).
//
// Bound by the element-wise loads: 8 experts of 1000 rows, 1001 x 2003: mm 464 us, dgrad 358, wgrad
// 423 (69 to 90 TFLOP/s; the FMA kernel 1210, 970, 1063).
#pragma once

#include "grouped_mm.cuh"

namespace moe {

constexpr int kGwpBK = 32;
constexpr int kGwpChunk = 15;   // steps per accumulator chain of a weight gradient: 480 rows

struct GroupedWarpArgs {
  const __nv_bfloat16* a;   // mm: x, dgrad: dy, wgrad: dy
  const __nv_bfloat16* b;   // mm, dgrad: W, wgrad: x
  const int32_t* counts;
  void* out;
  int G, rows, N, K;        // of the layer: W is [G, N, K]
  int accumulate;           // wgrad: add to out
  int splits;               // wgrad: parts of the rows, each with its own [G, N, K] in out
};

template <bool TRANS>
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One operand's tile in shared memory: TILE output indices x kGwpBK contraction values.
template <bool MN, int TILE>
struct WarpTile {
  static constexpr int kStride = MN ? TILE + 8 : kGwpBK;   // elements
  static constexpr int kSize = (MN ? kGwpBK : TILE) * kStride;
  static __device__ __forceinline__ int at(int o, int q) {
    return MN ? q * kStride + o : o * kStride + (((q >> 3) ^ (o >> 1 & 3)) << 3) + (q & 7);
  }
};

template <int OP, int BM, int BN, int WM, int WN, int MINB>
__global__ void __launch_bounds__((BM / WM) * (BN / WN) * 32, MINB) grouped_warp_kernel(GroupedWarpArgs p) {
  constexpr int kThreads = (BM / WM) * (BN / WN) * 32;
  constexpr bool W = OP == kGroupedWgrad, kAMn = W, kBMn = OP != kGroupedMM;
  using TA = WarpTile<kAMn, BM>;
  using TB = WarpTile<kBMn, BN>;
  constexpr int kA = BM * kGwpBK / kThreads, kB = BN * kGwpBK / kThreads;   // elements a thread loads
  constexpr int MI = WM / 16, NI = WN / 8;
  pdl_launch_dependents();
  pdl_wait();
  __shared__ GroupTable tab;
  __shared__ __align__(16) __nv_bfloat16 As[2][TA::kSize];
  __shared__ __align__(16) __nv_bfloat16 Bs[2][TB::kSize];
  const int out_cols = OP == kGroupedMM ? p.N : p.K;
  const int nt = (out_cols + BN - 1) / BN;
  const int mt_w = (p.N + BM - 1) / BM;   // row tiles of a weight gradient
  group_table(tab, p.counts, p.G, p.rows, W ? 0 : BM, W ? nt * mt_w * p.splits : nt);
  const int total = tab.tile0[p.G];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp % (BM / WM) * WM, wn = warp / (BM / WM) * WN;
  const int lda = OP == kGroupedMM ? p.K : p.N;
  for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
    const int g = group_of(tab, p.G, tile);
    int local = tile - tab.tile0[g], part = 0;
    int grow0 = tab.row0[g], grows = tab.row0[g + 1] - grow0;
    if constexpr (W) {
      part = local / (nt * mt_w);
      local -= part * (nt * mt_w);
      split_rows(grow0, grows, p.splits, part);
    }
    const int m0 = local / nt * BM, n0 = (local - local / nt * nt) * BN;
    const int M = W ? p.N : grows;
    const int Q = OP == kGroupedMM ? p.K : OP == kGroupedDgrad ? p.N : grows;
    const __nv_bfloat16* A = p.a + (size_t)grow0 * lda;
    const __nv_bfloat16* B = p.b + (W ? (size_t)grow0 * p.K : (size_t)g * p.N * p.K);
    __nv_bfloat16 ra[kA], rb[kB];
    const __nv_bfloat16 zero = __float2bfloat16_rn(0.f);
    // consecutive threads along each operand's contiguous index
    auto fetch = [&](int q0) {
#pragma unroll
      for (int l = 0; l < kA; ++l) {
        const int i = tid + l * kThreads;
        const int m = m0 + (kAMn ? i % BM : i / kGwpBK), q = q0 + (kAMn ? i / BM : i % kGwpBK);
        ra[l] = m < M && q < Q ? A[kAMn ? (size_t)q * lda + m : (size_t)m * lda + q] : zero;
      }
#pragma unroll
      for (int l = 0; l < kB; ++l) {
        const int i = tid + l * kThreads;
        const int n = n0 + (kBMn ? i % BN : i / kGwpBK), q = q0 + (kBMn ? i / BN : i % kGwpBK);
        rb[l] = n < out_cols && q < Q ? B[kBMn ? (size_t)q * p.K + n : (size_t)n * p.K + q] : zero;
      }
    };
    auto put = [&](int buf) {
#pragma unroll
      for (int l = 0; l < kA; ++l) {
        const int i = tid + l * kThreads;
        As[buf][TA::at(kAMn ? i % BM : i / kGwpBK, kAMn ? i / BM : i % kGwpBK)] = ra[l];
      }
#pragma unroll
      for (int l = 0; l < kB; ++l) {
        const int i = tid + l * kThreads;
        Bs[buf][TB::at(kBMn ? i % BN : i / kGwpBK, kBMn ? i / BN : i % kGwpBK)] = rb[l];
      }
    };
    float acc[MI][NI][4], sum[W ? MI : 1][W ? NI : 1][4];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          acc[i][j][x] = 0.f;
          if constexpr (W) sum[i][j][x] = 0.f;
        }
    if (Q > 0) {
      fetch(0);
      __syncthreads();   // the previous tile's last step has been read
      put(0);
      __syncthreads();
      int buf = 0, step = 0;
      for (int q0 = 0; q0 < Q; q0 += kGwpBK, buf ^= 1) {
        const bool more = q0 + kGwpBK < Q;
        if (more) fetch(q0 + kGwpBK);
#pragma unroll
        for (int k = 0; k < kGwpBK; k += 16) {
          uint32_t fa[MI][4];
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            const int m = wm + i * 16;
            const int o = kAMn ? TA::at(m + (lane >> 3 & 1) * 8, k + (lane & 7) + (lane >> 4) * 8)
                               : TA::at(m + (lane & 15), k + (lane >> 4) * 8);
            ldmatrix_x4<kAMn>(smem_u32(&As[buf][o]), fa[i]);
          }
#pragma unroll
          for (int j = 0; j < NI; j += 2) {
            uint32_t fb[4];
            const int n = wn + j * 8;
            const int o = kBMn ? TB::at(n + (lane >> 4) * 8, k + (lane & 7) + (lane >> 3 & 1) * 8)
                               : TB::at(n + (lane >> 4) * 8 + (lane & 7), k + (lane >> 3 & 1) * 8);
            ldmatrix_x4<kBMn>(smem_u32(&Bs[buf][o]), fb);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
              mma_16816(acc[i][j], fa[i], fb[0], fb[1]);
              mma_16816(acc[i][j + 1], fa[i], fb[2], fb[3]);
            }
          }
        }
        if constexpr (W) {
          if (++step % kGwpChunk == 0) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
              for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  sum[i][j][x] += acc[i][j][x];
                  acc[i][j][x] = 0.f;
                }
          }
        }
        if (more) {
          put(buf ^ 1);
          __syncthreads();
        }
      }
    }
    // accumulator (i, j): rows lane / 4 and + 8, columns 2 (lane % 4) and + 1
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int m = m0 + wm + i * 16 + (lane >> 2) + (x >> 1) * 8;
          const int n = n0 + wn + j * 8 + (lane & 3) * 2 + (x & 1);
          if (m >= M || n >= out_cols) continue;
          if constexpr (W) {
            if (Q == 0 && p.accumulate) continue;   // nothing to add: not touched
            float* o = static_cast<float*>(p.out) + (((size_t)part * p.G + g) * p.N + m) * p.K + n;
            const float v = sum[i][j][x] + acc[i][j][x];
            *o = p.accumulate ? *o + v : v;
          } else {
            static_cast<__nv_bfloat16*>(p.out)[(size_t)(grow0 + m) * out_cols + n] = __float2bfloat16_rn(acc[i][j][x]);
          }
        }
  }
}

}  // namespace moe
