// grouped_warp.cuh -- the products of grouped_mm.cuh for bf16 operands that TMA cannot take (a width
// that is no multiple of 8, a buffer off a 16-byte boundary): warp-level tensor-core products
// (mma.sync), operands read by the aligned 16 bytes that hold them and shifted in registers.
//
// BM x BN tiles, a warp WM x WN of it, 32 contraction values a step through two buffers in
// shared memory (the next step's elements are on their way in registers while this one is
// computed).  An operand whose contraction index is contiguous lies as [output][contraction],
// one whose output index is as [contraction][output], read with ldmatrix and ldmatrix.trans
// (16-byte chunks swizzled, or rows padded by 16 bytes, so that the reads do not meet in a bank).
// wgrad, and mm and dgrad with long contractions, add up their accumulators in registers every
// kGwpChunk steps (see grouped_wgrad.cuh, kGrChain in grouped_rows.cuh).
//
// 8 experts of 1000 rows, 1001 x 2003: mm 280 us, dgrad 296, wgrad 287 (108 to 115 TFLOP/s; loaded
// element by element 465, 358, 478; the FMA kernel 1210, 970, 1063).  Bound by the traffic between
// L1, registers and shared memory: most of a step's 64 wide loads touch eight lines each, and the
// MMAs' operands pass shared memory twice.
#pragma once

#include "grouped_mm.cuh"

namespace moe {

constexpr int kGwpBK = 32;
constexpr int kGwpChunk = 15;     // steps per accumulator chain of a weight gradient: 480 rows
constexpr int kGwpOneChain = 512;   // most steps of an uncut chain of mm and dgrad: 16,384 values

// The tiles' side: 64 where 128 x 128 would not give every SM a tile.
__host__ __device__ constexpr int warp_tile(int64_t tiles128, int n_sms) { return tiles128 >= n_sms ? 128 : 64; }

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

// Eight consecutive elements that start anywhere: the one or two aligned 16 bytes that hold them,
// and the elements to drop from the front.
struct WarpUnit {
  uint4 x, y;
  int drop;

  // Elements at `at`, zeros from the `valid`-th on; nothing outside [lo, hi) is read.
  __device__ __forceinline__ void load(const __nv_bfloat16* at, int valid, const __nv_bfloat16* lo,
                                       const __nv_bfloat16* hi) {
    x = y = make_uint4(0u, 0u, 0u, 0u);
    drop = 0;
    if (valid <= 0) return;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15u) >> 1;
    const __nv_bfloat16* from = at - off;
    if (valid >= 8 && from >= lo && hi - from >= (off ? 16 : 8)) {
      x = __ldg(reinterpret_cast<const uint4*>(from));
      if (off) y = __ldg(reinterpret_cast<const uint4*>(from) + 1);
      drop = off;
    } else {   // the row's end, or the buffer's
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < valid && hi - at > j)
          w[j >> 1] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(at) + j)) << (16 * (j & 1));
      x = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ uint4 aligned() const {
    const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    uint32_t u[7], v[5];
#pragma unroll
    for (int j = 0; j < 7; ++j) u[j] = drop & 2 ? w[j + 1] : w[j];
#pragma unroll
    for (int j = 0; j < 5; ++j) v[j] = drop & 4 ? u[j + 2] : u[j];
    const int bits = (drop & 1) * 16;
    return make_uint4(__funnelshift_r(v[0], v[1], bits), __funnelshift_r(v[1], v[2], bits),
                      __funnelshift_r(v[2], v[3], bits), __funnelshift_r(v[3], v[4], bits));
  }
};

// CUT: accumulators are added up every kGwpChunk steps.
template <int OP, int BM, int BN, int WM, int WN, int MINB, bool CUT>
__global__ void __launch_bounds__((BM / WM) * (BN / WN) * 32, MINB) grouped_warp_kernel(GroupedWarpArgs p) {
  constexpr int kThreads = (BM / WM) * (BN / WN) * 32;
  constexpr bool W = OP == kGroupedWgrad, kAMn = W, kBMn = OP != kGroupedMM;
  using TA = WarpTile<kAMn, BM>;
  using TB = WarpTile<kBMn, BN>;
  constexpr int kA = BM * kGwpBK / 8 / kThreads, kB = BN * kGwpBK / 8 / kThreads;   // units a thread loads
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
  const __nv_bfloat16* a_end = p.a + (size_t)p.rows * lda;
  const __nv_bfloat16* b_end = p.b + (W ? (size_t)p.rows * p.K : (size_t)p.G * p.N * p.K);
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
    WarpUnit ra[kA], rb[kB];
    // Consecutive threads along each operand's contiguous index.  Past the contraction's end
    // both operands are zeros; past an output index' end anything, since no result has it.
    auto fetch = [&](int q0) {
#pragma unroll
      for (int l = 0; l < kA; ++l) {
        const int i = tid + l * kThreads;
        const int m = m0 + (kAMn ? i % (BM / 8) * 8 : i / (kGwpBK / 8));
        const int q = q0 + (kAMn ? i / (BM / 8) : i % (kGwpBK / 8) * 8);
        ra[l].load(A + (kAMn ? (size_t)q * lda + m : (size_t)m * lda + q),
                   m >= M ? 0 : kAMn ? (q < Q ? 8 : 0) : Q - q, p.a, a_end);
      }
#pragma unroll
      for (int l = 0; l < kB; ++l) {
        const int i = tid + l * kThreads;
        const int n = n0 + (kBMn ? i % (BN / 8) * 8 : i / (kGwpBK / 8));
        const int q = q0 + (kBMn ? i / (BN / 8) : i % (kGwpBK / 8) * 8);
        rb[l].load(B + (kBMn ? (size_t)q * p.K + n : (size_t)n * p.K + q),
                   n >= out_cols ? 0 : kBMn ? (q < Q ? 8 : 0) : Q - q, p.b, b_end);
      }
    };
    auto put = [&](int buf) {
#pragma unroll
      for (int l = 0; l < kA; ++l) {
        const int i = tid + l * kThreads;
        const int o = kAMn ? i % (BM / 8) * 8 : i / (kGwpBK / 8), q = kAMn ? i / (BM / 8) : i % (kGwpBK / 8) * 8;
        *reinterpret_cast<uint4*>(&As[buf][TA::at(o, q)]) = ra[l].aligned();
      }
#pragma unroll
      for (int l = 0; l < kB; ++l) {
        const int i = tid + l * kThreads;
        const int o = kBMn ? i % (BN / 8) * 8 : i / (kGwpBK / 8), q = kBMn ? i / (BN / 8) : i % (kGwpBK / 8) * 8;
        *reinterpret_cast<uint4*>(&Bs[buf][TB::at(o, q)]) = rb[l].aligned();
      }
    };
    float acc[MI][NI][4], sum[CUT ? MI : 1][CUT ? NI : 1][4];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          acc[i][j][x] = 0.f;
          if constexpr (CUT) sum[i][j][x] = 0.f;
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
        if constexpr (CUT) {
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
          float v = acc[i][j][x];
          if constexpr (CUT) v += sum[i][j][x];
          if constexpr (W) {
            if (Q == 0 && p.accumulate) continue;   // nothing to add: not touched
            float* o = static_cast<float*>(p.out) + (((size_t)part * p.G + g) * p.N + m) * p.K + n;
            *o = p.accumulate ? *o + v : v;
          } else {
            static_cast<__nv_bfloat16*>(p.out)[(size_t)(grow0 + m) * out_cols + n] = __float2bfloat16_rn(v);
          }
        }
  }
}

}  // namespace moe
