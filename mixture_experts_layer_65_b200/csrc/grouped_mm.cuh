// grouped_mm.cuh -- matrix products grouped by expert over ragged rows.
//
// Expert e of G owns counts[e] consecutive rows (experts in order, no padding):
//   mm:     y[r, :]  = x[r, :] W_e^T        x [rows, K], W [G, N, K], y [rows, N]
//   dgrad:  dx[r, :] = dy[r, :] W_e         dy [rows, N], dx [rows, K]
//   wgrad:  dW_e     = dy_e^T x_e           dW [G, N, K] fp32, the sum over the expert's rows
// counts stays on the device (a router writes it): each CTA scans it in its prologue, so a
// product is one launch and needs no workspace.  Rows behind the last expert's are neither
// read into a result nor written.
#pragma once

#include "ptx.cuh"

namespace moe {

constexpr int kGroupedMaxGroups = 1024;

enum GroupedOp : int { kGroupedMM = 0, kGroupedDgrad = 1, kGroupedWgrad = 2 };

// The groups' first rows and tile prefix, in shared memory.
struct GroupTable {
  int32_t row0[kGroupedMaxGroups + 1];
  int32_t tile0[kGroupedMaxGroups + 1];
};

// The groups' first rows from counts: row0[g], and row0[G] the end of the last.  A negative
// count counts as 0 and rows past `rows` are cut off, so no index leaves the buffers.  Called by
// the whole CTA (a multiple of 32 threads); ends with a barrier.
__device__ __forceinline__ void group_rows(int32_t* row0, const int32_t* counts, int G, int rows) {
  __shared__ int64_t warp_rows[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // each thread owns a run of consecutive groups
  const int per = (G + (int)blockDim.x - 1) / (int)blockDim.x;
  const int g0 = tid * per < G ? tid * per : G;
  const int g1 = g0 + per < G ? g0 + per : G;
  int64_t c = 0;
  for (int g = g0; g < g1; ++g) {
    const int n = __ldg(counts + g);
    c += n > 0 ? n : 0;
  }
  int64_t inc = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) warp_rows[warp] = inc;
  __syncthreads();
  int64_t r = inc - c;
  for (int w = 0; w < warp; ++w) r += warp_rows[w];
  for (int g = g0; g < g1; ++g) {
    row0[g] = r < rows ? (int)r : rows;
    const int n = __ldg(counts + g);
    r += n > 0 ? n : 0;
    if (g == G - 1) row0[G] = r < rows ? (int)r : rows;
  }
  __syncthreads();
}

// The table: first rows, and the tile prefix -- nt tiles per `bm` rows of a group, or (bm == 0)
// nt tiles whatever its rows.  As group_rows.
__device__ __forceinline__ void group_table(GroupTable& t, const int32_t* counts, int G, int rows, int bm,
                                            int nt) {
  __shared__ int32_t warp_tiles[32];
  group_rows(t.row0, counts, G, rows);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (G + (int)blockDim.x - 1) / (int)blockDim.x;
  const int g0 = tid * per < G ? tid * per : G;
  const int g1 = g0 + per < G ? g0 + per : G;
  auto tiles_of = [&](int g) { return bm ? (t.row0[g + 1] - t.row0[g] + bm - 1) / bm * nt : nt; };
  int c = 0;
  for (int g = g0; g < g1; ++g) c += tiles_of(g);
  int inc = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) warp_tiles[warp] = inc;
  __syncthreads();
  int tile = inc - c;
  for (int w = 0; w < warp; ++w) tile += warp_tiles[w];
  for (int g = g0; g < g1; ++g) {
    t.tile0[g] = tile;
    tile += tiles_of(g);
    if (g == G - 1) t.tile0[G] = tile;
  }
  __syncthreads();
}

// The group of a tile: the last one whose tiles start at or before it (groups without tiles
// share their successor's start).
__device__ __forceinline__ int group_of(const GroupTable& t, int G, int tile) {
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.tile0[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// ------------------------------------------------------------------------ CUDA cores
// fp32 operands, and bf16 ones whose widths or addresses TMA cannot take: 64 x 64 tiles,
// 16-deep steps, 4 x 4 outputs a thread, fp32 FMA.
constexpr int kGsBM = 64, kGsBN = 64, kGsBK = 16, kGsThreads = 256;

struct GroupedSimtArgs {
  const void* a;        // mm: x, dgrad: dy, wgrad: dy
  const void* b;        // mm, dgrad: W, wgrad: x
  const int32_t* counts;
  void* out;
  int G, rows, N, K;    // of the layer: W is [G, N, K]
  int accumulate;       // wgrad: add to out
};

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(v);
  else return v;
}

// OP's tile: rows of out (M index) x columns (N index), contraction index q:
//   mm:    A[m, q] = x[row0 + m][q]       B[n, q] = W[n][q]      q < K
//   dgrad: A[m, q] = dy[row0 + m][q]      B[n, q] = W[q][n]      q < N
//   wgrad: A[m, q] = dy[row0 + q][m]      B[n, q] = x[row0 + q][n]   q < rows of the group
template <typename T, int OP>
__global__ void __launch_bounds__(kGsThreads) grouped_simt_kernel(GroupedSimtArgs p) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ GroupTable tab;
  __shared__ float As[kGsBK][kGsBM + 4];
  __shared__ float Bs[kGsBK][kGsBN + 4];
  constexpr bool W = OP == kGroupedWgrad;
  const int out_cols = OP == kGroupedMM ? p.N : p.K;
  const int nt = (out_cols + kGsBN - 1) / kGsBN;
  const int mt_w = (p.N + kGsBM - 1) / kGsBM;   // row tiles of a weight gradient
  group_table(tab, p.counts, p.G, p.rows, W ? 0 : kGsBM, W ? nt * mt_w : nt);
  const int total = tab.tile0[p.G];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
    const int g = group_of(tab, p.G, tile);
    const int local = tile - tab.tile0[g];
    const int m0 = local / nt * kGsBM, n0 = (local - local / nt * nt) * kGsBN;
    const int grow0 = tab.row0[g], grows = tab.row0[g + 1] - grow0;
    const int M = W ? p.N : grows;
    const int Q = OP == kGroupedMM ? p.K : OP == kGroupedDgrad ? p.N : grows;
    const T* A = static_cast<const T*>(p.a) + (size_t)grow0 * (OP == kGroupedMM ? p.K : p.N);
    const T* B = static_cast<const T*>(p.b) + (W ? (size_t)grow0 * p.K : (size_t)g * p.N * p.K);
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    for (int q0 = 0; q0 < Q; q0 += kGsBK) {
#pragma unroll
      for (int l = 0; l < kGsBM * kGsBK / kGsThreads; ++l) {
        const int idx = tid + l * kGsThreads;
        // consecutive threads along the operand's contiguous index
        int m, q;
        if constexpr (W) { m = idx % kGsBM; q = idx / kGsBM; }
        else { q = idx % kGsBK; m = idx / kGsBK; }
        float v = 0.f;
        if (m0 + m < M && q0 + q < Q)
          v = to_f32(W ? A[(size_t)(q0 + q) * p.N + m0 + m]
                       : A[(size_t)(m0 + m) * (OP == kGroupedMM ? p.K : p.N) + q0 + q]);
        As[q][m] = v;
        int n, r;
        if constexpr (OP == kGroupedMM) { r = idx % kGsBK; n = idx / kGsBK; }
        else { n = idx % kGsBN; r = idx / kGsBN; }
        v = 0.f;
        if (n0 + n < out_cols && q0 + r < Q)
          v = to_f32(OP == kGroupedMM ? B[(size_t)(n0 + n) * p.K + q0 + r] : B[(size_t)(q0 + r) * p.K + n0 + n]);
        Bs[r][n] = v;
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kGsBK; ++q) {
        float av[4], bv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) av[i] = As[q][ty * 4 + i];
#pragma unroll
        for (int j = 0; j < 4; ++j) bv[j] = Bs[q][tx * 4 + j];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + ty * 4 + i;
      if (m >= M) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx * 4 + j;
        if (n >= out_cols) continue;
        if constexpr (W) {
          float* o = static_cast<float*>(p.out) + ((size_t)g * p.N + m) * p.K + n;
          *o = p.accumulate ? *o + acc[i][j] : acc[i][j];
        } else {
          T* o = static_cast<T*>(p.out) + (size_t)(grow0 + m) * out_cols + n;
          if constexpr (sizeof(T) == 2) *o = __float2bfloat16_rn(acc[i][j]);
          else *o = acc[i][j];
        }
      }
    }
  }
}

}  // namespace moe
