// grouped_mm.cuh -- matrix products grouped by expert over ragged rows.
//
// Expert e of G owns counts[e] consecutive rows (experts in order, no padding):
//   mm:     y[r, :]  = x[r, :] W_e^T        x [rows, K], W [G, N, K], y [rows, N]
//   dgrad:  dx[r, :] = dy[r, :] W_e         dy [rows, N], dx [rows, K]
//   wgrad:  dW_e     = dy_e^T x_e           dW [G, N, K] fp32, the sum over the expert's rows
// counts stays on the device (a router writes it): each CTA scans it in its prologue, so a
// product is one launch.  Rows behind the last expert's are neither read into a result nor
// written.
//
// A weight gradient with fewer tiles than the GPU has room for, and long sums, is split: each
// expert's rows in `splits` parts, each part a gradient of its own in the workspace, added up in
// order by a second kernel.
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

// Tiles of bm x bn at most (every expert with rows has one ragged tile row).
__host__ __device__ constexpr int64_t grouped_tiles(int op, int64_t G, int64_t rows, int64_t n, int64_t k, int bm,
                                                    int bn) {
  const int64_t nt = ((op == kGroupedMM ? n : k) + bn - 1) / bn;
  return op == kGroupedWgrad ? G * nt * ((n + bm - 1) / bm) : ((rows + bm - 1) / bm + (G < rows ? G : rows)) * nt;
}

// Parts of each expert's rows in a weight gradient of `tiles` tiles whose kernel has room for
// `slots`: as many as fit, of at least `least` rows on average, 256 at most.
__host__ __device__ constexpr int wgrad_splits(int64_t rows, int G, int64_t tiles, int slots, int least) {
  const int64_t fill = slots / tiles, rest = rows / G / least;
  const int64_t s = fill < rest ? fill : rest;
  return s < 1 ? 1 : s > 256 ? 256 : (int)s;
}
// The same by the shape: for the tensor cores' kernel of 256 x 256 tiles (`tma`), or the others'
// smaller ones.  (Slots are those of a B200's 148 SMs, so that the workspace's size needs no device.)
// One expert of 100,000 rows, 64 x 64: 28 us in 74 parts, 0.5 ms in one; 72 tiles for 74 slots stay
// whole (split in two, 796 us against 478 for 65,536 rows).
__host__ __device__ constexpr int wgrad_parts(int G, int64_t rows, int n, int k, bool tma) {
  constexpr int kSms = 148;
  return tma ? wgrad_splits(rows, G, grouped_tiles(kGroupedWgrad, G, rows, n, k, 256, 256), kSms / 2, 1024)
             : wgrad_splits(rows, G, grouped_tiles(kGroupedWgrad, G, rows, n, k, 64, 64), 4 * kSms, 512);
}
// Part s of an expert's rows: whole MMA steps of 16 rows but for the last part.
__host__ __device__ inline void split_rows(int& row0, int& rows, int splits, int s) {
  const int per = ((rows + splits - 1) / splits + 15) & ~15;
  const int lo = s * per < rows ? s * per : rows;
  rows = rows - lo < per ? rows - lo : per;
  row0 += lo;
}

// dst[i] (+)= sum over the parts, in order.  V elements a thread and step.
template <int V>
__global__ void __launch_bounds__(256) wgrad_sum_kernel(const float* part, int splits, int64_t n, int accumulate,
                                                        float* dst) {
  pdl_launch_dependents();
  pdl_wait();
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V; i < n; i += (int64_t)gridDim.x * 256 * V) {
    float v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = 0.f;
    for (int s = 0; s < splits; ++s) {
      const float* p = part + (int64_t)s * n + i;
      if constexpr (V == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
      } else {
        v[0] += *p;
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) dst[i + j] = accumulate ? dst[i + j] + v[j] : v[j];
  }
}

// ------------------------------------------------------------------------ CUDA cores
// fp32 operands: fp32 FMA (two per instruction) on BM x BN tiles, a thread R x R outputs, 16-deep
// steps through two buffers in shared memory (the next step's elements are on their way in
// registers while this one is computed).  V elements a load: 4 when the widths are multiples of 4
// and the buffers 16-byte aligned, else 1.  Sums are cut into pieces of kGsChunk steps, added up
// apart: one chain of 4096 additions is off by 1e-6 of the result, pieces by a third of that.
// On the larger tiles 35 to 40 of the FMA units' 74 TFLOP/s (16 experts of 500 rows, 512 x 512: 116
// us; 4 of 2368, 1024 x 1024: 497 to 543; a library's batched product of equal sizes 45 to 61): a
// contraction value costs a thread four 16-byte shared loads for 32 paired FMAs.  The smallest are
// bound by latency (15 of 26 rows, 128 x 256: 9 to 10 us).
constexpr int kGsBK = 16;
constexpr int kGsChunk = 16;   // steps: 256 products

struct GroupedSimtArgs {
  const void* a;        // mm: x, dgrad: dy, wgrad: dy
  const void* b;        // mm, dgrad: W, wgrad: x
  const int32_t* counts;
  void* out;
  int G, rows, N, K;    // of the layer: W is [G, N, K]
  int accumulate;       // wgrad: add to out
  int splits;           // wgrad: parts of the rows, each with its own [G, N, K] in out
};

// Two fp32 fused multiply-adds, each rounded to nearest.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
        "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&d);
}

// OP's tile: rows of out (M index) x columns (N index), contraction index q:
//   mm:    A[m, q] = x[row0 + m][q]       B[n, q] = W[n][q]      q < K
//   dgrad: A[m, q] = dy[row0 + m][q]      B[n, q] = W[q][n]      q < N
//   wgrad: A[m, q] = dy[row0 + q][m]      B[n, q] = x[row0 + q][n]   q < rows of the group
// KS > 1: the CTA has KS such sets of threads, each with its own buffers and every KS-th step of the
// contraction; the sets' sums meet in shared memory, added in order.
// BM = 128: the pieces' sums wait in shared memory (each thread's own words), so that a thread gets
// by with 128 registers and an SM holds two CTAs (4 experts of 2368 rows, 1024 x 1024: mm 598 us ->
// 542, dgrad 593 -> 512; 16 of 500, 512 x 512, where there are few tiles for them, 114 -> 116).
constexpr bool simt_sums_shared(int bm) { return bm == 128; }
constexpr size_t simt_smem_bytes(int bm, int bn) {
  return simt_sums_shared(bm) ? (size_t)bm * bn * sizeof(float) : 0;
}
// The tiles' side: the largest that gives every SM two CTAs of 128 x 128 or three of 64 x 64; small
// problems take 32 x 32 with the contraction over four sets of threads (one expert of 384 rows,
// 1024 x 1024: 68 us -> 45) and one element a load (16-byte loads turned into K-major rows of so
// small a tile cost more than they save: 60 experts of 25 rows, 200 x 332, 27 us against 41; on
// larger tiles they save: 4 experts of 500 rows, 1000 x 1000, 126 us against 155).
__host__ __device__ constexpr int simt_tile(int64_t tiles128, int64_t tiles64, int n_sms) {
  return tiles128 >= 2 * n_sms ? 128 : tiles64 >= 3 * n_sms ? 64 : 32;
}
template <int OP, int BM, int BN, int R, int V, int KS>
__global__ void __launch_bounds__(BM * BN / (R * R) * KS, KS > 1 || simt_sums_shared(BM) ? 2 : 1)
grouped_simt_kernel(GroupedSimtArgs p) {
  constexpr bool kShared = simt_sums_shared(BM);
  extern __shared__ float2 piece_sums[];
  constexpr int kThreads = BM * BN / (R * R);   // of a set
  constexpr int kA = BM * kGsBK / kThreads / V, kB = BN * kGsBK / kThreads / V;   // loads of a thread
  constexpr bool W = OP == kGroupedWgrad;
  pdl_launch_dependents();
  pdl_wait();
  __shared__ GroupTable tab;
  __shared__ __align__(16) float Asets[KS][2][kGsBK][BM + 4];
  __shared__ __align__(16) float Bsets[KS][2][kGsBK][BN + 4];
  static_assert(KS == 1 || sizeof(Asets) >= sizeof(float) * (KS - 1) * kThreads * R * R, "the sums' meeting place");
  const int set = threadIdx.x / kThreads;
  auto& As = Asets[set];
  auto& Bs = Bsets[set];
  auto set_sync = [&] {
    if constexpr (KS == 1) __syncthreads();
    else named_bar_sync(1 + set, kThreads);
  };
  const int out_cols = OP == kGroupedMM ? p.N : p.K;
  const int nt = (out_cols + BN - 1) / BN;
  const int mt_w = (p.N + BM - 1) / BM;   // row tiles of a weight gradient
  group_table(tab, p.counts, p.G, p.rows, W ? 0 : BM, W ? nt * mt_w * p.splits : nt);
  const int total = tab.tile0[p.G];
  const int tid = threadIdx.x % kThreads, tx = tid % (BN / R), ty = tid / (BN / R);
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
    const float* A = static_cast<const float*>(p.a) + (size_t)grow0 * lda;
    const float* B = static_cast<const float*>(p.b) + (W ? (size_t)grow0 * p.K : (size_t)g * p.N * p.K);
    float ra[kA][V], rb[kB][V];
    // consecutive threads along each operand's contiguous index
    constexpr bool kAMn = W, kBMn = OP != kGroupedMM;   // contiguous along the output index
    constexpr int kQv = kGsBK / V;
    auto load = [&](float (&r)[V], const float* src, bool in) {
      if constexpr (V == 4) {
        const float4 v = in ? *reinterpret_cast<const float4*>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
        r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
      } else {
        r[0] = in ? *src : 0.f;
      }
    };
    auto fetch = [&](int q0) {
#pragma unroll
      for (int l = 0; l < kA; ++l) {
        const int i = tid + l * kThreads;
        const int m = m0 + (kAMn ? i % (BM / V) * V : i / kQv), q = q0 + (kAMn ? i / (BM / V) : i % kQv * V);
        load(ra[l], A + (kAMn ? (size_t)q * lda + m : (size_t)m * lda + q), m < M && q < Q);
      }
#pragma unroll
      for (int l = 0; l < kB; ++l) {
        const int i = tid + l * kThreads;
        const int n = n0 + (kBMn ? i % (BN / V) * V : i / kQv), q = q0 + (kBMn ? i / (BN / V) : i % kQv * V);
        load(rb[l], B + (kBMn ? (size_t)q * p.K + n : (size_t)n * p.K + q), n < out_cols && q < Q);
      }
    };
    auto put = [&](int buf) {
#pragma unroll
      for (int l = 0; l < kA; ++l) {
        const int i = tid + l * kThreads;
#pragma unroll
        for (int v = 0; v < V; ++v)
          As[buf][kAMn ? i / (BM / V) : i % kQv * V + v][kAMn ? i % (BM / V) * V + v : i / kQv] = ra[l][v];
      }
#pragma unroll
      for (int l = 0; l < kB; ++l) {
        const int i = tid + l * kThreads;
#pragma unroll
        for (int v = 0; v < V; ++v)
          Bs[buf][kBMn ? i / (BN / V) : i % kQv * V + v][kBMn ? i % (BN / V) * V + v : i / kQv] = rb[l][v];
      }
    };
    // a thread's outputs: R / 4 runs of four rows (columns), BM / (R / 4) (BN / (R / 4)) apart
    float2 acc[R][R / 2], sum[kShared ? 1 : R][R / 2];
    bool pieces = false;   // (kShared) sums are waiting
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < R / 2; ++j) {
        acc[i][j] = make_float2(0.f, 0.f);
        if constexpr (!kShared) sum[i][j] = make_float2(0.f, 0.f);
      }
    constexpr int kRunM = BM / (R / 4), kRunN = BN / (R / 4);
    __syncthreads();   // the previous tile's last step, and its sums, have been read
    if (set * kGsBK < Q) {
      fetch(set * kGsBK);
      put(0);
      set_sync();
      int buf = 0, steps = 0;
      for (int q0 = set * kGsBK; q0 < Q; q0 += KS * kGsBK, buf ^= 1) {
        const bool more = q0 + KS * kGsBK < Q;
        if (more) fetch(q0 + KS * kGsBK);
#pragma unroll
        for (int q = 0; q < kGsBK; ++q) {
          float av[R];
          float2 bv[R / 2];
#pragma unroll
          for (int i = 0; i < R; i += 4) {
            *reinterpret_cast<float4*>(&av[i]) = *reinterpret_cast<const float4*>(&As[buf][q][i / 4 * kRunM + ty * 4]);
            *reinterpret_cast<float4*>(&bv[i / 2]) = *reinterpret_cast<const float4*>(&Bs[buf][q][i / 4 * kRunN + tx * 4]);
          }
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < R / 2; ++j) acc[i][j] = fma2(make_float2(av[i], av[i]), bv[j], acc[i][j]);
        }
        if (++steps == kGsChunk) {
          steps = 0;
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < R / 2; ++j) {
              if constexpr (kShared) {
                float2& s = piece_sums[(i * (R / 2) + j) * kThreads + tid];
                s = pieces ? make_float2(s.x + acc[i][j].x, s.y + acc[i][j].y) : acc[i][j];
              } else {
                sum[i][j].x += acc[i][j].x;
                sum[i][j].y += acc[i][j].y;
              }
              acc[i][j] = make_float2(0.f, 0.f);
            }
          pieces = true;
        }
        if (more) {
          put(buf ^ 1);
          set_sync();
        }
      }
    }
    if constexpr (KS > 1) {
      float* meet = &Asets[0][0][0][0];
      __syncthreads();   // every set is done with its buffers
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < R / 2; ++j) {
          sum[i][j].x += acc[i][j].x;
          sum[i][j].y += acc[i][j].y;
          acc[i][j] = make_float2(0.f, 0.f);
          if (set > 0)
            *reinterpret_cast<float2*>(meet + (((set - 1) * R * R + i * R + 2 * j) * kThreads) + 2 * tid) = sum[i][j];
        }
      __syncthreads();
      if (set > 0) continue;
#pragma unroll
      for (int k = 0; k < KS - 1; ++k)
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < R / 2; ++j) {
            const float2 x = *reinterpret_cast<const float2*>(meet + ((k * R * R + i * R + 2 * j) * kThreads) + 2 * tid);
            sum[i][j].x += x.x;
            sum[i][j].y += x.y;
          }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int m = m0 + i / 4 * kRunM + ty * 4 + i % 4;
      if (m >= M) continue;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int n = n0 + j / 4 * kRunN + tx * 4 + j % 4;
        if (n >= out_cols) continue;
        float v = j & 1 ? acc[i][j / 2].y : acc[i][j / 2].x;
        if constexpr (!kShared) {
          v += j & 1 ? sum[i][j / 2].y : sum[i][j / 2].x;
        } else if (pieces) {
          const float2 s = piece_sums[(i * (R / 2) + j / 2) * kThreads + tid];
          v += j & 1 ? s.y : s.x;
        }
        if constexpr (W) {
          if (Q == 0 && p.accumulate) continue;   // nothing to add: not touched
          float* o = static_cast<float*>(p.out) + (((size_t)part * p.G + g) * p.N + m) * p.K + n;
          *o = p.accumulate ? *o + v : v;
        } else {
          static_cast<float*>(p.out)[(size_t)(grow0 + m) * out_cols + n] = v;
        }
      }
    }
  }
}

}  // namespace moe
