// moe_grouped.cu -- moe_grouped_mm, moe_grouped_mm_dgrad and moe_grouped_mm_wgrad
// (include/moe.h): checks, the choice of kernel, TMA descriptors and the launch.
#include "op_common.cuh"
#include "grouped_mm.cuh"
#include "grouped_rows.cuh"
#include "grouped_warp.cuh"
#include "grouped_wgrad.cuh"

using namespace moe;

namespace {

struct Shape {
  int32_t G;
  int64_t rows;
  int32_t n, k, dtype;
};

moe_status check_shape(const Shape& s) {
  if (s.dtype != MOE_BF16 && s.dtype != MOE_FP32)
    return fail(MOE_ERR_INVALID_ARG, "dtype=%d is not MOE_FP32 or MOE_BF16", s.dtype);
  if (s.G < 1 || s.G > kGroupedMaxGroups)
    return fail(MOE_ERR_UNSUPPORTED, "n_groups=%d outside [1, %d]", s.G, kGroupedMaxGroups);
  if (s.n < 1 || s.k < 1) return fail(MOE_ERR_INVALID_ARG, "n and k must be positive");
  if (s.n > (1 << 20) || s.k > (1 << 20)) return fail(MOE_ERR_UNSUPPORTED, "n=%d or k=%d above 2^20", s.n, s.k);
  if (s.rows < 0) return fail(MOE_ERR_INVALID_ARG, "rows must not be negative");
  // (one tile of a weight gradient whose expert has all the rows has to end well within the
  // kernels' bounded waits: 2^28 rows are 2^21 stages of at most half a microsecond)
  if (s.rows >= (int64_t(1) << 28)) return fail(MOE_ERR_UNSUPPORTED, "rows=%lld not below 2^28", (long long)s.rows);
  // tiles of the smallest kind, all groups together, are counted in 32 bits
  const int64_t nt = (s.n + 31) / 32, kt = (s.k + 31) / 32;
  const int64_t mt = (s.rows + 31) / 32 + s.G;
  if (mt * (nt > kt ? nt : kt) >= (int64_t(1) << 31) || nt * kt * s.G >= (int64_t(1) << 30))
    return fail(MOE_ERR_UNSUPPORTED, "too many tiles");
  return MOE_OK;
}

template <int OP>
int64_t tiles_of(const Shape& s, int bm, int bn) { return grouped_tiles(OP, s.G, s.rows, s.n, s.k, bm, bn); }

// fp32 (simt_tile).
template <int OP, int BM, int BN, int R, int V, int KS>
cudaError_t launch_simt_tile(const GroupedSimtArgs& a, const Shape& s, int n_sms, cudaStream_t st) {
  constexpr int kThreads = BM * BN / (R * R) * KS;
  constexpr size_t kSmem = simt_smem_bytes(BM, BN);
  const auto kernel = grouped_simt_kernel<OP, BM, BN, R, V, KS>;
  const int64_t tiles = a.splits * tiles_of<OP>(s, BM, BN), most = (int64_t)n_sms * ((kSmem ? 512 : 1024) / kThreads);
  if constexpr (kSmem > 0) {   // (once per device)
    static std::atomic<bool> set[64];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess && !(device < 64 && set[device].load(std::memory_order_acquire)))
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    if (device < 64) set[device].store(true, std::memory_order_release);
  }
  return launch_pdl(kernel, dim3((unsigned)(tiles < most ? tiles : most)), dim3(kThreads), kSmem, st, a);
}
template <int OP>
cudaError_t launch_simt(const GroupedSimtArgs& a, const Shape& s, int n_sms, cudaStream_t st) {
  const bool v4 = s.n % 4 == 0 && s.k % 4 == 0 && aligned16(a.a) && aligned16(a.b);
  switch (simt_tile(a.splits * tiles_of<OP>(s, 128, 128), a.splits * tiles_of<OP>(s, 64, 64), n_sms)) {
    case 128:
      return v4 ? launch_simt_tile<OP, 128, 128, 8, 4, 1>(a, s, n_sms, st)
                : launch_simt_tile<OP, 128, 128, 8, 1, 1>(a, s, n_sms, st);
    case 64:
      return v4 ? launch_simt_tile<OP, 64, 64, 8, 4, 1>(a, s, n_sms, st)
                : launch_simt_tile<OP, 64, 64, 8, 1, 1>(a, s, n_sms, st);
    default:
      return launch_simt_tile<OP, 32, 32, 4, 1, 4>(a, s, n_sms, st);
  }
}

// bf16 that TMA cannot take (warp_tile).  Weight gradients and long contractions, which keep two sets
// of sums, have an SM's registers for one CTA of the larger tiles (64 experts of 5 rows, 515 x 1027: 102 us, two that
// spill 131; one of 5000 rows, 777 x 1313: 189 against 175).
template <int OP, int BM, int BN, int WM, int WN, bool CUT>
cudaError_t launch_warp_tile(const GroupedWarpArgs& a, const Shape& s, int n_sms, cudaStream_t st) {
  constexpr int kThreads = (BM / WM) * (BN / WN) * 32;
  constexpr int kCtas = (CUT && BM == 128 ? 256 : 512) / kThreads;   // of an SM
  const int64_t tiles = a.splits * tiles_of<OP>(s, BM, BN), most = (int64_t)n_sms * kCtas;
  return launch_pdl(grouped_warp_kernel<OP, BM, BN, WM, WN, kCtas, CUT>, dim3((unsigned)(tiles < most ? tiles : most)),
                    dim3(kThreads), 0, st, a);
}
template <int OP, bool CUT>
cudaError_t launch_warp_cut(const GroupedWarpArgs& a, const Shape& s, int n_sms, cudaStream_t st) {
  if (warp_tile(a.splits * tiles_of<OP>(s, 128, 128), n_sms) == 128)
    return launch_warp_tile<OP, 128, 128, 64, 32, CUT>(a, s, n_sms, st);
  return launch_warp_tile<OP, 64, 64, 32, 32, CUT>(a, s, n_sms, st);
}
template <int OP>
cudaError_t launch_warp(const GroupedWarpArgs& a, const Shape& s, int n_sms, cudaStream_t st) {
  if constexpr (OP != kGroupedWgrad)
    if ((OP == kGroupedMM ? s.k : s.n) <= kGwpOneChain * kGwpBK) return launch_warp_cut<OP, false>(a, s, n_sms, st);
  return launch_warp_cut<OP, true>(a, s, n_sms, st);
}

// Clusters of `kernel` that can be resident at once on the current device (asked for once per
// device, which also sets the kernel's shared-memory limit; `kept` is the kernel's own).
moe_status pair_clusters(const void* kernel, int threads, size_t smem, std::atomic<int>* kept, int device, int n_sms,
                         int* out) {
  if (device < 64 && (*out = kept[device].load(std::memory_order_acquire)) > 0) return MOE_OK;
  MOE_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.gridDim = dim3(2 * (n_sms / 2), 1, 1);
  lc.blockDim = dim3(threads, 1, 1);
  lc.dynamicSmemBytes = smem;
  lc.attrs = attr;
  lc.numAttrs = 1;
  int n = 0;
  MOE_CUDA(cudaOccupancyMaxActiveClusters(&n, kernel, &lc));
  if (n < 1) return fail(MOE_ERR_UNSUPPORTED, "no CTA pair of the grouped product fits on this device");
  if (device < 64) kept[device].store(n, std::memory_order_release);
  *out = n;
  return MOE_OK;
}

// The products on the tensor cores: bf16, widths in whole 16-byte vectors, aligned buffers.
template <int OP>
moe_status launch_tc(const void* a, const void* b, const int32_t* counts, const Shape& s, int accumulate,
                     int splits, void* out, int device, int n_sms, cudaStream_t st) {
  static std::atomic<int> kept[2][64];   // of each of OP's kernels
  CUtensorMap tmA, tmB;
  int clusters = 0;
  if constexpr (OP == kGroupedWgrad) {
    if (!encode_2d(&tmA, a, s.n, s.rows, kGwRows) || !encode_2d(&tmB, b, s.k, s.rows, kGwRows))
      return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed for a grouped product's operand");
    MOE_TRY(pair_clusters((const void*)grouped_wgrad_kernel, kGwThreads, kGwSmemBytes, kept[0], device, n_sms, &clusters));
    // a cluster per tile
    const int64_t tiles = splits * tiles_of<OP>(s, kPairBM, kGemmBN);
    GroupedWgradArgs p{counts, static_cast<float*>(out), s.G, (int)s.rows, s.n, s.k, accumulate, splits};
    MOE_CUDA(launch_pdl(grouped_wgrad_kernel, dim3(2 * (unsigned)tiles), dim3(kGwThreads), kGwSmemBytes, st, tmB,
                        tmA, p));
  } else {
    const bool cut = (OP == kGroupedMM ? s.k : s.n) > kGrChain * kGemmBK;
    const auto kernel = cut ? grouped_rows_kernel<OP, true> : grouped_rows_kernel<OP, false>;
    const int rt = gr_tile_rows(s.rows, s.G);
    if (!encode_2d(&tmA, a, OP == kGroupedMM ? s.k : s.n, s.rows, rt / 2) ||
        !encode_3d(&tmB, b, s.k, s.n, s.G, OP == kGroupedMM ? 128 : kGemmKPS * kGemmBK))
      return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed for a grouped product's operand");
    MOE_TRY(pair_clusters((const void*)kernel, kGpThreads, kGrSmemBytes, kept[cut], device, n_sms, &clusters));
    // at most: every expert with rows has one ragged tile row
    const int64_t tiles = ((s.rows + rt - 1) / rt + (s.G < s.rows ? s.G : s.rows)) *
                          (((OP == kGroupedMM ? s.n : s.k) + kPairBM - 1) / kPairBM);
    GroupedRowsArgs p{counts, s.G, (int)s.rows, s.n, s.k, static_cast<__nv_bfloat16*>(out), rt};
    MOE_CUDA(launch_pdl(kernel, dim3(2 * (unsigned)(tiles < clusters ? tiles : clusters)),
                        dim3(kGpThreads), kGrSmemBytes, st, tmB, tmA, p));
  }
  return MOE_OK;
}

bool takes_tma(const Shape& s, const void* a, const void* b, const void* out) {
  return s.dtype == MOE_BF16 && s.n % 8 == 0 && s.k % 8 == 0 && s.rows > 0 && aligned16(a) && aligned16(b) &&
         aligned16(out);
}

int splits_of(const Shape& s, bool tma) { return wgrad_parts(s.G, s.rows, s.n, s.k, tma); }

template <int OP>
moe_status product(const void* a, const void* b, const int32_t* counts, const Shape& s, int accumulate,
                   void* out, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  MOE_TRY(check_shape(s));
  constexpr bool W = OP == kGroupedWgrad;
  const size_t es = s.dtype == MOE_BF16 ? 2 : 4;
  const size_t a_cols = OP == kGroupedMM ? s.k : s.n;
  const size_t a_bytes = (size_t)s.rows * a_cols * es;
  const size_t b_bytes = (W ? (size_t)s.rows * s.k : (size_t)s.G * s.n * s.k) * es;
  const size_t o_bytes = W ? (size_t)s.G * s.n * s.k * 4 : (size_t)s.rows * (OP == kGroupedMM ? s.n : s.k) * es;
  if (!W && s.rows == 0) return MOE_OK;   // nothing to write
  if (!counts || !out || (s.rows > 0 && !a) || ((!W || s.rows > 0) && !b))
    return fail(MOE_ERR_INVALID_ARG, "an input/output pointer is NULL");
  if (misaligned(a, es) || misaligned(b, es) || misaligned(out, W ? 4 : es) || misaligned(counts, 4))
    return fail(MOE_ERR_INVALID_ARG, "a pointer is not aligned to its type");
  if (overlaps(out, o_bytes, a, a_bytes) || overlaps(out, o_bytes, b, b_bytes) ||
      overlaps(out, o_bytes, counts, (size_t)s.G * 4))
    return fail(MOE_ERR_INVALID_ARG, "the output overlaps an input");
  const bool tma = takes_tma(s, a, b, out);
  const int splits = W ? splits_of(s, tma) : 1;
  void* dst = out;   // of the product's kernel
  if (splits > 1) {
    const size_t need = splits * o_bytes;
    if (!workspace || !aligned16(workspace) || workspace_bytes < need)
      return fail(MOE_ERR_INVALID_ARG, "workspace must be 16-byte aligned and hold moe_grouped_wgrad_workspace bytes");
    if (overlaps(workspace, need, a, a_bytes) || overlaps(workspace, need, b, b_bytes) ||
        overlaps(workspace, need, out, o_bytes) || overlaps(workspace, need, counts, (size_t)s.G * 4))
      return fail(MOE_ERR_INVALID_ARG, "the workspace overlaps an input or the output");
    dst = workspace;
  }
  int n_sms = 0, device = 0;
  MOE_TRY(op_device(&n_sms, &device));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int add = splits > 1 ? 0 : accumulate;
  if (tma) {
    MOE_TRY(launch_tc<OP>(a, b, counts, s, add, splits, dst, device, n_sms, st));
  } else if (s.dtype == MOE_BF16) {
    GroupedWarpArgs p{static_cast<const __nv_bfloat16*>(a), static_cast<const __nv_bfloat16*>(b), counts, dst, s.G,
                      (int)s.rows, s.n, s.k, add, splits};
    MOE_CUDA(launch_warp<OP>(p, s, n_sms, st));
  } else {
    GroupedSimtArgs p{a, b, counts, dst, s.G, (int)s.rows, s.n, s.k, add, splits};
    MOE_CUDA(launch_simt<OP>(p, s, n_sms, st));
  }
  if (splits > 1) {
    const int64_t n = (int64_t)s.G * s.n * s.k;
    const bool v4 = n % 4 == 0 && aligned16(out);
    int64_t grid = (n / (v4 ? 4 : 1) + 255) / 256;
    if (grid > 8 * (int64_t)n_sms) grid = 8 * (int64_t)n_sms;
    MOE_CUDA(launch_pdl(v4 ? wgrad_sum_kernel<4> : wgrad_sum_kernel<1>, dim3((unsigned)grid), dim3(256), 0, st,
                        static_cast<const float*>(workspace), splits, n, accumulate, static_cast<float*>(out)));
  }
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_grouped_mm(const void* x, const void* w, const int32_t* counts, int32_t n_groups, int64_t rows,
                          int32_t n, int32_t k, int32_t dtype, void* y, moe_stream_t stream) {
  return product<kGroupedMM>(x, w, counts, Shape{n_groups, rows, n, k, dtype}, 0, y, nullptr, 0, stream);
}

moe_status moe_grouped_mm_dgrad(const void* dy, const void* w, const int32_t* counts, int32_t n_groups,
                                int64_t rows, int32_t n, int32_t k, int32_t dtype, void* dx,
                                moe_stream_t stream) {
  return product<kGroupedDgrad>(dy, w, counts, Shape{n_groups, rows, n, k, dtype}, 0, dx, nullptr, 0,
                                stream);
}

size_t moe_grouped_wgrad_workspace(int32_t n_groups, int64_t rows, int32_t n, int32_t k, int32_t dtype) {
  const Shape s{n_groups, rows, n, k, dtype};
  if (check_shape(s) != MOE_OK || rows == 0) return 0;
  // (whether TMA takes the buffers is not known here: the larger of the two)
  const int a = splits_of(s, true), b = splits_of(s, false);
  const int splits = dtype == MOE_FP32 || n % 8 || k % 8 ? b : a > b ? a : b;
  return splits > 1 ? (size_t)splits * n_groups * n * k * sizeof(float) : 0;
}

moe_status moe_grouped_mm_wgrad(const void* dy, const void* x, const int32_t* counts, int32_t n_groups,
                                int64_t rows, int32_t n, int32_t k, int32_t dtype, int32_t accumulate,
                                float* dw, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  return product<kGroupedWgrad>(dy, x, counts, Shape{n_groups, rows, n, k, dtype}, accumulate, dw, workspace,
                                workspace_bytes, stream);
}

moe_status moe_grouped_device_status(moe_stream_t stream) {
  int n_sms = 0;
  MOE_TRY(op_device(&n_sms));
  MOE_CUDA(cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)));
  int code = 0;
  MOE_CUDA(cudaMemcpyFromSymbol(&code, g_grouped_err, sizeof(int)));
  if (code == 0) return MOE_OK;
  const int none = 0;
  MOE_CUDA(cudaMemcpyToSymbol(g_grouped_err, &none, sizeof(int)));
  return fail(MOE_ERR_DEVICE_CHECK, "a grouped product recorded device error 0x%x", code);
}

}  // extern "C"
