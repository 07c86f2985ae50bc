// moe_block_norm.cu -- moe_block_norm and moe_block_norm_backward (include/moe.h): checks,
// the choice of the row kernel's width, and the launches.
#include "op_common.cuh"
#include "block_norm.cuh"

using namespace moe;

namespace {

// the widest ring: a backward CTA of 512 threads with two accesses each
constexpr size_t kNormMaxSmem = norm_ring_bytes(4, 2, 512);

template <int N>
using Int = std::integral_constant<int, N>;

// How rows are read: 16 bytes at a time, d being a whole number of them and every row and parameter
// pointer aligned; by the aligned 16 bytes that a row touches, when the row pointers are; or one
// element at a time.
enum class RowRead { kWhole, kShifted, kSingle };

// Call f(V, NV, MAXT, SHIFT, threads, rows per CTA) for rows of d elements of T.  A warp per row up
// to 64 accesses (a CTA of one warp would leave the SM half empty, a wider one waits at
// barriers); above, per access half a thread (forward) or one (backward, whose column sums take
// registers; half a thread again past 512).  bf16 rows just past a size at which one CTA fewer
// fits an SM are run by CTAs held to the registers of one more: backward of 2056 columns 485 us
// -> 366 (2816: 331 against 411, so up to 320 accesses), of 5000 518 -> 402 (6000: 447 against
// 454, so up to 640), forward of 5000 232 -> 190 (not of 4501 by single accesses at its ends:
// 331 against 354), all of 1.2e8 elements.
template <typename T, bool BWD, class F>
cudaError_t with_row_shape(int d, RowRead read, F&& f) {
  auto threads = [](int n) { return (n + 31) / 32 * 32; };
  constexpr int V = 16 / sizeof(T);
  constexpr int NV = BWD ? 1 : 2;
  auto ringed = [&](auto shift, int n) {   // n <= 1024
    if (n <= 32) return f(Int<V>{}, Int<1>{}, Int<32>{}, shift, 32 * kNormWarps, kNormWarps);
    if (n <= 64) return f(Int<V>{}, Int<2>{}, Int<32>{}, shift, 32 * kNormWarps, kNormWarps);
    if (n <= NV * 256) return f(Int<V>{}, Int<NV>{}, Int<256>{}, shift, threads((n + NV - 1) / NV), 1);
    if constexpr (BWD && V == 8)
      if (n <= 320) return f(Int<V>{}, Int<2>{}, Int<160>{}, shift, threads((n + 1) / 2), 1);
    if constexpr (BWD)
      if (n <= 512) return f(Int<V>{}, Int<1>{}, Int<512>{}, shift, threads(n), 1);
    if constexpr (BWD && V == 8)
      if (n <= 640) return f(Int<V>{}, Int<2>{}, Int<320>{}, shift, threads((n + 1) / 2), 1);
    if constexpr (!BWD && V == 8 && !shift())
      if (n <= 768) return f(Int<V>{}, Int<2>{}, Int<384>{}, shift, threads((n + 1) / 2), 1);
    return f(Int<V>{}, Int<2>{}, Int<512>{}, shift, threads((n + 1) / 2), 1);
  };
  if (read == RowRead::kWhole) {
    const int n = d / V;
    if (n <= 1024) return ringed(std::false_type{}, n);
    if constexpr (V < 8)   // (kNormMaxD is 2048 accesses of 8)
      if (n > 2048) return f(Int<V>{}, Int<4>{}, Int<1024>{}, std::false_type{}, threads((n + 3) / 4), 1);
    return f(Int<V>{}, Int<2>{}, Int<1024>{}, std::false_type{}, threads((n + 1) / 2), 1);
  }
  // (narrow bf16 rows would be all ends: forward of 129 columns 511 us, 378 by single elements; of 257
  // 396, 637 by single elements; 1.2e8 elements)
  if (read == RowRead::kShifted && (V < 8 || d > 256)) {
    const int n = (d + 2 * V - 2) / V;   // at most: V - 1 elements before the row
    if (n <= 1024) return ringed(std::true_type{}, n);
  }
  constexpr std::false_type no{};
  if (d <= 256) return f(Int<1>{}, Int<8>{}, Int<32>{}, no, 32 * kNormWarps, kNormWarps);
  if (d <= 2048) return f(Int<1>{}, Int<8>{}, Int<256>{}, no, threads((d + 7) / 8), 1);
  if (d <= 4096) return f(Int<1>{}, Int<8>{}, Int<512>{}, no, threads((d + 7) / 8), 1);
  if (d <= 8192) return f(Int<1>{}, Int<8>{}, Int<1024>{}, no, threads((d + 7) / 8), 1);
  return f(Int<1>{}, Int<16>{}, Int<1024>{}, no, threads((d + 15) / 16), 1);
}

// CTAs of a persistent kernel: as many as are resident at once (asked for once per device and
// CTA size, which also raises the kernel's shared-memory limit), at most one per row (or eight); a
// multiple of `period` when a CTA takes several rows.
struct NormOccupancy {
  std::atomic<int> per_sm[64][33];
};
cudaError_t norm_grid(const void* kernel, NormOccupancy& kept, int device, int threads, size_t smem,
                      int rows_per_cta, int period, int64_t T, int n_sms, int* grid) {
  std::atomic<int>* known = device < 64 ? &kept.per_sm[device][threads / 32] : nullptr;
  int per_sm = known ? known->load(std::memory_order_acquire) : 0;
  if (per_sm == 0) {
    // the widest CTA's need: the limit is the kernel's, whatever this call's size
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kNormMaxSmem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) per_sm = 1;
    if (known) known->store(per_sm, std::memory_order_release);
  }
  int64_t g = (T + rows_per_cta - 1) / rows_per_cta;
  if (g > (int64_t)n_sms * per_sm) g = (int64_t)n_sms * per_sm / period * period;
  *grid = (int)g;
  return cudaSuccess;
}

int norm_max_parts(int64_t T) { return T < kNormMaxParts ? (int)T : kNormMaxParts; }

moe_status check_shape(int64_t T, int32_t d, int32_t dtype, int32_t gate_kind, const float* gate,
                       const void* y, const float* w_post, const float* w_pre, float beta) {
  if (dtype != MOE_BF16 && dtype != MOE_FP32)
    return fail(MOE_ERR_INVALID_ARG, "dtype=%d is not MOE_FP32 or MOE_BF16", dtype);
  if (T < 0 || T > (int64_t(1) << 31) - 1) return fail(MOE_ERR_INVALID_ARG, "T=%lld outside [0, 2^31)", (long long)T);
  if (d < 1) return fail(MOE_ERR_INVALID_ARG, "d must be positive");
  if (d > kNormMaxD) return fail(MOE_ERR_UNSUPPORTED, "d=%d above %d", d, kNormMaxD);
  if (gate_kind < kGateNone || gate_kind > kGateToken)
    return fail(MOE_ERR_INVALID_ARG, "gate_kind=%d is not MOE_GATE_NONE, _CHANNEL or _TOKEN", gate_kind);
  if (!(beta - beta == 0.0f)) return fail(MOE_ERR_INVALID_ARG, "beta is not finite");
  if (T == 0) return MOE_OK;   // (empty buffers may be NULL)
  if ((gate_kind != kGateNone) != (gate != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "gate is given exactly when gate_kind is not MOE_GATE_NONE");
  if (!y && (gate || w_post || beta != 1.0f))
    return fail(MOE_ERR_INVALID_ARG, "without y there is no gate, no post_weight, and beta is 1");
  if (!y && !w_pre) return fail(MOE_ERR_INVALID_ARG, "neither y nor pre_weight is given");
  return MOE_OK;
}

// rows: [T, d] buffers of the row kernel; params: [d] fp32
RowRead row_read(int32_t d, int es, std::initializer_list<const void*> rows,
                 std::initializer_list<const void*> params) {
  for (const void* p : rows)
    if (!aligned16(p)) return RowRead::kSingle;
  for (const void* p : params)
    if (!aligned16(p)) return RowRead::kShifted;
  return d % (16 / es) ? RowRead::kShifted : RowRead::kWhole;
}

// Rows after which a row starts at the same offset from 16 bytes again, when one CTA's have to.
constexpr int row_period(bool shift, int v) { return shift ? v : 1; }

template <typename T>
cudaError_t launch_fwd(const BlockNormArgs& a, RowRead read, int device, int n_sms, cudaStream_t st) {
  return with_row_shape<T, false>(a.d, read, [&](auto v, auto nv, auto maxt, auto shift, int threads, int rows) {
    static NormOccupancy kept;
    auto kernel = block_norm_kernel<T, v(), nv(), maxt(), shift()>;
    const size_t smem = norm_rings(v(), maxt()) ? norm_ring_bytes(2, nv(), threads) : 0;
    int grid = 0;
    const cudaError_t e = norm_grid((const void*)kernel, kept, device, threads, smem, rows,
                                    row_period(shift(), v()), a.T, n_sms, &grid);
    return e != cudaSuccess ? e : launch_pdl(kernel, dim3(grid), dim3(threads), smem, st, a);
  });
}

// *parts: the CTAs, each with its own partial sums.
template <typename T>
cudaError_t launch_bwd(const BlockNormBwdArgs& a, RowRead read, int device, int n_sms, int* parts, cudaStream_t st) {
  return with_row_shape<T, true>(a.d, read, [&](auto v, auto nv, auto maxt, auto shift, int threads, int rows) {
    static NormOccupancy kept;
    auto kernel = block_norm_bwd_kernel<T, v(), nv(), maxt(), shift()>;
    const size_t smem = norm_rings(v(), maxt()) ? norm_ring_bytes(4, nv(), threads) : 0;
    const cudaError_t e = norm_grid((const void*)kernel, kept, device, threads, smem, rows,
                                    row_period(shift(), v()), a.T, n_sms, parts);
    if (e != cudaSuccess) return e;
    if (*parts > kNormMaxParts) *parts = kNormMaxParts;   // (a multiple of every period)
    return launch_pdl(kernel, dim3(*parts), dim3(threads), smem, st, a);
  });
}

}  // namespace

extern "C" {

moe_status moe_block_norm(const void* x, const void* y, const float* gate, int32_t gate_kind,
                          const float* post_weight, const float* pre_weight, int64_t T, int32_t d,
                          int32_t dtype, float beta, float eps, void* r, void* u, float* post_rstd,
                          float* pre_rstd, moe_stream_t stream) {
  MOE_TRY(check_shape(T, d, dtype, gate_kind, gate, y, post_weight, pre_weight, beta));
  if (!(eps > 0.0f) || !(eps - eps == 0.0f)) return fail(MOE_ERR_INVALID_ARG, "eps must be positive and finite");
  if (T == 0) return MOE_OK;
  if (!x || (y != nullptr) != (r != nullptr) || (pre_weight != nullptr) != (u != nullptr) ||
      (post_weight != nullptr) != (post_rstd != nullptr) || (pre_weight != nullptr) != (pre_rstd != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "x is required; r goes with y, u and pre_rstd with pre_weight, "
                                     "post_rstd with post_weight");
  const int es = dtype == MOE_BF16 ? 2 : 4;
  for (const void* p : {x, y, (const void*)r, (const void*)u})
    if (misaligned(p, es)) return fail(MOE_ERR_INVALID_ARG, "a row pointer is not aligned to its type");
  const size_t bytes = (size_t)T * d * es;
  // r and u are written while other rows are read: only a buffer's own rows may be written
  if (overlaps(r, bytes, u, bytes)) return fail(MOE_ERR_INVALID_ARG, "r and u overlap");
  for (const void* o : {(const void*)r, (const void*)u})
    for (const void* i : {x, y})
      if (o != i && overlaps(o, bytes, i, bytes))
        return fail(MOE_ERR_INVALID_ARG, "an output overlaps an input without being the same buffer");
  const size_t tok = (size_t)T * 4, ch = (size_t)d * 4;
  if (!apart({{post_rstd, tok}, {pre_rstd, tok}},
             {{x, bytes}, {y, bytes}, {r, bytes}, {u, bytes}, {post_weight, ch}, {pre_weight, ch},
              {gate, gate_kind == kGateToken ? tok : ch}}))
    return fail(MOE_ERR_INVALID_ARG, "a statistic overlaps another buffer");
  if (!apart({{r, bytes}, {u, bytes}},
             {{post_weight, ch}, {pre_weight, ch}, {gate, gate_kind == kGateToken ? tok : ch}}))
    return fail(MOE_ERR_INVALID_ARG, "r or u overlaps a parameter");
  int n_sms = 0, device = 0;
  MOE_TRY(op_device(&n_sms, &device));
  BlockNormArgs a{x, y, gate, post_weight, pre_weight, r, u, post_rstd, pre_rstd, T, d, gate_kind, beta, eps};
  const RowRead read = row_read(d, es, {x, y, r, u},
                                {post_weight, pre_weight, gate_kind == kGateChannel ? gate : nullptr});
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  MOE_CUDA((dtype == MOE_BF16 ? launch_fwd<__nv_bfloat16>(a, read, device, n_sms, st)
                              : launch_fwd<float>(a, read, device, n_sms, st)));
  return MOE_OK;
}

size_t moe_block_norm_workspace(int64_t T, int32_t d) {
  if (T < 1 || d < 1 || d > kNormMaxD) return 0;
  return (size_t)norm_max_parts(T) * d * 2 * sizeof(float);
}

moe_status moe_block_norm_backward(const void* y, const void* r, const void* dr, const void* du,
                                   const float* gate, int32_t gate_kind, const float* post_weight,
                                   const float* pre_weight, const float* post_rstd, const float* pre_rstd,
                                   int64_t T, int32_t d, int32_t dtype, float beta, void* dx, void* dy,
                                   float* d_gate, float* d_post_weight, float* d_pre_weight,
                                   void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  MOE_TRY(check_shape(T, d, dtype, gate_kind, gate, y, post_weight, pre_weight, beta));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool channel = gate_kind == kGateChannel;
  if (T == 0) {   // no rows: zero parameter gradients
    for (float* p : {d_pre_weight, d_post_weight, channel ? d_gate : nullptr})
      if (p) MOE_CUDA(cudaMemsetAsync(p, 0, (size_t)d * 4, st));
    return MOE_OK;
  }
  if ((gate != nullptr) != (d_gate != nullptr) || (post_weight != nullptr) != (d_post_weight != nullptr) ||
      (pre_weight != nullptr) != (d_pre_weight != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "each of d_gate, d_post_weight, d_pre_weight goes with its parameter");
  if ((pre_weight != nullptr) != (du != nullptr) || (!pre_weight && !dr) || (pre_weight && !r) ||
      (post_weight != nullptr) != (post_rstd != nullptr) || (pre_weight != nullptr) != (pre_rstd != nullptr) ||
      !dx || (y != nullptr) != (dy != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "du, r and pre_rstd go with pre_weight (dr without it), post_rstd "
                                     "with post_weight, dy with y; dx is required");
  const int es = dtype == MOE_BF16 ? 2 : 4;
  for (const void* p : {y, r, dr, du, (const void*)dx, (const void*)dy})
    if (misaligned(p, es)) return fail(MOE_ERR_INVALID_ARG, "a row pointer is not aligned to its type");
  const size_t bytes = (size_t)T * d * es;
  if (overlaps(dx, bytes, dy, bytes)) return fail(MOE_ERR_INVALID_ARG, "dx and dy overlap");
  for (const void* o : {(const void*)dx, (const void*)dy})
    for (const void* i : {y, r, dr, du})
      if (o != i && overlaps(o, bytes, i, bytes))
        return fail(MOE_ERR_INVALID_ARG, "an output overlaps an input without being the same buffer");
  if (!workspace || !aligned16(workspace) || workspace_bytes < moe_block_norm_workspace(T, d))
    return fail(MOE_ERR_INVALID_ARG, "workspace must be 16-byte aligned and hold moe_block_norm_workspace bytes");
  const size_t tok = (size_t)T * 4, ch = (size_t)d * 4, gb = gate_kind == kGateToken ? tok : ch;
  if (!apart({{d_gate, gb}, {d_post_weight, ch}, {d_pre_weight, ch}, {workspace, moe_block_norm_workspace(T, d)}},
             {{y, bytes}, {r, bytes}, {dr, bytes}, {du, bytes}, {dx, bytes}, {dy, bytes}, {post_rstd, tok},
              {pre_rstd, tok}, {gate, gb}, {post_weight, ch}, {pre_weight, ch}}))
    return fail(MOE_ERR_INVALID_ARG, "a parameter's gradient or the workspace overlaps another buffer");
  if (!apart({{dx, bytes}, {dy, bytes}},
             {{post_rstd, tok}, {pre_rstd, tok}, {gate, gb}, {post_weight, ch}, {pre_weight, ch}}))
    return fail(MOE_ERR_INVALID_ARG, "dx or dy overlaps a parameter or a statistic");
  int n_sms = 0, device = 0;
  MOE_TRY(op_device(&n_sms, &device));
  const bool need_s = post_weight || channel;
  int parts = 0;
  float* part = static_cast<float*>(workspace);
  float* part_pre = pre_weight ? part : nullptr;
  float* part_s = need_s ? part + (size_t)norm_max_parts(T) * d : nullptr;
  BlockNormBwdArgs a{y, r, dr, du, gate, post_weight, pre_weight, post_rstd, pre_rstd, dx, dy,
                     gate_kind == kGateToken ? d_gate : nullptr, part_pre, part_s, T, d, gate_kind, beta};
  const RowRead read = row_read(d, es, {y, r, dr, du, dx, dy},
                                {post_weight, pre_weight, channel ? gate : nullptr});
  MOE_CUDA((dtype == MOE_BF16 ? launch_bwd<__nv_bfloat16>(a, read, device, n_sms, &parts, st)
                              : launch_bwd<float>(a, read, device, n_sms, &parts, st)));
  if (part_pre || part_s) {
    NormReduceArgs ra{part_pre, part_s, parts, d, post_weight, channel ? gate : nullptr, d_pre_weight,
                      d_post_weight, channel ? d_gate : nullptr};
    MOE_CUDA(launch_pdl(block_norm_reduce_kernel, dim3((d + 31) / 32, 2), dim3(32 * kNormRedRows), 0, st, ra));
  }
  return MOE_OK;
}

}  // extern "C"
