// moe_block_norm.cu -- moe_block_norm and moe_block_norm_backward (include/moe.h): checks,
// the choice of the row kernel's width, and the launches.
#include "op_common.cuh"
#include "block_norm.cuh"

using namespace moe;

namespace {

// Call f(V, NV, TPR) for rows of d elements of T: 16-byte accesses when d is a multiple of
// their elements and every row pointer is 16-byte aligned, else one element an access; the
// fewest threads (64 to 1024) that hold a row in two 16-byte accesses each (eight single
// elements), more accesses a thread only for rows past 1024 threads' worth.
template <typename T, class F>
cudaError_t with_row_shape(int d, bool vec, F&& f) {
  auto c = [](auto v) { return v; };
  (void)c;
  if (vec) {
    constexpr int V = 16 / sizeof(T);
    std::integral_constant<int, V> v;
    const int n = d / V;
    std::integral_constant<int, 1> one;
    std::integral_constant<int, 2> two;
    std::integral_constant<int, 4> four;
    if (n <= 64) return f(v, one, std::integral_constant<int, 64>{});
    if (n <= 128) return f(v, one, std::integral_constant<int, 128>{});
    if (n <= 256) return f(v, two, std::integral_constant<int, 128>{});
    if (n <= 512) return f(v, two, std::integral_constant<int, 256>{});
    if (n <= 1024) return f(v, two, std::integral_constant<int, 512>{});
    if (n <= 2048) return f(v, two, std::integral_constant<int, 1024>{});
    return f(v, four, std::integral_constant<int, 1024>{});
  }
  std::integral_constant<int, 1> v;
  std::integral_constant<int, 8> eight;
  std::integral_constant<int, 16> sixteen;
  if (d <= 512) return f(v, eight, std::integral_constant<int, 64>{});
  if (d <= 1024) return f(v, eight, std::integral_constant<int, 128>{});
  if (d <= 4096) return f(v, eight, std::integral_constant<int, 512>{});
  if (d <= 8192) return f(v, eight, std::integral_constant<int, 1024>{});
  return f(v, sixteen, std::integral_constant<int, 1024>{});
}

int norm_parts(int64_t T) { return T < kNormMaxParts ? (int)T : kNormMaxParts; }

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
bool rows_vec(int32_t d, int es, std::initializer_list<const void*> rows,
              std::initializer_list<const void*> params) {
  if (d % (16 / es)) return false;
  for (const void* p : rows)
    if (!aligned16(p)) return false;
  for (const void* p : params)
    if (!aligned16(p)) return false;
  return true;
}

template <typename T>
cudaError_t launch_fwd(const BlockNormArgs& a, bool vec, cudaStream_t st) {
  return with_row_shape<T>(a.d, vec, [&](auto v, auto nv, auto tpr) {
    return launch_pdl(block_norm_kernel<T, v(), nv(), tpr()>, dim3((unsigned)a.T), dim3(tpr()), 0, st, a);
  });
}

template <typename T>
cudaError_t launch_bwd(const BlockNormBwdArgs& a, int parts, bool vec, cudaStream_t st) {
  return with_row_shape<T>(a.d, vec, [&](auto v, auto nv, auto tpr) {
    return launch_pdl(block_norm_bwd_kernel<T, v(), nv(), tpr()>, dim3(parts), dim3(tpr()), 0, st, a);
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
  int n_sms = 0;
  MOE_TRY(op_device(&n_sms));
  BlockNormArgs a{x, y, gate, post_weight, pre_weight, r, u, post_rstd, pre_rstd, T, d, gate_kind, beta, eps};
  const bool vec = rows_vec(d, es, {x, y, r, u},
                            {post_weight, pre_weight, gate_kind == kGateChannel ? gate : nullptr});
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  MOE_CUDA(dtype == MOE_BF16 ? launch_fwd<__nv_bfloat16>(a, vec, st) : launch_fwd<float>(a, vec, st));
  return MOE_OK;
}

size_t moe_block_norm_workspace(int64_t T, int32_t d) {
  if (T < 1 || d < 1 || d > kNormMaxD) return 0;
  return (size_t)norm_parts(T) * d * 2 * sizeof(float);
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
  int n_sms = 0;
  MOE_TRY(op_device(&n_sms));
  const bool need_s = post_weight || channel;
  const int parts = norm_parts(T);
  float* part = static_cast<float*>(workspace);
  float* part_pre = pre_weight ? part : nullptr;
  float* part_s = need_s ? part + (size_t)parts * d : nullptr;
  BlockNormBwdArgs a{y, r, dr, du, gate, post_weight, pre_weight, post_rstd, pre_rstd, dx, dy,
                     gate_kind == kGateToken ? d_gate : nullptr, part_pre, part_s, T, d, gate_kind, beta};
  const bool vec = rows_vec(d, es, {y, r, dr, du, dx, dy},
                            {post_weight, pre_weight, channel ? gate : nullptr});
  MOE_CUDA((dtype == MOE_BF16 ? launch_bwd<__nv_bfloat16>(a, parts, vec, st)
                              : launch_bwd<float>(a, parts, vec, st)));
  if (part_pre || part_s) {
    NormReduceArgs ra{part_pre, part_s, parts, d, post_weight, channel ? gate : nullptr, d_pre_weight,
                      d_post_weight, channel ? d_gate : nullptr};
    MOE_CUDA(launch_pdl(block_norm_reduce_kernel, dim3((d + 31) / 32, 2), dim3(32 * kNormRedRows), 0, st, ra));
  }
  return MOE_OK;
}

}  // extern "C"
