// moe_grad_clip.cu -- moe_grad_sumsq, moe_grad_scale and moe_clip_grad_norm (include/moe.h).
#include <algorithm>
#include <new>

#include "op_common.cuh"
#include "grad_clip.cuh"

using namespace moe;

namespace {

// Every output is written by its own chunks while other chunks are read and written: no two
// outputs may share a byte, nor an output and another tensor's gradients (the same buffer
// listed twice would be scaled twice, in no order).
moe_status check_disjoint(const void* const* grads, void* const* outs, const int64_t* numels,
                          const int32_t* dtypes, int n) {
  struct Range {
    uintptr_t lo, hi;
    int tensor;
    bool out;
  };
  std::vector<Range> spans;
  try {
    spans.reserve(2 * (size_t)n);
  } catch (const std::bad_alloc&) {
    return fail(MOE_ERR_OOM, "host allocation failed");
  }
  for (int i = 0; i < n; ++i) {
    if (numels[i] == 0) continue;
    const size_t bytes = (size_t)numels[i] * (dtypes[i] == MOE_BF16 ? 2 : 4);
    const uintptr_t o = reinterpret_cast<uintptr_t>(outs[i]), g = reinterpret_cast<uintptr_t>(grads[i]);
    spans.push_back(Range{o, o + bytes, i, true});
    if (g != o) spans.push_back(Range{g, g + bytes, i, false});
  }
  auto before = [](const Range& a, const Range& b) { return a.lo < b.lo; };
  if (!std::is_sorted(spans.begin(), spans.end(), before)) std::sort(spans.begin(), spans.end(), before);
  // in order of their starts: the furthest end so far of the outputs and of all spans
  uintptr_t out_end = 0, end = 0;
  for (const Range& s : spans) {
    if (s.lo < out_end || (s.out && s.lo < end))
      return fail(MOE_ERR_INVALID_ARG, "tensor %d shares memory with another tensor's output", s.tensor);
    if (s.out) out_end = std::max(out_end, s.hi);
    end = std::max(end, s.hi);
  }
  return MOE_OK;
}

// `own`: what the call reads and writes besides the tensors, apart from them and from each other.
moe_status check_tensors(const void* const* grads, void* const* outs, const int64_t* numels,
                         const int32_t* dtypes, int32_t n, std::initializer_list<Span> own) {
  if (n < 0) return fail(MOE_ERR_INVALID_ARG, "n_tensors must not be negative");
  if (n > 0 && (!grads || !numels || !dtypes)) return fail(MOE_ERR_INVALID_ARG, "a table pointer is NULL");
  if (!apart(own, {})) return fail(MOE_ERR_INVALID_ARG, "sumsq, norm and workspace overlap");
  int64_t chunks = 0;
  for (int i = 0; i < n; ++i) {
    if (dtypes[i] != MOE_BF16 && dtypes[i] != MOE_FP32)
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: dtype=%d is not MOE_FP32 or MOE_BF16", i, dtypes[i]);
    if (numels[i] < 0 || numels[i] >= (int64_t(1) << 40))
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: %lld elements", i, (long long)numels[i]);
    if (numels[i] == 0) continue;
    const size_t es = dtypes[i] == MOE_BF16 ? 2 : 4, bytes = (size_t)numels[i] * es;
    if (!grads[i] || (outs && !outs[i])) return fail(MOE_ERR_INVALID_ARG, "tensor %d: NULL pointer", i);
    if (misaligned(grads[i], es) || (outs && misaligned(outs[i], es)))
      return fail(MOE_ERR_INVALID_ARG, "tensor %d is not aligned to its type", i);
    if (outs && outs[i] != grads[i] && overlaps(outs[i], bytes, grads[i], bytes))
      return fail(MOE_ERR_INVALID_ARG, "tensor %d overlaps its output without being the same buffer", i);
    for (const Span& o : own)
      if (overlaps(o.p, o.n, grads[i], bytes) || (outs && overlaps(o.p, o.n, outs[i], bytes)))
        return fail(MOE_ERR_INVALID_ARG, "tensor %d overlaps sumsq, norm or the workspace", i);
    chunks += (numels[i] + kClipChunk - 1) / kClipChunk;
  }
  if (chunks >= (int64_t(1) << 31)) return fail(MOE_ERR_UNSUPPORTED, "too many elements in one call");
  return outs ? check_disjoint(grads, outs, numels, dtypes, n) : MOE_OK;
}

// Tensors [i, j) fill one launch's table: non-empty ones, at most N.
template <int N>
int fill_table(ClipTable<N>& t, const void* const* grads, void* const* outs, const int64_t* numels,
               const int32_t* dtypes, int n, int i) {
  t.n_tensors = 0;
  t.chunk0[0] = 0;
  for (uint32_t& w : t.bf16) w = 0;
  for (; i < n && t.n_tensors < N; ++i) {
    if (numels[i] == 0) continue;
    const int k = t.n_tensors++;
    t.e[k] = ClipEntry{grads[i], outs ? outs[i] : nullptr, numels[i]};
    t.chunk0[k + 1] = t.chunk0[k] + (int32_t)((numels[i] + kClipChunk - 1) / kClipChunk);
    if (dtypes[i] == MOE_BF16) t.bf16[k >> 5] |= 1u << (k & 31);
  }
  return i;
}

int non_empty(const int64_t* numels, int n) {
  int c = 0;
  for (int i = 0; i < n; ++i) c += numels[i] != 0;
  return c;
}

int clip_grid(int chunks, int n_sms) {
  const int g = 4 * n_sms < kClipMaxCtas ? 4 * n_sms : kClipMaxCtas;
  return chunks < g ? chunks : g;
}

// Partial sums of every launch, one after the other, into `partial`; *n_sums their number.
template <int N>
moe_status sumsq_launches(const void* const* grads, const int64_t* numels, const int32_t* dtypes, int n,
                          double* partial, int* n_sums, int n_sms, cudaStream_t st) {
  ClipTable<N> t;
  *n_sums = 0;
  for (int i = 0; i < n;) {
    i = fill_table(t, grads, nullptr, numels, dtypes, n, i);
    if (t.n_tensors == 0) break;
    const int grid = clip_grid(t.chunk0[t.n_tensors], n_sms);
    MOE_CUDA(launch_pdl(grad_sumsq_kernel<N>, dim3(grid), dim3(kClipThreads), 0, st, t, partial + *n_sums));
    *n_sums += grid;
  }
  return MOE_OK;
}

template <int N>
moe_status scale_launches(const void* const* grads, void* const* outs, const int64_t* numels,
                          const int32_t* dtypes, int n, ClipScaleArgs a, int n_sms, cudaStream_t st) {
  ClipTable<N> t;
  for (int i = 0; i < n;) {
    i = fill_table(t, grads, outs, numels, dtypes, n, i);
    if (t.n_tensors == 0) break;
    const int grid = clip_grid(t.chunk0[t.n_tensors], n_sms);
    MOE_CUDA(launch_pdl(grad_scale_kernel<N>, dim3(grid), dim3(kClipThreads), 0, st, t, a));
    a.norm = nullptr;   // written once
  }
  return MOE_OK;
}

moe_status check_workspace(const void* ws, size_t bytes, int32_t n) {
  if (!ws || misaligned(ws, 8) || bytes < moe_grad_workspace(n))
    return fail(MOE_ERR_INVALID_ARG, "workspace must be 8-byte aligned and hold moe_grad_workspace bytes");
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_grad_workspace(int32_t n_tensors) {
  const size_t launches = n_tensors < 1 ? 1 : ((size_t)n_tensors + kClipTable - 1) / kClipTable;
  return launches * kClipMaxCtas * sizeof(double);
}

moe_status moe_grad_sumsq(const void* const* grads, const int64_t* numels, const int32_t* dtypes,
                          int32_t n_tensors, double* sumsq, float* norm, void* workspace,
                          size_t workspace_bytes, moe_stream_t stream) {
  MOE_TRY(check_tensors(grads, nullptr, numels, dtypes, n_tensors,
                        {{sumsq, 8}, {norm, 4}, {workspace, moe_grad_workspace(n_tensors)}}));
  if (!sumsq && !norm) return fail(MOE_ERR_INVALID_ARG, "neither sumsq nor norm is given");
  MOE_TRY(check_workspace(workspace, workspace_bytes, n_tensors));
  int n_sms = 0, sums = 0;
  MOE_TRY(op_device(&n_sms));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(workspace);
  if (non_empty(numels, n_tensors) <= kClipTableSmall)
    MOE_TRY(sumsq_launches<kClipTableSmall>(grads, numels, dtypes, n_tensors, partial, &sums, n_sms, st));
  else
    MOE_TRY(sumsq_launches<kClipTable>(grads, numels, dtypes, n_tensors, partial, &sums, n_sms, st));
  MOE_CUDA(launch_pdl(grad_sumsq_total_kernel, dim3(1), dim3(kClipThreads), 0, st, (const double*)partial, sums,
                      sumsq, norm));
  return MOE_OK;
}

moe_status moe_grad_scale(const void* const* grads, void* const* outs, const int64_t* numels,
                          const int32_t* dtypes, int32_t n_tensors, const double* sumsq, double max_norm,
                          float* norm, moe_stream_t stream) {
  if (n_tensors > 0 && !outs) return fail(MOE_ERR_INVALID_ARG, "a table pointer is NULL");
  MOE_TRY(check_tensors(grads, outs, numels, dtypes, n_tensors, {{sumsq, 8}, {norm, 4}}));
  if (!sumsq) return fail(MOE_ERR_INVALID_ARG, "sumsq is NULL");
  if (!(max_norm >= 0.0)) return fail(MOE_ERR_INVALID_ARG, "max_norm must not be negative or NaN");
  int n_sms = 0;
  MOE_TRY(op_device(&n_sms));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  ClipScaleArgs a{sumsq, 1, max_norm, norm};
  const int k = non_empty(numels, n_tensors);
  if (k == 0) {
    if (norm) MOE_CUDA(launch_pdl(grad_sumsq_total_kernel, dim3(1), dim3(kClipThreads), 0, st, sumsq, 1,
                                  (double*)nullptr, norm));
    return MOE_OK;
  }
  if (k <= kClipTableSmall)
    return scale_launches<kClipTableSmall>(grads, outs, numels, dtypes, n_tensors, a, n_sms, st);
  return scale_launches<kClipTable>(grads, outs, numels, dtypes, n_tensors, a, n_sms, st);
}

moe_status moe_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* numels,
                              const int32_t* dtypes, int32_t n_tensors, double max_norm, float* norm,
                              void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  if (n_tensors > 0 && !outs) return fail(MOE_ERR_INVALID_ARG, "a table pointer is NULL");
  MOE_TRY(check_tensors(grads, outs, numels, dtypes, n_tensors,
                        {{norm, 4}, {workspace, moe_grad_workspace(n_tensors)}}));
  if (!norm) return fail(MOE_ERR_INVALID_ARG, "norm is NULL");
  if (!(max_norm >= 0.0)) return fail(MOE_ERR_INVALID_ARG, "max_norm must not be negative or NaN");
  MOE_TRY(check_workspace(workspace, workspace_bytes, n_tensors));
  int n_sms = 0, sums = 0;
  MOE_TRY(op_device(&n_sms));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(workspace);
  const int k = non_empty(numels, n_tensors);
  if (k == 0) {   // nothing to scale: the norm of nothing is 0
    MOE_CUDA(cudaMemsetAsync(norm, 0, sizeof(float), st));
    return MOE_OK;
  }
  if (k <= kClipTableSmall) {
    MOE_TRY(sumsq_launches<kClipTableSmall>(grads, numels, dtypes, n_tensors, partial, &sums, n_sms, st));
    return scale_launches<kClipTableSmall>(grads, outs, numels, dtypes, n_tensors,
                                           ClipScaleArgs{partial, sums, max_norm, norm}, n_sms, st);
  }
  MOE_TRY(sumsq_launches<kClipTable>(grads, numels, dtypes, n_tensors, partial, &sums, n_sms, st));
  return scale_launches<kClipTable>(grads, outs, numels, dtypes, n_tensors,
                                    ClipScaleArgs{partial, sums, max_norm, norm}, n_sms, st);
}

}  // extern "C"
