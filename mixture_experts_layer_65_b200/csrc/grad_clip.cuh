// grad_clip.cuh -- the global 2-norm of many gradient tensors, and their scaling to at most
// a given norm:
//   N = sqrt(sum over all tensors and elements of g^2),   g *= min(1, max_norm / N)
//
// The tensors come as a table in the kernel's parameters (no copy of pointers to the device,
// so a call can be captured into a graph); each is cut into chunks, and the CTAs take chunks
// round-robin, so a few huge tensors and thousands of tiny ones both fill the SMs.  Squares
// and sums are 64-bit: a sum over 10^9 elements loses nothing, and gradients of 1e-30 or 1e30,
// whose squares leave the fp32 range, count.  The order of the sums is fixed by the sizes, the
// buffers' offsets from 16 bytes and the SM count.
//
// Bound by HBM: the norm reads each gradient once (881 MB of fp32: 127 us, 6.9 TB/s), clipping reads
// it again and writes it (2.28 GB: 1.08 to 1.10 ms, 6.3 TB/s over the three passes); the second pass runs
// backwards through the tensors, whose ends are still in L2.  Small sets are bound by launches
// (600 tensors of 0.9 million elements: 11.5 us on the device).
#pragma once

#include "ptx.cuh"

namespace moe {

constexpr int kClipThreads = 512;
constexpr int kClipChunk = 32768;       // elements
constexpr int kClipMaxCtas = 592;       // partial sums per launch
constexpr int kClipTableSmall = 48;     // tensors per launch: two table sizes, since the
constexpr int kClipTable = 1100;        // parameters (up to 32 KB) are copied at each launch

struct ClipEntry {
  const void* src;
  void* dst;
  int64_t n;            // elements
};

template <int N>
struct ClipTable {
  ClipEntry e[N];
  int32_t chunk0[N + 1];   // chunk prefix: tensor i has chunks [chunk0[i], chunk0[i + 1])
  uint32_t bf16[(N + 31) / 32];
  int n_tensors;
};

struct ClipScaleArgs {
  const double* sumsq;  // [n_sums] added in order
  int n_sums;
  double max_norm;
  float* norm;          // [1], written by CTA 0 of the launch that has it
};

// Chunk c of the table: its tensor, element range and type.
template <int N>
__device__ __forceinline__ int clip_tensor(const ClipTable<N>& t, int c) {
  int lo = 0, hi = t.n_tensors - 1;   // largest i with chunk0[i] <= c (every tensor has a chunk)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.chunk0[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double sq(float f) { return (double)f * (double)f; }

template <typename T>
__device__ __forceinline__ float clip_load1(const T* p) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(*p);
  else return *p;
}

template <typename T>
__device__ __forceinline__ double sum_sq_16(const uint4& v) {
  if constexpr (sizeof(T) == 2) {
    float f[8];
    bf16x8_to_f32(v, f);
    return ((sq(f[0]) + sq(f[1])) + (sq(f[2]) + sq(f[3]))) + ((sq(f[4]) + sq(f[5])) + (sq(f[6]) + sq(f[7])));
  } else {
    return (sq(__uint_as_float(v.x)) + sq(__uint_as_float(v.y))) +
           (sq(__uint_as_float(v.z)) + sq(__uint_as_float(v.w)));
  }
}

// This thread's part of sum g^2 over n elements at p (any alignment of T).
template <typename T>
__device__ __forceinline__ double chunk_sum_sq(const T* p, int n) {
  constexpr int V = 16 / sizeof(T);
  const int tid = threadIdx.x;
  int head = (int)(((16u - (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / sizeof(T));
  if (head > n) head = n;
  double s = 0.0;
  if (tid < head) s = sq(clip_load1(p + tid));
  const uint4* q = reinterpret_cast<const uint4*>(p + head);
  const int nv = (n - head) / V;
  constexpr int U = 4;
  for (int i = tid; i < nv; i += U * kClipThreads) {
    uint4 v[U];
#pragma unroll
    for (int j = 0; j < U; ++j)
      v[j] = i + j * kClipThreads < nv ? __ldg(q + i + j * kClipThreads) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < U; ++j) s += sum_sq_16<T>(v[j]);
  }
  const int done = head + nv * V;
  if (tid < n - done) s += sq(clip_load1(p + done + tid));
  return s;
}

// Sum over the CTA in a fixed order; valid in thread 0.
__device__ __forceinline__ double cta_sum(double v) {
  __shared__ double warp_sum[kClipThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < kClipThreads / 32; ++w) v += warp_sum[w];
  return v;
}

template <int N>
__global__ void __launch_bounds__(kClipThreads)
grad_sumsq_kernel(const __grid_constant__ ClipTable<N> t, double* partial) {
  pdl_launch_dependents();
  pdl_wait();
  const int chunks = t.chunk0[t.n_tensors];
  double s = 0.0;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = clip_tensor(t, c);
    const int64_t off = (int64_t)(c - t.chunk0[i]) * kClipChunk;
    const int64_t left = t.e[i].n - off;
    const int n = left < kClipChunk ? (int)left : kClipChunk;
    if (t.bf16[i >> 5] >> (i & 31) & 1u) s += chunk_sum_sq(static_cast<const __nv_bfloat16*>(t.e[i].src) + off, n);
    else s += chunk_sum_sq(static_cast<const float*>(t.e[i].src) + off, n);
  }
  s = cta_sum(s);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// Total of n partial sums by one CTA, in a fixed order (every thread returns it).
__device__ __forceinline__ double total_of(const double* p, int n) {
  __shared__ double total;
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kClipThreads) s += p[i];
  s = cta_sum(s);
  if (threadIdx.x == 0) total = s;
  __syncthreads();
  return total;
}

// The total itself and, if asked for, the norm.
static __global__ void __launch_bounds__(kClipThreads)
grad_sumsq_total_kernel(const double* partial, int n, double* sumsq, float* norm) {
  pdl_launch_dependents();
  pdl_wait();
  const double s = total_of(partial, n);
  if (threadIdx.x == 0) {
    if (sumsq) *sumsq = s;
    if (norm) *norm = (float)sqrt(s);
  }
}

// The coefficient as the sum of two fp32 values: 48 of its bits, so that a scaled gradient is
// rounded once (with an fp32 coefficient twice: up to a whole step of fp32 off, and the norm
// after clipping off by the coefficient's rounding).  It costs a multiplication, which HBM hides.
// A coefficient below 2^-100, whose low part fp32 would lose (below 2^-126 the high one too, while the
// gradients that made so large a norm may scale to ordinary values), multiplies in 64 bits.
// (One form per launch, not per value: 600 MB of bf16 into others 399 us with the choice in the loop,
// 391 without.)
struct ScaleFp32 {   // 1, when f may be infinite, and values that fp32 has
  float c;
  __device__ __forceinline__ float operator()(float f) const { return f * c; }
};
struct ScaleTwoFp32 {
  float hi, lo;
  __device__ __forceinline__ float operator()(float f) const { return fmaf(f, hi, f * lo); }
};
struct ScaleFp64 {
  double c;
  __device__ __forceinline__ float operator()(float f) const { return (float)((double)f * c); }
};

template <class S>
__device__ __forceinline__ uint4 scale_16(const uint4& v, const S& c, __nv_bfloat16) {
  float f[8];
  bf16x8_to_f32(v, f);
  return make_uint4(pack_bf16x2(c(f[0]), c(f[1])), pack_bf16x2(c(f[2]), c(f[3])),
                    pack_bf16x2(c(f[4]), c(f[5])), pack_bf16x2(c(f[6]), c(f[7])));
}
template <class S>
__device__ __forceinline__ uint4 scale_16(const uint4& v, const S& c, float) {
  return make_uint4(__float_as_uint(c(__uint_as_float(v.x))), __float_as_uint(c(__uint_as_float(v.y))),
                    __float_as_uint(c(__uint_as_float(v.z))), __float_as_uint(c(__uint_as_float(v.w))));
}

// dst = c src over n elements; 16-byte accesses where both sides have the same offset from a
// 16-byte boundary.  src and dst are the same buffer or do not overlap.
template <typename T, class S>
__device__ __forceinline__ void chunk_scale(const T* src, T* dst, int n, const S& c) {
  constexpr int V = 16 / sizeof(T);
  const int tid = threadIdx.x;
  auto one = [&](int i) {
    const float f = c(clip_load1(src + i));
    if constexpr (sizeof(T) == 2) dst[i] = __float2bfloat16_rn(f);
    else dst[i] = f;
  };
  if ((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(dst)) & 15u) {
    for (int i = tid; i < n; i += kClipThreads) one(i);
    return;
  }
  int head = (int)(((16u - (uint32_t)(reinterpret_cast<uintptr_t>(src) & 15u)) & 15u) / sizeof(T));
  if (head > n) head = n;
  if (tid < head) one(tid);
  const uint4* q = reinterpret_cast<const uint4*>(src + head);
  uint4* o = reinterpret_cast<uint4*>(dst + head);
  const int nv = (n - head) / V;
  constexpr int U = 4;
  for (int i = tid; i < nv; i += U * kClipThreads) {
    uint4 v[U];
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (i + j * kClipThreads < nv) v[j] = q[i + j * kClipThreads];
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (i + j * kClipThreads < nv) o[i + j * kClipThreads] = scale_16(v[j], c, T{});
  }
  const int done = head + nv * V;
  if (tid < n - done) one(done + tid);
}

// The coefficient: 1 when the norm is within max_norm or not finite (the caller sees the norm
// and skips the step; a NaN that spread to every gradient could not be told from its source).
__device__ __forceinline__ double clip_coef(double norm, double max_norm) {
  return norm > max_norm && norm < __longlong_as_double(0x7ff0000000000000LL) ? max_norm / norm : 1.0;
}

template <int N>
__global__ void __launch_bounds__(kClipThreads)
grad_scale_kernel(const __grid_constant__ ClipTable<N> t, ClipScaleArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const double norm = sqrt(total_of(a.sumsq, a.n_sums));
  if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
  const double coef = clip_coef(norm, a.max_norm);
  const int chunks = t.chunk0[t.n_tensors];
  auto scale = [&](const auto& c) {
    // last chunks first: they were read last and may still be in L2
    for (int k = blockIdx.x; k < chunks; k += gridDim.x) {
      const int i = clip_tensor(t, chunks - 1 - k);
      if (coef == 1.0 && t.e[i].src == t.e[i].dst) continue;   // in place and nothing to scale
      const int64_t off = (int64_t)(chunks - 1 - k - t.chunk0[i]) * kClipChunk;
      const int64_t left = t.e[i].n - off;
      const int n = left < kClipChunk ? (int)left : kClipChunk;
      if (t.bf16[i >> 5] >> (i & 31) & 1u)
        chunk_scale(static_cast<const __nv_bfloat16*>(t.e[i].src) + off, static_cast<__nv_bfloat16*>(t.e[i].dst) + off, n, c);
      else
        chunk_scale(static_cast<const float*>(t.e[i].src) + off, static_cast<float*>(t.e[i].dst) + off, n, c);
    }
  };
  const float hi = (float)coef, lo = (float)(coef - (double)hi);
  if (coef < 0x1p-100) scale(ScaleFp64{coef});
  else if (lo == 0.0f) scale(ScaleFp32{hi});
  else scale(ScaleTwoFp32{hi, lo});
}

}  // namespace moe
