// block_norm.cuh -- the norms before and after a block, fused with its gate, the residual
// scale and the residual add, forward and backward.
//
// Per row of width d, x the residual stream, y the block's output, s(v) = 1 / sqrt(mean v^2 + eps):
//   p = y s(y) w_post         (p = y without a norm after the block)
//   r = beta x + gate p       (gate per channel, per token, or absent)
//   u = r s(r) w_pre          (the next block's input; absent without a norm before it)
// and with dr, du the gradients of r and u, xh = r s(r), yh = y s(y), means over the row:
//   g      = dr + s(r) (du w_pre - xh mean(du w_pre xh))
//   dx     = beta g
//   dy     = s(y) (q - yh mean(q yh)),  q = g gate w_post     (without w_post: dy = g gate)
//   d_pre  = sum_t du xh,  d_post = sum_t g gate yh,
//   d_gate = sum_t g p (per channel) or sum_j g p (per token)
//
// One CTA of TPR threads holds a row in registers (NV accesses of V elements a thread), so
// each tensor crosses HBM once; every sum and statistic is fp32.  u and the statistic s(r)
// come from r before it is rounded to its type (one rounding less than reading it back).
#pragma once

#include "ptx.cuh"

namespace moe {

constexpr int kNormMaxD = 16384;
constexpr int kNormMaxParts = 592;   // CTAs of the backward, each with its own column sums

enum NormGate : int { kGateNone = 0, kGateChannel = 1, kGateToken = 2 };

struct BlockNormArgs {
  const void* x;       // [T, d]
  const void* y;       // [T, d] or nullptr: r = x is not written
  const float* gate;   // [d], [T] or nullptr
  const float* w_post; // [d] or nullptr
  const float* w_pre;  // [d] or nullptr
  void* r;             // [T, d] (y given)
  void* u;             // [T, d] (w_pre given)
  float* s_post;       // [T] (w_post given)
  float* s_pre;        // [T] (w_pre given)
  int64_t T;
  int d, gate_kind;
  float beta, eps;
};

struct BlockNormBwdArgs {
  const void* y;       // [T, d] or nullptr
  const void* r;       // [T, d]
  const void* dr;      // [T, d] or nullptr: zero
  const void* du;      // [T, d] (w_pre given)
  const float* gate;
  const float* w_post;
  const float* w_pre;
  const float* s_post;
  const float* s_pre;
  void* dx;
  void* dy;            // (y given)
  float* d_gate_tok;   // [T] (gate per token)
  float* part_pre;     // [gridDim.x, d] column sums of this CTA's rows: du xh
  float* part_s;       // [gridDim.x, d]                               g (token gate) yh
  int64_t T;
  int d, gate_kind;
  float beta;
};

// V consecutive elements of T widened to fp32, and back with one rounding.
template <typename T, int V>
struct RowVec;
template <>
struct RowVec<__nv_bfloat16, 8> {
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&f)[8]) {
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i), f);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) =
        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct RowVec<float, 4> {
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&f)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[4]) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct RowVec<__nv_bfloat16, 1> {
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&f)[1]) {
    f[0] = __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[1]) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f[0]);
  }
};
template <>
struct RowVec<float, 1> {
  static __device__ __forceinline__ void load(const void* p, int64_t i, float (&f)[1]) {
    f[0] = static_cast<const float*>(p)[i];
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[1]) {
    static_cast<float*>(p)[i] = f[0];
  }
};

// V consecutive fp32 parameters (weights, channel gate): 16-byte loads when V allows.
template <int V>
__device__ __forceinline__ void load_param(const float* p, int i, float (&f)[V]) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int q = 0; q < V / 4; ++q) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + i) + q);
      f[4 * q] = v.x; f[4 * q + 1] = v.y; f[4 * q + 2] = v.z; f[4 * q + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < V; ++q) f[q] = __ldg(p + i + q);
  }
}

// Sum of v over the CTA's TPR threads, the same value in each (lanes by butterfly, then the
// warps in order).  The next call that uses `buf` comes after another call's barrier.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR > 32) {
    constexpr int kWarps = TPR / 32;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += buf[w];
  }
  return v;
}

template <typename T, int V, int NV, int TPR>
__global__ void __launch_bounds__(TPR) block_norm_kernel(BlockNormArgs a) {
  using RV = RowVec<T, V>;
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float red[2][32];
  const int64_t row = blockIdx.x;
  const int64_t base = row * a.d;
  const float inv_d = 1.0f / (float)a.d;
  float r[NV][V], y[NV][V];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (threadIdx.x + i * TPR) * V;
    if (c < a.d) {
      RV::load(a.x, base + c, r[i]);
      if (a.y) RV::load(a.y, base + c, y[i]);
    }
  }
  if (a.y) {
    float s = 1.0f;
    if (a.w_post) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((threadIdx.x + i * TPR) * V < a.d)
#pragma unroll
          for (int j = 0; j < V; ++j) ss = fmaf(y[i][j], y[i][j], ss);
      s = __frsqrt_rn(fmaf(row_sum<TPR>(ss, red[0]), inv_d, a.eps));
      if (threadIdx.x == 0) a.s_post[row] = s;
    }
    const float gt = a.gate_kind == kGateToken ? __ldg(a.gate + row) : 1.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (threadIdx.x + i * TPR) * V;
      if (c < a.d) {
        float w[V], gc[V];
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] = gc[j] = 1.0f;
        if (a.w_post) load_param<V>(a.w_post, c, w);
        if (a.gate_kind == kGateChannel) load_param<V>(a.gate, c, gc);
#pragma unroll
        for (int j = 0; j < V; ++j) r[i][j] = fmaf(a.beta, r[i][j], y[i][j] * s * w[j] * (gc[j] * gt));
        RV::store(a.r, base + c, r[i]);
      }
    }
  }
  if (a.w_pre) {
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((threadIdx.x + i * TPR) * V < a.d)
#pragma unroll
        for (int j = 0; j < V; ++j) ss = fmaf(r[i][j], r[i][j], ss);
    const float s = __frsqrt_rn(fmaf(row_sum<TPR>(ss, red[1]), inv_d, a.eps));
    if (threadIdx.x == 0) a.s_pre[row] = s;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (threadIdx.x + i * TPR) * V;
      if (c < a.d) {
        float w[V];
        load_param<V>(a.w_pre, c, w);
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] *= r[i][j] * s;
        RV::store(a.u, base + c, w);
      }
    }
  }
}

// The CTA walks rows blockIdx.x, blockIdx.x + gridDim.x, ... and keeps its columns' sums in
// registers, so the parameter gradients cost one [gridDim.x, d] array of partial sums.
template <typename T, int V, int NV, int TPR>
__global__ void __launch_bounds__(TPR) block_norm_bwd_kernel(BlockNormBwdArgs a) {
  using RV = RowVec<T, V>;
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float red[2][2][32];   // two rows' sums: a row's may still be read while the next's come
  int par = 0;
  const float inv_d = 1.0f / (float)a.d;
  float acc_pre[NV][V], acc_s[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) acc_pre[i][j] = acc_s[i][j] = 0.f;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, par ^= 1) {
    const int64_t base = row * a.d;
    float g[NV][V], y[NV][V];
    if (a.w_pre) {
      float xh[NV][V], dh[NV][V];
      const float s = __ldg(a.s_pre + row);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (threadIdx.x + i * TPR) * V;
        if (c < a.d) {
          RV::load(a.r, base + c, xh[i]);
          RV::load(a.du, base + c, dh[i]);
          if (a.dr) RV::load(a.dr, base + c, g[i]);
          if (a.y) RV::load(a.y, base + c, y[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (threadIdx.x + i * TPR) * V;
        if (c < a.d) {
          float w[V];
          load_param<V>(a.w_pre, c, w);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            xh[i][j] *= s;
            acc_pre[i][j] = fmaf(dh[i][j], xh[i][j], acc_pre[i][j]);
            dh[i][j] *= w[j];
            sum = fmaf(dh[i][j], xh[i][j], sum);
          }
        }
      }
      const float mean = row_sum<TPR>(sum, red[par][0]) * inv_d;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float t = s * (dh[i][j] - xh[i][j] * mean);
          g[i][j] = a.dr ? g[i][j] + t : t;
        }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (threadIdx.x + i * TPR) * V;
        if (c < a.d) {
          RV::load(a.dr, base + c, g[i]);
          if (a.y) RV::load(a.y, base + c, y[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (threadIdx.x + i * TPR) * V;
      if (c < a.d) {
        float dx[V];
#pragma unroll
        for (int j = 0; j < V; ++j) dx[j] = a.beta * g[i][j];
        RV::store(a.dx, base + c, dx);
      }
    }
    if (a.y) {
      const float s = a.w_post ? __ldg(a.s_post + row) : 1.0f;
      const float gt = a.gate_kind == kGateToken ? __ldg(a.gate + row) : 1.0f;
      float sum = 0.f;
      // y becomes yh, g becomes g times the channel gate and w_post (q without the token gate)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (threadIdx.x + i * TPR) * V;
        if (c < a.d) {
          float w[V], gc[V];
#pragma unroll
          for (int j = 0; j < V; ++j) w[j] = gc[j] = 1.0f;
          if (a.w_post) load_param<V>(a.w_post, c, w);
          if (a.gate_kind == kGateChannel) load_param<V>(a.gate, c, gc);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            y[i][j] *= s;
            acc_s[i][j] = fmaf(g[i][j] * gt, y[i][j], acc_s[i][j]);
            g[i][j] *= gc[j] * w[j];
            sum = fmaf(g[i][j], y[i][j], sum);
          }
        }
      }
      float mean = 0.f;
      if (a.w_post || a.gate_kind == kGateToken) {   // uniform over the CTA
        sum = row_sum<TPR>(sum, red[par][1]);
        if (a.gate_kind == kGateToken && threadIdx.x == 0) a.d_gate_tok[row] = sum;
        if (a.w_post) mean = sum * inv_d;
      }
      const float sg = s * gt;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (threadIdx.x + i * TPR) * V;
        if (c < a.d) {
          float dy[V];
#pragma unroll
          for (int j = 0; j < V; ++j) dy[j] = sg * (g[i][j] - y[i][j] * mean);
          RV::store(a.dy, base + c, dy);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (threadIdx.x + i * TPR) * V;
    if (c < a.d) {
      const int64_t o = (int64_t)blockIdx.x * a.d + c;
      if (a.part_pre) RowVec<float, V % 4 == 0 ? 4 : 1>::store(a.part_pre, o, *reinterpret_cast<float(*)[V % 4 == 0 ? 4 : 1]>(&acc_pre[i][0]));
      if (a.part_s) RowVec<float, V % 4 == 0 ? 4 : 1>::store(a.part_s, o, *reinterpret_cast<float(*)[V % 4 == 0 ? 4 : 1]>(&acc_s[i][0]));
      if constexpr (V == 8) {
        if (a.part_pre) RowVec<float, 4>::store(a.part_pre, o + 4, *reinterpret_cast<float(*)[4]>(&acc_pre[i][4]));
        if (a.part_s) RowVec<float, 4>::store(a.part_s, o + 4, *reinterpret_cast<float(*)[4]>(&acc_s[i][4]));
      }
    }
  }
}

// Column totals of the partial sums, in a fixed order; the channel gate's gradient and the
// weight's after a block share one sum: d_gate = w_post S, d_post = gate S.
struct NormReduceArgs {
  const float* part_pre;   // [parts, d] or nullptr
  const float* part_s;     // [parts, d] or nullptr
  int parts, d;
  const float* w_post;     // or nullptr
  const float* gate_ch;    // channel gate or nullptr
  float* d_pre;
  float* d_post;           // (w_post given)
  float* d_gate;           // (channel gate)
};

constexpr int kNormRedRows = 32;

static __global__ void __launch_bounds__(32 * kNormRedRows) block_norm_reduce_kernel(NormReduceArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float sh[kNormRedRows][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  const float* part = blockIdx.y == 0 ? a.part_pre : a.part_s;
  if (!part) return;   // uniform over the CTA
  float v = 0.f;
  if (c < a.d)
    for (int p = ty; p < a.parts; p += kNormRedRows) v += part[(int64_t)p * a.d + c];
  sh[ty][tx] = v;
  __syncthreads();
  if (ty != 0 || c >= a.d) return;
  v = 0.f;
#pragma unroll
  for (int q = 0; q < kNormRedRows; ++q) v += sh[q][tx];
  if (blockIdx.y == 0) {
    a.d_pre[c] = v;
  } else {
    if (a.d_post) a.d_post[c] = a.gate_ch ? v * a.gate_ch[c] : v;
    if (a.d_gate) a.d_gate[c] = a.w_post ? v * a.w_post[c] : v;
  }
}

}  // namespace moe
