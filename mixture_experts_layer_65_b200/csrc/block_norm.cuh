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
// A row belongs to one CTA (to one warp up to 64 accesses of V elements), so each tensor crosses
// HBM once.  CTAs are persistent: parameters stay in registers, the next row is on its way
// to shared memory while this one is reduced (each thread copies, and later reads, its own 16
// bytes, so nothing waits for another thread's copies), and the backward's column sums are
// kept per CTA.  Rows of other widths than whole 16-byte accesses start anywhere: their accesses
// still are the aligned ones that the row touches (SHIFT), the elements of neighbouring rows in the
// first and the last masked; a CTA (a warp) takes rows that all start alike, so that a thread's
// columns, its parameters and column sums stay its own.  Sums and statistics are fp32, the CTAs'
// column sums added up in 64 bits.  u and the statistic s(r) come from r before it is rounded to its
// type (one rounding less than reading it back).
//
// Bound by HBM: bf16, both norms and a channel gate, forward 6.2 TB/s at 32,768 x 4096 (174 us, 0.94
// of the copy rate; 185 us with other buffers each time) and 5.8 at 16,384 x 2048 (46 us); backward
// 5.3 and 5.2 to 5.3 (303 and 75 to 77 us), where two chained row sums and 20 instructions a value
// begin to show.  Odd widths are bound by those instructions (1.2e8 elements of bf16, d = 2001: 210 us
// and 365, 4.6 and 3.9 TB/s; by single elements 491 and 899), rows of 64 columns by their number (8 of 32 lanes read: 1.8 TB/s), rows
// past 8192 columns by barriers of 1024 threads (3.4 and 1.9 TB/s).
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

// V consecutive elements of T: as loaded, widened to fp32, and stored with one rounding.
template <typename T, int V>
struct RowVec;
template <>
struct RowVec<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ Raw load(const void* p, int64_t i) {
    return *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
  }
  static __device__ __forceinline__ void widen(const Raw& r, float (&f)[8]) { bf16x8_to_f32(r, f); }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) =
        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct RowVec<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ Raw load(const void* p, int64_t i) {
    return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  }
  static __device__ __forceinline__ void widen(const Raw& r, float (&f)[4]) {
    f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[4]) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct RowVec<__nv_bfloat16, 1> {
  using Raw = __nv_bfloat16;
  static __device__ __forceinline__ Raw load(const void* p, int64_t i) { return static_cast<const __nv_bfloat16*>(p)[i]; }
  static __device__ __forceinline__ void widen(const Raw& r, float (&f)[1]) { f[0] = __bfloat162float(r); }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[1]) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f[0]);
  }
};
template <>
struct RowVec<float, 1> {
  using Raw = float;
  static __device__ __forceinline__ Raw load(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
  static __device__ __forceinline__ void widen(const Raw& r, float (&f)[1]) { f[0] = r; }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[1]) {
    static_cast<float*>(p)[i] = f[0];
  }
};

// Whether columns [c, c + V) reach over the row's ends (only with SHIFT), and column c + j is inside.
template <int V, bool SHIFT>
__device__ __forceinline__ bool at_edge(int c, int d) { return SHIFT && (c < 0 || c + V > d); }
__device__ __forceinline__ bool inside(int c, int d) { return c >= 0 && c < d; }

// V columns of a row's result, those inside the row: `base` is the row's first element.
template <typename T, int V, bool SHIFT>
__device__ __forceinline__ void store_row(void* p, int64_t base, int c, int d, const float (&f)[V]) {
  if (at_edge<V, SHIFT>(c, d)) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (inside(c + j, d)) {
        const float one[1] = {f[j]};
        RowVec<T, 1>::store(p, base + c + j, one);
      }
  } else {
    RowVec<T, V>::store(p, base + c, f);
  }
}

// V consecutive fp32 parameters (weights, channel gate): 16-byte loads when V allows; with SHIFT one
// by one, 0 outside the row.
template <int V, bool SHIFT>
__device__ __forceinline__ void load_param(const float* p, int i, int d, float (&f)[V]) {
  if constexpr (SHIFT) {
#pragma unroll
    for (int q = 0; q < V; ++q) f[q] = inside(i + q, d) ? __ldg(p + i + q) : 0.f;
  } else if constexpr (V % 4 == 0) {
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

// V consecutive fp32 values stored to columns c.. of p.
template <int V, bool SHIFT>
__device__ __forceinline__ void store_f32(float* p, int c, int d, const float (&f)[V]) {
  if constexpr (SHIFT) {
#pragma unroll
    for (int q = 0; q < V; ++q)
      if (inside(c + q, d)) p[c + q] = f[q];
  } else if constexpr (V % 4 == 0) {
#pragma unroll
    for (int q = 0; q < V / 4; ++q)
      *(reinterpret_cast<float4*>(p + c) + q) = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
  } else {
#pragma unroll
    for (int q = 0; q < V; ++q) p[c + q] = f[q];
  }
}

// V values at a time, two per instruction where V is even (each product and sum rounded to
// nearest, as the scalar instructions do).
__device__ __forceinline__ uint64_t as_pair(float x, float y) {
  return static_cast<uint64_t>(__float_as_uint(x)) | static_cast<uint64_t>(__float_as_uint(y)) << 32;
}
__device__ __forceinline__ void from_pair(uint64_t v, float& x, float& y) {
  x = __uint_as_float(static_cast<uint32_t>(v));
  y = __uint_as_float(static_cast<uint32_t>(v >> 32));
}
// d = a b + c
template <int V>
__device__ __forceinline__ void vfma(float (&d)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      uint64_t v;
      asm("fma.rn.f32x2 %0, %1, %2, %3;"
          : "=l"(v)
          : "l"(as_pair(a[j], a[j + 1])), "l"(as_pair(b[j], b[j + 1])), "l"(as_pair(c[j], c[j + 1])));
      from_pair(v, d[j], d[j + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = fmaf(a[j], b[j], c[j]);
  }
}
// d = a b
template <int V>
__device__ __forceinline__ void vmul(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      uint64_t v;
      asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(as_pair(a[j], a[j + 1])), "l"(as_pair(b[j], b[j + 1])));
      from_pair(v, d[j], d[j + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = a[j] * b[j];
  }
}
// d += a
template <int V>
__device__ __forceinline__ void vadd(float (&d)[V], const float (&a)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      uint64_t v;
      asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(as_pair(d[j], d[j + 1])), "l"(as_pair(a[j], a[j + 1])));
      from_pair(v, d[j], d[j + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] += a[j];
  }
}
template <int V>
__device__ __forceinline__ void vset(float (&d)[V], float x) {
#pragma unroll
  for (int j = 0; j < V; ++j) d[j] = x;
}
template <int V>
__device__ __forceinline__ float vsum(const float (&a)[V]) {
  float t = a[0];
#pragma unroll
  for (int j = 1; j < V; ++j) t += a[j];
  return t;
}

// Sum of v over a row's threads, the same value in each: lanes by butterfly, then (WARP_ROW:
// a warp has the row to itself) the CTA's warps by another.  The next call that uses `buf` comes
// after another call's barrier.
template <bool WARP_ROW>
__device__ __forceinline__ float row_sum(float v, float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (!WARP_ROW) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < (int)(blockDim.x >> 5) ? buf[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// Threads of a kernel: MAXT = 32 stands for one warp per row, eight rows a CTA; else the CTA has
// as many threads as a row needs, at most MAXT.  The kernels' second launch bound is the CTAs that
// are to fit an SM: without it the forward's took up to 163 registers, one CTA (bf16, d = 333: 475
// us against 323; d = 3333: 376 against 236; 1.2e8 elements).
constexpr int kNormWarps = 8;
constexpr int kNormRing = 2;   // rows in shared memory: the one at work and the next
                               // (three: 2% faster at d = 4096, up to 11% slower elsewhere)
__host__ __device__ constexpr int norm_max_threads(int maxt) { return maxt == 32 ? 32 * kNormWarps : maxt; }
// Parameters are kept in registers up to 512 threads a CTA (128 registers a thread).
__host__ __device__ constexpr bool norm_keeps(int maxt) { return maxt <= 512; }
// Rows go through the ring there too, when they are read 16 bytes at a time.
__host__ __device__ constexpr bool norm_rings(int v, int maxt) { return v > 1 && norm_keeps(maxt); }
__host__ __device__ constexpr size_t norm_ring_bytes(int streams, int nv, int threads) {
  return (size_t)kNormRing * streams * nv * threads * 16;
}

// K row streams of one thread, NV accesses each: through the ring, or (no ring) to registers: one
// row ahead (EARLY) or when the row's turn comes.  An absent stream has a null pointer.
template <typename T, int V, int NV, int K, bool RING, bool EARLY, bool SHIFT>
struct RowStreams {
  using RV = RowVec<T, V>;
  using Raw = typename RV::Raw;
  const void* src[K];
  uint32_t smem;      // this thread's first 16 bytes
  uint32_t pitch;     // bytes between a thread's slots
  int slot;           // of the row at work
  Raw cur[RING ? 1 : K][NV], coming[EARLY ? K : 1][NV];

  __device__ __forceinline__ void init(uint8_t* ring) {
    if constexpr (RING) {
      smem = smem_u32(ring) + threadIdx.x * 16;
      pitch = blockDim.x * 16;
      slot = 0;
    }
  }
  // Ask for a row (col(i): this thread's columns) into the ring, `ahead` rows behind the one at
  // work; a row past the end only keeps the count.
  template <class C>
  __device__ __forceinline__ void ask(int64_t row, int64_t T_, int d, int ahead, C&& col) {
    if constexpr (RING) {
      if (row < T_) {
        const int to = (slot + ahead) % kNormRing;
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (src[k])
#pragma unroll
            for (int i = 0; i < NV; ++i)
              if (col(i) < d) {
                const T* from = static_cast<const T*>(src[k]) + row * d + col(i);
                const uint32_t at = smem + ((to * K + k) * NV + i) * pitch;
                if constexpr (SHIFT) {   // not past the tensor's end
                  const int64_t left = ((T_ - row) * d - col(i)) * (int64_t)sizeof(T);
                  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from),
                               "r"(left < 16 ? (int)left : 16)
                               : "memory");
                } else {
                  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
                }
              }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    } else if constexpr (EARLY) {
      if (row < T_ && ahead == 0)
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (src[k])
#pragma unroll
            for (int i = 0; i < NV; ++i)
              if (col(i) < d) coming[k][i] = RV::load(src[k], row * d + col(i));
    }
  }
  // The row at work is there.
  template <class C>
  __device__ __forceinline__ void take(int64_t row, int d, C&& col) {
    if constexpr (RING) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kNormRing - 1) : "memory");
    } else if constexpr (EARLY) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i) cur[k][i] = coming[k][i];
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (src[k])
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (col(i) < d) cur[k][i] = RV::load(src[k], row * d + col(i));
    }
  }
  // Access i of stream k, columns c..; zeros outside the row.
  __device__ __forceinline__ void get(int k, int i, int c, int d, float (&f)[V]) const {
    if constexpr (RING) {
      uint32_t x, y, z, w;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(x), "=r"(y), "=r"(z), "=r"(w)
                   : "r"(smem + ((slot * K + k) * NV + i) * pitch)
                   : "memory");
      if constexpr (sizeof(T) == 2) {
        RV::widen(make_uint4(x, y, z, w), f);
      } else {
        f[0] = __uint_as_float(x); f[1] = __uint_as_float(y); f[2] = __uint_as_float(z); f[3] = __uint_as_float(w);
      }
    } else {
      RV::widen(cur[k][i], f);
    }
    if (at_edge<V, SHIFT>(c, d)) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (!inside(c + j, d)) f[j] = 0.f;
    }
  }
  __device__ __forceinline__ void next() {
    if constexpr (RING) slot = slot + 1 == kNormRing ? 0 : slot + 1;
  }
};

// The columns' parameters of one thread: post weight times channel gate, and the pre weight, in
// registers (KEEP) or read again for every row.
template <int V, int NV, bool KEEP, bool SHIFT>
struct RowParams {
  const float *w_post, *gate_ch, *w_pre;   // nullptr: ones
  int d;
  float wq[KEEP ? NV : 1][V], wp[KEEP ? NV : 1][V];

  __device__ __forceinline__ void scale_of(int c, float (&w)[V]) const {
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] = 1.0f;
    if (w_post) load_param<V, SHIFT>(w_post, c, d, w);
    if (gate_ch) {
      float gc[V];
      load_param<V, SHIFT>(gate_ch, c, d, gc);
#pragma unroll
      for (int j = 0; j < V; ++j) w[j] *= gc[j];
    }
  }
  template <class C>
  __device__ __forceinline__ void init(C&& col) {
    if constexpr (KEEP) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < d) {
          scale_of(col(i), wq[i]);
          if (w_pre) load_param<V, SHIFT>(w_pre, col(i), d, wp[i]);
        }
    }
  }
  __device__ __forceinline__ void post(int i, int c, float (&w)[V]) const {
    if constexpr (KEEP) {
#pragma unroll
      for (int j = 0; j < V; ++j) w[j] = wq[i][j];
    } else {
      scale_of(c, w);
    }
  }
  __device__ __forceinline__ void pre(int i, int c, float (&w)[V]) const {
    if constexpr (KEEP) {
#pragma unroll
      for (int j = 0; j < V; ++j) w[j] = wp[i][j];
    } else {
      load_param<V, SHIFT>(w_pre, c, d, w);
    }
  }
};

template <typename T, int V, int NV, int MAXT, bool SHIFT>
__global__ void __launch_bounds__(norm_max_threads(MAXT), V > 1 && MAXT <= 384 ? 2 : 1) block_norm_kernel(BlockNormArgs a) {
  constexpr bool kWarpRow = MAXT == 32;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][2][32];   // two rows' sums: a row's may still be read while the next's come
  pdl_launch_dependents();
  pdl_wait();
  const int tid = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int tpr = kWarpRow ? 32 : blockDim.x;
  const int64_t step = kWarpRow ? (int64_t)gridDim.x * kNormWarps : gridDim.x;
  const float inv_d = 1.0f / (float)a.d;
  int64_t row = kWarpRow ? (int64_t)blockIdx.x * kNormWarps + (threadIdx.x >> 5) : blockIdx.x;
  // elements between an aligned access and the row's start, the same for all of this thread's rows
  const int shift = SHIFT ? (int)(row % V) * (a.d % V) % V : 0;
  auto col = [&](int i) { return (tid + i * tpr) * V - shift; };
  constexpr bool kRing = norm_rings(V, MAXT), kEarly = !kRing && norm_keeps(MAXT);
  RowStreams<T, V, NV, 2, kRing, kEarly, SHIFT> in{{a.x, a.y}};
  in.init(ring);
#pragma unroll
  for (int i = 0; i < kNormRing - 1; ++i) in.ask(row + i * step, a.T, a.d, i, col);
  RowParams<V, NV, norm_keeps(MAXT), SHIFT> par{a.w_post, a.gate_kind == kGateChannel ? a.gate : nullptr, a.w_pre,
                                                a.d};
  par.init(col);
  // the row's own parameter is loaded a row ahead too
  auto token_gate = [&](int64_t i) { return a.gate_kind == kGateToken && i < a.T ? __ldg(a.gate + i) : 1.0f; };
  float gt_next = token_gate(row);
  for (int odd = 0; row < a.T; row += step, odd ^= 1) {
    in.ask(row + (kNormRing - 1) * step, a.T, a.d, kNormRing - 1, col);
    in.take(row, a.d, col);
    if (kEarly) in.ask(row + step, a.T, a.d, 0, col);
    const float gt = gt_next;
    gt_next = token_gate(row + step);
    const int64_t base = row * a.d;
    float r[NV][V], p[NV][V], k[V], ss[V];
    vset(ss, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (col(i) < a.d) {
        in.get(0, i, col(i), a.d, r[i]);
        if (a.y) {
          in.get(1, i, col(i), a.d, p[i]);
          vfma(ss, p[i], p[i], ss);
        }
      }
    in.next();
    if (a.y) {
      float s = 1.0f;
      if (a.w_post) {
        s = __frsqrt_rn(fmaf(row_sum<kWarpRow>(vsum(ss), red[odd][0]), inv_d, a.eps));
        if (tid == 0) a.s_post[row] = s;
      }
      float b[V];
      vset(k, s * gt);
      vset(b, a.beta);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < a.d) {
          float w[V];
          par.post(i, col(i), w);
          vmul(p[i], p[i], w);
          vmul(r[i], r[i], b);
          vfma(r[i], p[i], k, r[i]);
          store_row<T, V, SHIFT>(a.r, base, col(i), a.d, r[i]);
        }
    }
    if (a.w_pre) {
      vset(ss, 0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < a.d) vfma(ss, r[i], r[i], ss);
      const float s = __frsqrt_rn(fmaf(row_sum<kWarpRow>(vsum(ss), red[odd][1]), inv_d, a.eps));
      if (tid == 0) a.s_pre[row] = s;
      vset(k, s);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < a.d) {
          float w[V];
          par.pre(i, col(i), w);
          vmul(r[i], r[i], k);
          vmul(w, w, r[i]);
          store_row<T, V, SHIFT>(a.u, base, col(i), a.d, w);
        }
    }
  }
}

// Column sums of the warps of a CTA (one warp per row), added in order by the CTA.
template <int V, int NV, bool SHIFT>
__device__ __forceinline__ void cta_columns(float (&acc)[NV][V], float* sh, float* part, int d, int shift) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWidth = NV * V * 32;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (lane + i * 32) * V + j - shift;
      if (!SHIFT || c >= 0) sh[warp * kWidth + c] = acc[i][j];
    }
  __syncthreads();
  for (int c = threadIdx.x; c < d; c += 32 * kNormWarps) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kNormWarps; ++w) v += sh[w * kWidth + c];
    part[c] = v;
  }
}

// As block_norm_kernel; the columns' sums stay in registers over a CTA's (warp's) rows, so the
// parameter gradients cost one [gridDim.x, d] array of partial sums each.
template <typename T, int V, int NV, int MAXT, bool SHIFT>
__global__ void __launch_bounds__(norm_max_threads(MAXT), MAXT == 160 ? 3 : MAXT == 320 ? 2 : 1) block_norm_bwd_kernel(BlockNormBwdArgs a) {
  constexpr bool kWarpRow = MAXT == 32;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int tpr = kWarpRow ? 32 : blockDim.x;
  const int64_t step = kWarpRow ? (int64_t)gridDim.x * kNormWarps : gridDim.x;
  const float inv_d = 1.0f / (float)a.d;
  int64_t row = kWarpRow ? (int64_t)blockIdx.x * kNormWarps + (threadIdx.x >> 5) : blockIdx.x;
  // elements between an aligned access and the row's start, the same for all of this thread's rows
  const int shift = SHIFT ? (int)(row % V) * (a.d % V) % V : 0;
  auto col = [&](int i) { return (tid + i * tpr) * V - shift; };
  enum { kR = 0, kDu = 1, kDr = 2, kY = 3 };
  constexpr bool kRing = norm_rings(V, MAXT);
  // values held from one sum to the next; without, they are read again behind the sum: there are too
  // few registers for two accesses' values beside their column sums
  constexpr bool kHolds = kRing && !(NV == 2 && MAXT >= 160);
  constexpr int kHeld = kHolds ? NV : 1;
  RowStreams<T, V, NV, 4, kRing, false, SHIFT> in{{a.w_pre ? a.r : nullptr, a.w_pre ? a.du : nullptr, a.dr, a.y}};
  in.init(ring);
#pragma unroll
  for (int i = 0; i < kNormRing - 1; ++i) in.ask(row + i * step, a.T, a.d, i, col);
  RowParams<V, NV, norm_keeps(MAXT), SHIFT> par{a.w_post, a.gate_kind == kGateChannel ? a.gate : nullptr, a.w_pre,
                                                a.d};
  par.init(col);
  float acc_pre[NV][V], acc_s[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) acc_pre[i][j] = acc_s[i][j] = 0.f;
  // the row's own values are loaded a row ahead too
  auto own = [&](const float* p, bool on, int64_t i) { return on && i < a.T ? __ldg(p + i) : 1.0f; };
  float pre_next = own(a.s_pre, a.w_pre, row), post_next = own(a.s_post, a.w_post, row);
  float gt_next = own(a.gate, a.gate_kind == kGateToken, row);
  for (int odd = 0; row < a.T; row += step, odd ^= 1) {
    in.ask(row + (kNormRing - 1) * step, a.T, a.d, kNormRing - 1, col);
    in.take(row, a.d, col);
    const float s_pre = pre_next, s_post = post_next, gt = gt_next;
    pre_next = own(a.s_pre, a.w_pre, row + step);
    post_next = own(a.s_post, a.w_post, row + step);
    gt_next = own(a.gate, a.gate_kind == kGateToken, row + step);
    const int64_t base = row * a.d;
    float g[NV][V], k[V], t[V], sum[V];
    if (a.w_pre) {
      float x[kHeld][V], u[kHeld][V];   // xh, du
      vset(sum, 0.f);
      vset(k, s_pre);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < a.d) {
          float w[V];
          in.get(kR, i, col(i), a.d, x[kHolds ? i : 0]);
          in.get(kDu, i, col(i), a.d, u[kHolds ? i : 0]);
          vmul(x[kHolds ? i : 0], x[kHolds ? i : 0], k);
          vmul(t, u[kHolds ? i : 0], x[kHolds ? i : 0]);
          vadd(acc_pre[i], t);
          par.pre(i, col(i), w);
          vfma(sum, t, w, sum);
        }
      const float mean = row_sum<kWarpRow>(vsum(sum), red[odd][0]) * inv_d;
      float m[V];
      vset(m, -mean * s_pre);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < a.d) {
          float w[V];
          if constexpr (!kHolds) {
            in.get(kR, i, col(i), a.d, x[kHolds ? i : 0]);
            in.get(kDu, i, col(i), a.d, u[kHolds ? i : 0]);
            vmul(x[kHolds ? i : 0], x[kHolds ? i : 0], k);
          }
          if (a.dr) in.get(kDr, i, col(i), a.d, g[i]);
          else vset(g[i], 0.f);
          par.pre(i, col(i), w);
          vmul(w, w, u[kHolds ? i : 0]);
          vfma(g[i], w, k, g[i]);
          vfma(g[i], x[kHolds ? i : 0], m, g[i]);
        }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < a.d) in.get(kDr, i, col(i), a.d, g[i]);
    }
    vset(k, a.beta);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (col(i) < a.d) {
        vmul(t, g[i], k);
        store_row<T, V, SHIFT>(a.dx, base, col(i), a.d, t);
      }
    if (a.y) {
      // g becomes q without the token gate: g times post weight and channel gate
      float y[kHeld][V], ks[V];   // yh
      vset(sum, 0.f);
      vset(k, gt);
      vset(ks, s_post);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < a.d) {
          float w[V];
          in.get(kY, i, col(i), a.d, y[kHolds ? i : 0]);
          vmul(y[kHolds ? i : 0], y[kHolds ? i : 0], ks);
          vmul(t, g[i], y[kHolds ? i : 0]);
          vfma(acc_s[i], t, k, acc_s[i]);
          par.post(i, col(i), w);
          vfma(sum, t, w, sum);
          vmul(g[i], g[i], w);
        }
      float mean = 0.f;
      if (a.w_post || a.gate_kind == kGateToken) {   // the same for every thread
        mean = row_sum<kWarpRow>(vsum(sum), red[odd][1]);
        if (a.gate_kind == kGateToken && tid == 0) a.d_gate_tok[row] = mean;
        mean *= inv_d;
      }
      float m[V];
      vset(k, s_post * gt);
      vset(m, -mean * (s_post * gt));
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (col(i) < a.d) {
          if constexpr (!kHolds) {
            in.get(kY, i, col(i), a.d, y[kHolds ? i : 0]);
            vmul(y[kHolds ? i : 0], y[kHolds ? i : 0], ks);
          }
          vmul(g[i], g[i], k);
          // (without a norm y has no part in dy, and 0 times an infinite y would be NaN)
          if (a.w_post) vfma(g[i], y[kHolds ? i : 0], m, g[i]);
          store_row<T, V, SHIFT>(a.dy, base, col(i), a.d, g[i]);
        }
    }
    in.next();
  }
  const int64_t o = (int64_t)blockIdx.x * a.d;
  if constexpr (kWarpRow) {
    __shared__ float sh[kNormWarps * NV * V * 32];
    if (a.part_pre) cta_columns<V, NV, SHIFT>(acc_pre, sh, a.part_pre + o, a.d, shift);
    if (a.part_s) cta_columns<V, NV, SHIFT>(acc_s, sh, a.part_s + o, a.d, shift);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (col(i) < a.d) {
        if (a.part_pre) store_f32<V, SHIFT>(a.part_pre + o, col(i), a.d, acc_pre[i]);
        if (a.part_s) store_f32<V, SHIFT>(a.part_s + o, col(i), a.d, acc_s[i]);
      }
  }
}

// Column totals of the partial sums, in a fixed order and 64 bits (in fp32 chains of 19 + 32 they
// gave most of the error: 1001 x 333, d_pre off by 1.4e-7 of its norm, 5e-8 now); the channel
// gate's gradient and the weight's after a block share one sum: d_gate = w_post S, d_post = gate S.
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
  __shared__ double sh[kNormRedRows][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  const float* part = blockIdx.y == 0 ? a.part_pre : a.part_s;
  if (!part) return;   // uniform over the CTA
  double sum = 0.0;
  if (c < a.d)
    for (int p = ty; p < a.parts; p += kNormRedRows) sum += (double)part[(int64_t)p * a.d + c];
  sh[ty][tx] = sum;
  __syncthreads();
  if (ty != 0 || c >= a.d) return;
  sum = 0.0;
#pragma unroll
  for (int q = 0; q < kNormRedRows; ++q) sum += sh[q][tx];
  const float v = (float)sum;
  if (blockIdx.y == 0) {
    a.d_pre[c] = v;
  } else {
    if (a.d_post) a.d_post[c] = a.gate_ch ? v * a.gate_ch[c] : v;
    if (a.d_gate) a.d_gate[c] = a.w_post ? v * a.w_post[c] : v;
  }
}

}  // namespace moe
