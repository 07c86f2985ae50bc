// grouped_tc.cuh -- what the tensor-core products of grouped_rows.cuh and grouped_wgrad.cuh share:
// operand tiles that are read where they lie, without transposed copies.  An operand whose
// contraction index is contiguous arrives as a K-major tile; one whose output index is (W of
// dgrad, dy and x of wgrad) as an MN-major tile -- boxes of 64 output indices x contraction
// rows, 128-byte swizzled, which the MMA reads through the descriptor's strides.
#pragma once

#include "gemm_tc.cuh"
#include "grouped_mm.cuh"

namespace moe {

// Error word of the grouped kernels on this device (moe_grouped_device_status).
static __device__ int g_grouped_err;

constexpr int kGpEpiWarps = 8;
constexpr int kGpThreads = 64 + 32 * kGpEpiWarps;

// MN-major tile of 64-element blocks, each a box of rows of 128 bytes (128-byte swizzle): leading
// offset = distance of two blocks (64 output columns: a box), stride offset = 8 contraction
// rows.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t box) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(box >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}
constexpr uint32_t kIdescAMn = 1u << 15, kIdescBMn = 1u << 16;   // A / B is MN-major

// mbar_wait whose acquire covers the writes of the peer CTA's threads.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                                  int* err, int code) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if ((it & 255u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        record_error(err, code);
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// Arrive on a barrier that hands no memory over (a tensor-memory accumulator that has been
// read into registers, a slot whose value has been used).  A releasing arrive would first wait
// for the thread's earlier global stores.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_relaxed_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

}  // namespace moe
