// op_common.cuh -- host-side checks shared by the entry points that have no handle: the
// current device, its SM count, and buffers that may not overlap.
#pragma once

#include <atomic>
#include <initializer_list>

#include "api_common.cuh"

namespace moe {

// SM count of the current device; fails unless it is sm_100.  (Attribute queries are allowed
// during stream capture; the count is kept per device.)
inline moe_status op_device(int* n_sms, int* device = nullptr) {
  static std::atomic<int> sms[64];   // 0: not asked yet
  int dev = 0;
  MOE_CUDA(cudaGetDevice(&dev));
  if (device) *device = dev;
  if (dev >= 0 && dev < 64 && sms[dev].load(std::memory_order_relaxed) > 0) {
    *n_sms = sms[dev].load(std::memory_order_relaxed);
    return MOE_OK;
  }
  int major = 0, minor = 0, n = 0;
  MOE_CUDA(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
  MOE_CUDA(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
  if (major != 10 || minor != 0)
    return fail(MOE_ERR_UNSUPPORTED, "this library is built for sm_100a (B200); device is sm_%d%d",
                major, minor);
  MOE_CUDA(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev));
  if (dev >= 0 && dev < 64) sms[dev].store(n, std::memory_order_relaxed);
  *n_sms = n;
  return MOE_OK;
}

// Whether [p, p + n) and [q, q + m) share a byte.
inline bool overlaps(const void* p, size_t n, const void* q, size_t m) {
  if (!p || !q || n == 0 || m == 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + m && b < a + n;
}

// A buffer a call reads or writes (nullptr or 0 bytes: none).
struct Span {
  const void* p;
  size_t n;
};
// Whether every output is apart from all inputs and from the outputs before it.
inline bool apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (overlaps(o->p, o->n, i.p, i.n)) return false;
    for (const Span* q = outs.begin(); q != o; ++q)
      if (overlaps(o->p, o->n, q->p, q->n)) return false;
  }
  return true;
}

inline bool misaligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

}  // namespace moe
