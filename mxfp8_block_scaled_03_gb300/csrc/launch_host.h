// launch_host.h -- what the host side of the decode operators and of the cross entropy needs: the tensor-map encoder and the
// limit of pipeline waits.  (grouped_gemm.cu has its own: counters are kept for its code as it is.)
#pragma once
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstdlib>

namespace mx {

// The driver's entry point, fetched at run time; nullptr where there is none (asked again by the next call).
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::atomic<void*> entry{nullptr};
  void* fn = entry.load(std::memory_order_acquire);
  if (fn == nullptr) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    entry.store(fn, std::memory_order_release);
  }
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
}

// Limit of every pipeline wait: 2 s, or the value in ns of the environment variable
// MXFP8MOE_WAIT_LIMIT_NS when it holds a positive integer (read at each call; failure-path tests
// use it to make waits run out without any change to the kernels).  Teardown waits for copies and
// MMAs in flight always keep the full 2 s.
constexpr uint64_t kWaitTimeoutNs = 2000000000ull;
inline uint64_t pipeline_wait_ns() {
  const char* v = getenv("MXFP8MOE_WAIT_LIMIT_NS");
  if (v == nullptr || *v == 0) return kWaitTimeoutNs;
  char* end = nullptr;
  const unsigned long long n = strtoull(v, &end, 10);
  return (end != nullptr && *end == 0 && n > 0) ? static_cast<uint64_t>(n) : kWaitTimeoutNs;
}

}  // namespace mx
