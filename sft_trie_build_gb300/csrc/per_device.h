// Settings that belong to a device, made by the host once per device.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace stp {

// Runs `set` (a kernel's shared-memory limit, say) where the current device has
// not had it yet; one that failed is tried again by the next call.  Several
// threads may run it at the same time.
class PerDevice {
 public:
  template <typename F>
  cudaError_t operator()(F set) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool kept = dev >= 0 && dev < kMost;
    if (kept && done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = set();
    if (e != cudaSuccess)
      cudaGetLastError();   // reported here, not by the next launch
    else if (kept)
      done_[dev].store(true, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int kMost = 64;
  std::atomic<bool> done_[kMost] = {};
};

}  // namespace stp
