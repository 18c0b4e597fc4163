// kda_device.cuh -- what launches keep about the devices they go to.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace kda {

// A positive number that belongs to a device (a kernel's resident CTAs, the
// number of SMs), found once for each: a process may call the library on several,
// and a kernel's shared-memory limit has to be set on every one of them. `find`
// makes the settings on the current device and gives the number. A failure is
// returned and not kept: the next call tries again.
class PerDevice {
 public:
  template <typename F>
  cudaError_t get(int64_t* value, const F& find) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) {
      const bool keep = dev >= 0 && dev < kDevices;
      *value = keep ? kept_[dev].load(std::memory_order_relaxed) : 0;
      if (*value > 0) return cudaSuccess;
      e = find(dev, value);
      if (e == cudaSuccess && keep) kept_[dev].store(*value, std::memory_order_relaxed);
    }
    if (e != cudaSuccess) cudaGetLastError();  // returned here, not to a later call
    return e;
  }

 private:
  static constexpr int kDevices = 64;  // beyond these it is found on every call
  std::atomic<int64_t> kept_[kDevices] = {};
};

}  // namespace kda
