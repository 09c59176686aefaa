// smem_once.cuh -- a kernel's leave to use more dynamic shared memory than the
// default.  Host code only.
#pragma once
#include <cuda_runtime.h>

#include <mutex>

namespace pararnn {

// One for each kernel: asks for the leave when a launch needs more than was
// asked for before on its device (a call of its own costs about a microsecond).
// Launches of one kernel come from several host threads with different sizes;
// the leave is set and recorded under a lock and never made smaller, so no
// launch finds less than is recorded.
struct SmemOnce {
  int allow(const void* kernel, int most) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return (int)e;
    if (dev >= kDevices) return (int)cudaErrorInvalidDevice;
    const std::lock_guard<std::mutex> hold(lock);
    if (bytes[dev] >= most) return 0;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess) bytes[dev] = most;
    return (int)e;
  }

 private:
  static constexpr int kDevices = 128;
  std::mutex lock;
  int bytes[kDevices] = {};
};

}  // namespace pararnn
