// What a kernel has to be told once on every device before its first launch there
// (host side).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include <atomic>

namespace nvfp4 {

// A function attribute holds on the device that was current when it was set.  Runs f,
// which may be repeated, on each device's first call, and again after it failed;
// `done` has a bit per device (devices from 64 on, and none, run f every time).
template <typename F>
hipError_t once_per_device(std::atomic<uint64_t>& done, F&& f) {
  int dev = 0;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return hipSuccess;
  const hipError_t r = f();
  if (r == hipSuccess) done.fetch_or(bit, std::memory_order_release);
  return r;
}

// Allows kernels `bytes` of dynamic LDS, which beyond 64 KB they have to be: a kernel's most,
// whatever a call takes, so that none takes away what a call of another host thread is
// about to launch with.
template <typename... K>
hipError_t allow_lds(std::atomic<uint64_t>& done, int bytes, K*... kernels) {
  return once_per_device(done, [&] {
    hipError_t e = hipSuccess;
    auto allow = [&](const void* f) {
      if (e == hipSuccess) e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    };
    (allow(reinterpret_cast<const void*>(kernels)), ...);
    return e;
  });
}

}  // namespace nvfp4
