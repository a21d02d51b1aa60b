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

}  // namespace nvfp4
