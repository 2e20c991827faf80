// What launches of kernels with a large dynamic LDS share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace rs {

namespace {

// Lets KERNEL use `bytes` of dynamic LDS (past 64 KiB it has to be asked for, once per device).
template <typename K, K KERNEL>
hipError_t allow_lds(int bytes) {
  if (bytes <= 64 * 1024) return hipSuccess;
  static std::atomic<uint64_t> done{0};  // a bit per device
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(KERNEL), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace

}  // namespace rs
