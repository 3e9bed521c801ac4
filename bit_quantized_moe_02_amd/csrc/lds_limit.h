// A kernel's limit of dynamic LDS, for the step kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <mutex>
#include <set>
#include <utility>

namespace qmoe {

// Raises a kernel's dynamic-LDS limit to the device maximum less what it
// declares (`declared` bytes at most), once per kernel and device: each device
// has a limit of its own (an upper bound, the launch passes the size).
inline hipError_t raise_dyn_lds(const void* fn, int declared) {
  static std::mutex mu;
  static std::set<std::pair<int, const void*>> done;
  std::lock_guard<std::mutex> lock(mu);
  int dev = 0, max_lds = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess && done.count({dev, fn})) return hipSuccess;
  if (e == hipSuccess) e = hipDeviceGetAttribute(&max_lds, hipDeviceAttributeMaxSharedMemoryPerBlock, dev);
  if (e == hipSuccess) e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, max_lds - declared);
  if (e == hipSuccess) done.insert({dev, fn});
  return e;
}

}  // namespace qmoe
