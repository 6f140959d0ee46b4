// Host helpers of the launch code: error status, device properties, shared-memory
// limits, alignment. Internal linkage: each translation unit has its own.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>
#include <unordered_map>

#include "status.h"

namespace {

using kvp::fail;

constexpr int kMaxDevices = 64;

int cuda_fail(cudaError_t e, const char* what) {
  return fail(KVP_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

int current_device() {
  int d = 0;
  cudaGetDevice(&d);
  return d;
}

int sm_count() {
  static std::atomic<int> cache[kMaxDevices];
  const int d = current_device();
  if (d < 0 || d >= kMaxDevices) return 148;
  int n = cache[d].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d);
    if (n <= 0) n = 148;
    cache[d].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Raises a kernel's dynamic shared-memory limit once per (kernel, device), so
// always to the same value.
template <typename K>
cudaError_t ensure_smem(K kernel, int bytes) {
  static std::mutex mu;
  static std::unordered_map<const void*, uint64_t> done;  // kernel -> device bit mask
  const int d = current_device();
  const uint64_t bit = d < 64 ? (1ull << d) : 0;
  const void* key = reinterpret_cast<const void*>(kernel);
  {
    std::lock_guard<std::mutex> g(mu);
    auto it = done.find(key);
    if (bit && it != done.end() && (it->second & bit)) return cudaSuccess;
  }
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit) {
    std::lock_guard<std::mutex> g(mu);
    done[key] |= bit;
  }
  return e;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int ilog2(int64_t v) {
  int l = 0;
  while ((int64_t(1) << l) < v) ++l;
  return (int64_t(1) << l) == v ? l : -1;
}

}  // namespace
