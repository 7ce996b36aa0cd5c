// The dynamic shared memory that kernels are allowed, which launches ask for from any host thread.
#pragma once

#include <atomic>
#include <mutex>

#include "bskv.h"

namespace bskv {

// Calls set(bytes), which allows one kernel on one device that much and replaces what it was allowed,
// unless `allowed` says that it has as much. Calls run one after another and never lower the amount: a
// launch that was allowed its size stays so whatever other threads ask for.
template <typename Set>
bskv_status raise_smem_limit(std::atomic<int>& allowed, std::mutex& mu, int bytes, Set set) {
  if (allowed.load(std::memory_order_acquire) >= bytes) return BSKV_OK;
  std::lock_guard<std::mutex> lock(mu);
  if (allowed.load(std::memory_order_relaxed) >= bytes) return BSKV_OK;
  if (bskv_status s = set(bytes)) return s;
  allowed.store(bytes, std::memory_order_release);
  return BSKV_OK;
}

}  // namespace bskv
