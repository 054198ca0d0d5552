// Host helpers of the layers' part of the C ABI: argument checks and the status
// of a launch. (The codecs' part, csrc/taco_abi.hip, has its own; both take
// tensors of up to 2^35 elements.)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "taco.h"

namespace taco {

// Largest tensor (rows * cols) a call accepts: 2^35 elements keeps every
// one-wave-per-tile grid under 2^32 threads.
constexpr int64_t kMaxElems = int64_t(1) << 35;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + (uintptr_t)nb && b0 < a0 + (uintptr_t)na;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? TACO_OK : TACO_ERR_HIP; }

// A launch's status is read with hipGetLastError afterwards, so drop any error an
// earlier, unrelated runtime call on this thread left behind.
inline void clear_stale_error() { (void)hipGetLastError(); }

}  // namespace taco
