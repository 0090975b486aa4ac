// Host-side argument checks shared by the entry points (api.hip,
// api_attention.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "pq1.h"

namespace pq1 {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlaps(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + bn && b0 < a0 + an;
}

// PQ1_OK if the current device is a gfx950 (checked once per device); *cus is
// its compute-unit count.
pq1_status check_device(int* cus = nullptr);

// PQ1_OK, or PQ1_ERR_LAUNCH with the error kept for pq1_last_hip_error.
pq1_status launched(hipError_t e);

}  // namespace pq1
