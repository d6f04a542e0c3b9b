// Pieces of the C ABI shared by api.hip (bank step) and train_api.hip (training operators).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace anvil {

// ANVIL_OK, or ANVIL_ERR_HIP with the error kept for anvil_last_hip_error.
int hip_status(hipError_t e);

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na && nb && x < y + nb && y < x + na;
}

}  // namespace anvil
