// Element types of the training operators: conversions to and from fp32, and accesses of several
// consecutive elements at any element alignment.
#pragma once

#include "device_common.h"

namespace anvil {

typedef __bf16 bf16;
typedef _Float16 f16;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16 v) {
  return bf16_to_f32(__builtin_bit_cast(uint16_t, v));
}
__device__ __forceinline__ float to_f32(f16 v) { return static_cast<float>(v); }

// Round to nearest even.
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  return static_cast<T>(v);
}

// N consecutive elements, in accesses of up to 16 bytes: gfx950 takes global addresses of any
// alignment, so rows that start at odd elements need no path of their own.
template <typename T, int N>
__device__ __forceinline__ void load_vec(const T* p, float v[N]) {
  T t[N];
  __builtin_memcpy(t, p, sizeof(t));
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = to_f32(t[e]);
}

template <typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const float v[N]) {
  T t[N];
#pragma unroll
  for (int e = 0; e < N; ++e) t[e] = from_f32<T>(v[e]);
  __builtin_memcpy(p, t, sizeof(t));
}

}  // namespace anvil
