// Activations of the linear layers and their derivatives, in fp32.  Comparisons are written so that
// NaN passes through (a maximum against zero would drop it).
#pragma once

#include <hip/hip_runtime.h>

namespace anvil {

enum Act { kActNone = 0, kActRelu = 1, kActRelu2 = 2, kActGelu = 3, kActSilu = 4 };

__device__ __forceinline__ float relu(float z) { return z < 0.0f ? 0.0f : z; }

// Standard normal distribution function.
__device__ __forceinline__ float normal_cdf(float z) {
  return 0.5f * erfcf(-0.70710678118654752f * z);
}

__device__ __forceinline__ float logistic(float z) { return 1.0f / (1.0f + __expf(-z)); }

__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case kActRelu: return relu(z);
    case kActRelu2: { const float r = relu(z); return r * r; }
    case kActGelu: return z * normal_cdf(z);
    case kActSilu: return z * logistic(z);
    default: return z;
  }
}

// d act / dz; 0 at z = 0 for the two rectifiers.
__device__ __forceinline__ float act_slope(int act, float z) {
  switch (act) {
    case kActRelu: return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    case kActRelu2: return 2.0f * relu(z);
    case kActGelu:
      return fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z), normal_cdf(z));
    case kActSilu: {
      const float s = logistic(z);
      return s * fmaf(z, 1.0f - s, 1.0f);
    }
    default: return 1.0f;
  }
}

// N values at once, the choice of the activation outside the loop.
template <int N>
__device__ __forceinline__ void activate(int act, float v[N]) {
  auto all = [&](auto f) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = f(v[e]);
  };
  switch (act) {
    case kActRelu: return all([](float z) { return act_value(kActRelu, z); });
    case kActRelu2: return all([](float z) { return act_value(kActRelu2, z); });
    case kActGelu: return all([](float z) { return act_value(kActGelu, z); });
    case kActSilu: return all([](float z) { return act_value(kActSilu, z); });
    default: return;
  }
}

// v[e] *= act'(z[e])
template <int N>
__device__ __forceinline__ void scale_by_slope(int act, const float z[N], float v[N]) {
  auto all = [&](auto f) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] *= f(z[e]);
  };
  switch (act) {
    case kActRelu: return all([](float x) { return act_slope(kActRelu, x); });
    case kActRelu2: return all([](float x) { return act_slope(kActRelu2, x); });
    case kActGelu: return all([](float x) { return act_slope(kActGelu, x); });
    case kActSilu: return all([](float x) { return act_slope(kActSilu, x); });
    default: return;
  }
}

}  // namespace anvil
