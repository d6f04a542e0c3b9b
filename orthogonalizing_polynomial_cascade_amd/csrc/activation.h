// Activations of the linear layers and their derivatives, in fp32.  Comparisons are written so that
// NaN passes through (a maximum against zero would drop it).
#pragma once

#include <hip/hip_runtime.h>

namespace anvil {

enum Act { kActNone = 0, kActRelu = 1, kActRelu2 = 2, kActGelu = 3, kActSilu = 4 };

__device__ __forceinline__ float relu(float z) { return z < 0.0f ? 0.0f : z; }

// exp(-z^2 / 2).
__device__ __forceinline__ float gauss(float z) {
  return __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z);   // log2(e) / 2
}

// Standard normal distribution function, given g = gauss(z).  With x = |z| / sqrt(2) and
// t = 1 / (1 + 0.4 x), exp(x^2) erfc(x) / t is smooth on 0 < t <= 1; the polynomial is its
// least-maximum fit of degree 8 (relative error 6e-8).  Evaluated in fp32 the tail erfc(x) / 2 is off by
// at most 5e-7 + 6e-8 z^2 of itself: the exponent -z^2 / 2 is rounded before the power is taken, so
// the error grows with it (4e-7 below |z| = 2, 2e-6 at 6, 8e-6 at 13), and the hardware's power and
// reciprocal add a step each.  A sixteen-bit result, whose half step is 4.9e-4 or more, rounds as the
// exact one but for the nearest ties.  A third of the
// instructions of the library's erfcf, which kept the epilogue of a 256x256 tile busy for longer
// than the multiplies of depth 768.
__device__ __forceinline__ float normal_cdf(float z, float g) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.28284271247461901f, fabsf(z), 1.0f));
  float r = 0.0412530415f;
  r = fmaf(r, t, -0.140319243f);
  r = fmaf(r, t, 0.0839872956f);
  r = fmaf(r, t, 0.0879643261f);
  r = fmaf(r, t, 0.0797564983f);
  r = fmaf(r, t, 0.193393201f);
  r = fmaf(r, t, 0.201887593f);
  r = fmaf(r, t, 0.226443112f);
  r = fmaf(r, t, 0.225634232f);
  const float upper = 0.5f * t * r * g;
  return z < 0.0f ? upper : 1.0f - upper;
}

// 1 / (1 + exp(-z)), the reciprocal within one step of fp32.
__device__ __forceinline__ float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case kActRelu: return relu(z);
    case kActRelu2: { const float r = relu(z); return r * r; }
    case kActGelu: return z * normal_cdf(z, gauss(z));
    case kActSilu: return z * logistic(z);
    default: return z;
  }
}

// d act / dz; 0 at z = 0 for the two rectifiers.
__device__ __forceinline__ float act_slope(int act, float z) {
  switch (act) {
    case kActRelu: return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    case kActRelu2: return 2.0f * relu(z);
    case kActGelu: {
      const float g = gauss(z);
      return fmaf(z * 0.39894228040143268f, g, normal_cdf(z, g));
    }
    case kActSilu: {
      const float s = logistic(z);
      return s * fmaf(z, 1.0f - s, 1.0f);
    }
    default: return 1.0f;
  }
}

}  // namespace anvil
