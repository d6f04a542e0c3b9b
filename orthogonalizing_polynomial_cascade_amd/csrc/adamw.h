// The AdamW step: its plan in device memory and its launch.
#pragma once

#include "launchers.h"

namespace anvil {

constexpr int kAdamwPiece = 2048;   // elements of one workgroup
constexpr int kAdamwBlock = 256;    // elements that share a scale

// A plan is `tensors` of these and then its pieces.
struct AdamwTensor {
  void* param;
  uint16_t* mantissa;    // or null
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t count;
  int param_type, grad_type;
  float lr_mul, wd_mul;
  int state_bits;        // 32 or 8
  int pad;
};
static_assert(sizeof(AdamwTensor) == 88, "the plan's size");
struct AdamwPiece {
  uint32_t tensor, index;
};

struct AdamwStep {
  float lr, wd, beta1, one_beta1, beta2, one_beta2, eps, fix1, fix2;
  uint32_t seed;
  const float* device;       // values in place of some of these, or null
  const float* grad_scale;   // or null
};
hipError_t launch_adamw(const void* plan, int64_t tensors, int64_t pieces, const AdamwStep& step,
                        hipStream_t stream);

}  // namespace anvil
