// C ABI of the AdamW step: the plan of a list of tensors, checked and laid out in host memory, and the
// step on its copy in device memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "../../include/anvil.h"
#include "adamw.h"
#include "api_common.h"

namespace {

using anvil::aligned;
using anvil::AdamwPiece;
using anvil::AdamwTensor;

constexpr int64_t kMostTensors = int64_t(1) << 20;
constexpr int64_t kMostElements = int64_t(1) << 40;   // of one tensor: pieces are numbered in 32 bits
constexpr int64_t kMostPieces = int64_t(1) << 31;

int64_t pieces_of(int64_t count) { return (count + anvil::kAdamwPiece - 1) / anvil::kAdamwPiece; }

int elem_bytes(int dtype) { return dtype == ANVIL_F32 ? 4 : 2; }
bool known(int dtype) { return dtype == ANVIL_F32 || dtype == ANVIL_BF16 || dtype == ANVIL_F16; }

int check_tensor(const anvil_adamw_tensor& t) {
  if (t.count < 0 || !known(t.param_dtype) || !known(t.grad_dtype) ||
      (t.state_bits != 8 && t.state_bits != 32) || (t.mantissa && t.param_dtype != ANVIL_BF16))
    return ANVIL_ERR_INVALID_ARG;
  if (t.count == 0) return ANVIL_OK;
  if (t.count > kMostElements) return ANVIL_ERR_UNSUPPORTED;
  if (!t.param || !t.grad || !t.m || !t.v || (t.state_bits == 8 && (!t.m_scale || !t.v_scale)))
    return ANVIL_ERR_INVALID_ARG;
  const int sb = t.state_bits / 8;
  if (!aligned(t.param, elem_bytes(t.param_dtype)) || !aligned(t.grad, elem_bytes(t.grad_dtype)) ||
      !aligned(t.mantissa, 2) || !aligned(t.m, sb) || !aligned(t.v, sb))
    return ANVIL_ERR_MISALIGNED;
  if (t.state_bits == 8 && (!aligned(t.m_scale, 4) || !aligned(t.v_scale, 4)))
    return ANVIL_ERR_MISALIGNED;
  return ANVIL_OK;
}

struct Span {
  uintptr_t begin, end;
  bool written;
};

// Whether anything that is written shares memory with anything else.
bool any_shared(std::vector<Span>& spans) {
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t end = 0, written_end = 0;   // of what begins no later than the span at hand
  for (const Span& s : spans) {
    if (s.begin < (s.written ? end : written_end)) return true;
    end = std::max(end, s.end);
    if (s.written) written_end = std::max(written_end, s.end);
  }
  return false;
}

int64_t count_pieces(const anvil_adamw_tensor* tensors, int64_t count) {
  int64_t pieces = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (tensors[i].count < 0 || tensors[i].count > kMostElements) return -1;
    pieces += pieces_of(tensors[i].count);
    if (pieces > kMostPieces) return -1;
  }
  return pieces;
}

int run(const void* plan, size_t plan_bytes, int64_t tensors, anvil::AdamwStep step, double beta1,
        double beta2, double eps, const float* grad_scale, void* stream) {
  if (tensors < 0 || tensors > kMostTensors || !(beta1 >= 0 && beta1 < 1) ||
      !(beta2 >= 0 && beta2 < 1) || !(eps >= 0))
    return ANVIL_ERR_INVALID_ARG;
  const size_t head = static_cast<size_t>(tensors) * sizeof(AdamwTensor);
  if (plan_bytes < head || (plan_bytes - head) % sizeof(AdamwPiece)) return ANVIL_ERR_INVALID_ARG;
  const int64_t pieces = static_cast<int64_t>((plan_bytes - head) / sizeof(AdamwPiece));
  if (pieces > kMostPieces) return ANVIL_ERR_INVALID_ARG;
  if (pieces == 0) return ANVIL_OK;
  if (!plan) return ANVIL_ERR_INVALID_ARG;
  if (!aligned(plan, 16) || !aligned(grad_scale, 4)) return ANVIL_ERR_MISALIGNED;
  step.beta1 = static_cast<float>(beta1);
  step.one_beta1 = static_cast<float>(1.0 - beta1);
  step.beta2 = static_cast<float>(beta2);
  step.one_beta2 = static_cast<float>(1.0 - beta2);
  step.eps = static_cast<float>(eps);
  step.grad_scale = grad_scale;
  return anvil::hip_status(anvil::launch_adamw(plan, tensors, pieces, step, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t anvil_adamw_plan_bytes(const anvil_adamw_tensor* tensors, int64_t count) {
  if (count <= 0 || count > kMostTensors || !tensors) return 0;
  const int64_t pieces = count_pieces(tensors, count);
  return pieces < 0 ? 0
                    : static_cast<size_t>(count) * sizeof(AdamwTensor) +
                          static_cast<size_t>(pieces) * sizeof(AdamwPiece);
}

int anvil_adamw_plan(const anvil_adamw_tensor* tensors, int64_t count, void* plan, size_t plan_bytes) {
  if (count < 0) return ANVIL_ERR_INVALID_ARG;
  if (count == 0) return ANVIL_OK;
  if (!tensors) return ANVIL_ERR_INVALID_ARG;
  if (count > kMostTensors) return ANVIL_ERR_UNSUPPORTED;
  for (int64_t i = 0; i < count; ++i) {
    const int st = check_tensor(tensors[i]);
    if (st != ANVIL_OK) return st;
  }
  const size_t need = anvil_adamw_plan_bytes(tensors, count);
  if (need == 0) return ANVIL_ERR_UNSUPPORTED;
  if (!plan) return ANVIL_ERR_INVALID_ARG;
  if (plan_bytes != need) return ANVIL_ERR_UNSUPPORTED;
  if (!aligned(plan, 8)) return ANVIL_ERR_MISALIGNED;
  try {
    std::vector<Span> spans;
    spans.reserve(static_cast<size_t>(count) * 7);
    auto add = [&](const void* p, int64_t bytes, bool written) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p);
      if (p && bytes > 0) spans.push_back({at, at + static_cast<uintptr_t>(bytes), written});
    };
    for (int64_t i = 0; i < count; ++i) {
      const anvil_adamw_tensor& t = tensors[i];
      const int64_t n = t.count, blocks = (n + anvil::kAdamwBlock - 1) / anvil::kAdamwBlock;
      add(t.param, n * elem_bytes(t.param_dtype), true);
      add(t.mantissa, n * 2, true);
      add(t.grad, n * elem_bytes(t.grad_dtype), false);
      add(t.m, n * (t.state_bits / 8), true);
      add(t.v, n * (t.state_bits / 8), true);
      if (t.state_bits == 8) {
        add(t.m_scale, blocks * 4, true);
        add(t.v_scale, blocks * 4, true);
      }
    }
    if (any_shared(spans)) return ANVIL_ERR_ALIAS;
  } catch (const std::bad_alloc&) {
    return ANVIL_ERR_OOM;
  }
  AdamwTensor* to = static_cast<AdamwTensor*>(plan);
  AdamwPiece* piece = reinterpret_cast<AdamwPiece*>(to + count);
  for (int64_t i = 0; i < count; ++i) {
    const anvil_adamw_tensor& t = tensors[i];
    to[i] = AdamwTensor{t.param, t.mantissa, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.count,
                        t.param_dtype, t.grad_dtype, t.lr_mul, t.wd_mul, t.state_bits, 0};
    const int64_t n = pieces_of(t.count);
    for (int64_t k = 0; k < n; ++k)
      *piece++ = AdamwPiece{static_cast<uint32_t>(i), static_cast<uint32_t>(k)};
  }
  return ANVIL_OK;
}

int anvil_adamw(const void* plan, size_t plan_bytes, int64_t tensors, float lr, double beta1,
                double beta2, double eps, float weight_decay, int64_t step, uint32_t seed,
                const float* grad_scale, void* stream) {
  if (step < 1) return ANVIL_ERR_INVALID_ARG;
  anvil::AdamwStep s{};
  s.lr = lr;
  s.wd = weight_decay;
  s.fix1 = static_cast<float>(1.0 / (1.0 - std::pow(beta1, static_cast<double>(step))));
  s.fix2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, static_cast<double>(step))));
  s.seed = seed;
  return run(plan, plan_bytes, tensors, s, beta1, beta2, eps, grad_scale, stream);
}

int anvil_adamw_dev(const void* plan, size_t plan_bytes, int64_t tensors, const float* scalars,
                    double beta1, double beta2, double eps, const float* grad_scale, void* stream) {
  if (!scalars) return ANVIL_ERR_INVALID_ARG;
  if (!aligned(scalars, 4)) return ANVIL_ERR_MISALIGNED;
  anvil::AdamwStep s{};
  s.device = scalars;
  return run(plan, plan_bytes, tensors, s, beta1, beta2, eps, grad_scale, stream);
}

}  // extern "C"
