// C ABI of the linear head's cross entropy.  Argument checks and launches; nothing is allocated,
// synchronised or read back here, so every call may be captured into a HIP graph.
#include <hip/hip_runtime.h>

#include "api_views.h"
#include "cross_entropy.h"

namespace {

using anvil::aligned;
using anvil::check_views;
using anvil::dense;
using anvil::elem_bytes;

int check_head(int dtype, int w_kn, int target_bits, int64_t rows, int64_t vocab, int64_t k) {
  if (dtype != ANVIL_BF16 && dtype != ANVIL_F16)
    return anvil::elem_known(dtype) ? ANVIL_ERR_UNSUPPORTED : ANVIL_ERR_INVALID_ARG;
  if ((w_kn != 0 && w_kn != 1) || (target_bits != 32 && target_bits != 64)) return ANVIL_ERR_INVALID_ARG;
  if (rows < 0 || vocab < 1 || k < 0) return ANVIL_ERR_INVALID_ARG;
  // Offsets within a tile depend on widths and pitches alone and addresses are 64-bit: the bounds on the products
  // keep their tiles within a launch's grid (2^31 weights: 2^17 tiles of dw) and the workspace within memory.
  if (rows > (int64_t(1) << 22) || vocab > anvil::kMaxWidth || k > anvil::kMaxWidth ||
      vocab * k >= (int64_t(1) << 31) || rows * vocab > (int64_t(1) << 37) ||
      rows * k > (int64_t(1) << 37))
    return ANVIL_ERR_UNSUPPORTED;
  return ANVIL_OK;
}

// Which of x and w the kernels read where they lie.
int in_place_of(const void* x, int64_t ldx, const void* w) {
  return (aligned(x, 16) && ldx % 8 == 0 ? ANVIL_X_IN_PLACE : 0) |
         (aligned(w, 16) ? ANVIL_W_IN_PLACE : 0);
}

int check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return ANVIL_OK;
  if (!workspace) return ANVIL_ERR_INVALID_ARG;
  if (bytes < need) return ANVIL_ERR_UNSUPPORTED;
  return aligned(workspace, 256) ? ANVIL_OK : ANVIL_ERR_MISALIGNED;
}

}  // namespace

extern "C" {

size_t anvil_cross_entropy_workspace(int w_kn, int in_place, int64_t rows, int64_t vocab, int64_t k) {
  if (check_head(ANVIL_BF16, w_kn, 32, rows, vocab, k) != ANVIL_OK || rows == 0) return 0;
  return anvil::head_plan(false, false, false, w_kn != 0, false, in_place, rows, vocab, k).bytes;
}

int anvil_cross_entropy(const void* x, int64_t ldx, const void* w, int w_kn, const void* targets,
                        int target_bits, float* loss, float* lse, int dtype, int64_t rows,
                        int64_t vocab, int64_t k, void* workspace, size_t workspace_bytes,
                        void* stream) {
  int st = check_head(dtype, w_kn, target_bits, rows, vocab, k);
  if (st != ANVIL_OK) return st;
  if (rows == 0) return ANVIL_OK;
  if (!targets || !loss || !lse || (k > 0 && (!x || !w))) return ANVIL_ERR_INVALID_ARG;
  if (!anvil::take_pitch(x, &ldx, k, rows)) return ANVIL_ERR_UNSUPPORTED;
  if (!aligned(x, 2) || !aligned(w, 2) || !aligned(targets, target_bits / 8) || !aligned(loss, 4) ||
      !aligned(lse, 4))
    return ANVIL_ERR_MISALIGNED;
  const int in_place = in_place_of(x, ldx, w);
  const size_t need =
      anvil::head_plan(false, false, false, w_kn != 0, dtype == ANVIL_F16, in_place, rows, vocab, k).bytes;
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != ANVIL_OK) return st;
  st = check_views({{x, rows, k * 2, ldx * 2, false},
                    dense(w, vocab * k * 2, false),
                    dense(targets, rows * (target_bits / 8), false),
                    dense(loss, rows * 4, true),
                    dense(lse, rows * 4, true),
                    dense(need ? workspace : nullptr, need, true)});
  if (st != ANVIL_OK) return st;
  anvil::HeadCall a{};
  a.x = x; a.ldx = ldx; a.w = w; a.w_kn = w_kn != 0; a.f16 = dtype == ANVIL_F16;
  a.in_place = in_place;
  a.rows = rows; a.vocab = vocab; a.depth = static_cast<int>(k);
  a.targets = targets; a.wide = target_bits == 64;
  a.loss = loss; a.lse = lse;
  return anvil::hip_status(anvil::launch_cross_entropy(a, static_cast<char*>(workspace),
                                                       static_cast<hipStream_t>(stream)));
}

size_t anvil_cross_entropy_grad_workspace(int want_dx, int want_dw, int w_kn, int in_place, int dtype,
                                          int64_t rows, int64_t vocab, int64_t k) {
  if (check_head(dtype, w_kn, 32, rows, vocab, k) != ANVIL_OK || rows == 0 || k == 0 ||
      (!want_dx && !want_dw))
    return 0;
  return anvil::head_plan(true, want_dx != 0, want_dw != 0, w_kn != 0, dtype == ANVIL_F16,
                          in_place, rows, vocab, k).bytes;
}

int anvil_cross_entropy_grad(const void* x, int64_t ldx, const void* w, int w_kn, const void* targets,
                             int target_bits, const float* lse, const float* dloss, void* dx,
                             int64_t lddx, void* dw, int dw_dtype, int dtype, int64_t rows,
                             int64_t vocab, int64_t k, void* workspace, size_t workspace_bytes,
                             void* stream) {
  int st = check_head(dtype, w_kn, target_bits, rows, vocab, k);
  if (st != ANVIL_OK) return st;
  if (dw && dw_dtype != ANVIL_F32 && dw_dtype != dtype) return ANVIL_ERR_INVALID_ARG;
  if (k == 0 || (!dx && !dw)) return ANVIL_OK;
  if (rows > 0 && (!x || !w || !targets || !lse || !dloss)) return ANVIL_ERR_INVALID_ARG;
  if (!anvil::take_pitch(x, &ldx, k, rows) || !anvil::take_pitch(dx, &lddx, k, rows))
    return ANVIL_ERR_UNSUPPORTED;
  const int wb = dw ? elem_bytes(dw_dtype) : 1;
  if (!aligned(x, 2) || !aligned(w, 2) || !aligned(targets, target_bits / 8) || !aligned(lse, 4) ||
      !aligned(dloss, 4) || !aligned(dx, 2) || !aligned(dw, wb))
    return ANVIL_ERR_MISALIGNED;
  const int in_place = in_place_of(x, ldx, w);
  const size_t need =
      rows == 0 ? 0
                : anvil::head_plan(true, dx != nullptr, dw != nullptr, w_kn != 0, dtype == ANVIL_F16,
                                   in_place, rows, vocab, k).bytes;
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != ANVIL_OK) return st;
  st = check_views({{x, rows, k * 2, ldx * 2, false},
                    dense(w, vocab * k * 2, false),
                    dense(targets, rows * (target_bits / 8), false),
                    dense(lse, rows * 4, false),
                    dense(dloss, rows * 4, false),
                    {dx, rows, k * 2, lddx * 2, true},
                    dense(dw, dw ? vocab * k * wb : 0, true),
                    dense(need ? workspace : nullptr, need, true)});
  if (st != ANVIL_OK) return st;
  anvil::HeadCall a{};
  a.x = x; a.ldx = ldx; a.w = w; a.w_kn = w_kn != 0; a.f16 = dtype == ANVIL_F16;
  a.in_place = in_place;
  a.rows = rows; a.vocab = vocab; a.depth = static_cast<int>(k);
  a.targets = targets; a.wide = target_bits == 64;
  a.lse = const_cast<float*>(lse); a.dloss = dloss;
  a.dx = rows ? dx : nullptr; a.lddx = lddx;
  a.dw = dw; a.dw_f32 = dw_dtype == ANVIL_F32;
  return anvil::hip_status(anvil::launch_cross_entropy_grad(a, static_cast<char*>(workspace),
                                                            static_cast<hipStream_t>(stream)));
}

}  // extern "C"
