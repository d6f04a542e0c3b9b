// C ABI of the training operators around a bank: layer norm, linear layers and the linear layers
// of a stack of experts, each with its backward pass.  Argument checks and launches; nothing is
// allocated, synchronised or read back here, so every call may be captured into a HIP graph.
#include <hip/hip_runtime.h>

#include "../../include/anvil.h"
#include "api_views.h"
#include "launchers.h"

namespace {

using anvil::aligned;
using anvil::check_views;
using anvil::dense;
using anvil::elem_bytes;
using anvil::elem_known;
using anvil::hip_status;
using anvil::kMaxRows;
using anvil::kMaxWidth;
using anvil::take_pitch;
using anvil::View;

// ------------------------------------------------------------------------------------------
// Linear layers
// ------------------------------------------------------------------------------------------

struct GroupIn {
  const void* offsets;
  int bits;
  int64_t count;
};

// Sizes and flags shared by the linear entry points.
int check_sizes(int dtype, const GroupIn& g, bool grouped, int64_t rows, int64_t n, int64_t k) {
  if (dtype != ANVIL_BF16 && dtype != ANVIL_F16)
    return elem_known(dtype) ? ANVIL_ERR_UNSUPPORTED : ANVIL_ERR_INVALID_ARG;
  if (rows < 0 || n < 0 || k < 0 || g.count < 0) return ANVIL_ERR_INVALID_ARG;
  if (grouped && g.bits != 32 && g.bits != 64) return ANVIL_ERR_INVALID_ARG;
  if (rows >= kMaxRows || n > kMaxWidth || k > kMaxWidth || n * k > (int64_t(1) << 30) ||
      g.count > 65535 || g.count * n * k > (int64_t(1) << 35))
    return ANVIL_ERR_UNSUPPORTED;
  if (grouped && !aligned(g.offsets, g.bits / 8)) return ANVIL_ERR_MISALIGNED;
  return ANVIL_OK;
}

View offsets_view(const GroupIn& g) {
  return dense(g.offsets, g.offsets ? (g.count + 1) * (g.bits / 8) : 0, false);
}

anvil::Groups groups_of(const GroupIn& g, bool grouped) {
  return {grouped ? g.offsets : nullptr, g.bits == 64, static_cast<int>(grouped ? g.count : 1)};
}

bool act_known(int act) { return act >= ANVIL_ACT_NONE && act <= ANVIL_ACT_SILU; }

int rows_forward(const void* x, int64_t ldx, const void* w, int w_kn, const GroupIn& g,
                 bool grouped, const void* bias, int bias_dtype, int act, const void* residual,
                 int64_t ldr, void* y, int64_t ldy, void* preact, int64_t ldz, int dtype,
                 int64_t rows, int64_t n, int64_t k, void* stream) {
  int st = check_sizes(dtype, g, grouped, rows, n, k);
  if (st != ANVIL_OK) return st;
  if ((w_kn != 0 && w_kn != 1) || !act_known(act)) return ANVIL_ERR_INVALID_ARG;
  if (bias && bias_dtype != ANVIL_F32 && bias_dtype != dtype) return ANVIL_ERR_INVALID_ARG;
  if (rows == 0 || n == 0) return ANVIL_OK;
  const int64_t count = grouped ? g.count : 1;
  if (grouped && !g.offsets) return ANVIL_ERR_INVALID_ARG;
  if (!y || (k > 0 && !x) || (k > 0 && count > 0 && !w)) return ANVIL_ERR_INVALID_ARG;
  if (!take_pitch(x, &ldx, k, rows) || !take_pitch(y, &ldy, n, rows) ||
      !take_pitch(preact, &ldz, n, rows) || !take_pitch(residual, &ldr, n, rows))
    return ANVIL_ERR_UNSUPPORTED;
  const int eb = elem_bytes(dtype);
  if (!aligned(x, eb) || !aligned(w, eb) || !aligned(y, eb) || !aligned(preact, eb) ||
      !aligned(residual, eb) || !aligned(bias, bias ? elem_bytes(bias_dtype) : 1))
    return ANVIL_ERR_MISALIGNED;
  st = check_views({{x, rows, k * eb, ldx * eb, false},
                    dense(w, count * n * k * eb, false),
                    dense(bias, bias ? count * n * elem_bytes(bias_dtype) : 0, false),
                    {residual, rows, n * eb, ldr * eb, false},
                    {y, rows, n * eb, ldy * eb, true},
                    {preact, rows, n * eb, ldz * eb, true},
                    offsets_view(g)});
  if (st != ANVIL_OK) return st;
  anvil::RowsProduct a{};
  a.a = x; a.lda = ldx; a.b = w; a.b_kmajor = w_kn != 0;
  a.rows = rows; a.cols = static_cast<int>(n); a.depth = static_cast<int>(k);
  a.groups = groups_of(g, grouped);
  a.f16 = dtype == ANVIL_F16;
  a.act = act;
  a.bias = bias; a.bias_f32 = bias && bias_dtype == ANVIL_F32;
  a.add = residual; a.ldadd = ldr;
  a.keep = preact; a.ldkeep = ldz;
  a.out = y; a.ldout = ldy;
  return hip_status(anvil::launch_rows_product(a, static_cast<hipStream_t>(stream)));
}

int rows_backward(const void* dz, int64_t lddz, const void* w, int w_kn, const GroupIn& g,
                  bool grouped, const void* preact, int64_t ldz, int act, const void* add,
                  int64_t ldadd, void* dx, int64_t lddx, int dtype, int64_t rows, int64_t n,
                  int64_t k, void* stream) {
  int st = check_sizes(dtype, g, grouped, rows, n, k);
  if (st != ANVIL_OK) return st;
  if ((w_kn != 0 && w_kn != 1) || !act_known(act)) return ANVIL_ERR_INVALID_ARG;
  if (rows == 0 || k == 0) return ANVIL_OK;
  const int64_t count = grouped ? g.count : 1;
  if (grouped && !g.offsets) return ANVIL_ERR_INVALID_ARG;
  if (!dx || (n > 0 && !dz) || (n > 0 && count > 0 && !w)) return ANVIL_ERR_INVALID_ARG;
  if (act != ANVIL_ACT_NONE && !preact) return ANVIL_ERR_INVALID_ARG;
  if (!take_pitch(dz, &lddz, n, rows) || !take_pitch(dx, &lddx, k, rows) ||
      !take_pitch(preact, &ldz, k, rows) || !take_pitch(add, &ldadd, k, rows))
    return ANVIL_ERR_UNSUPPORTED;
  const int eb = elem_bytes(dtype);
  if (!aligned(dz, eb) || !aligned(w, eb) || !aligned(dx, eb) || !aligned(preact, eb) ||
      !aligned(add, eb))
    return ANVIL_ERR_MISALIGNED;
  if (act == ANVIL_ACT_NONE) preact = nullptr;   // its derivative is 1: not read
  st = check_views({{dz, rows, n * eb, lddz * eb, false},
                    dense(w, count * n * k * eb, false),
                    {preact, rows, k * eb, ldz * eb, false},
                    {add, rows, k * eb, ldadd * eb, false},
                    {dx, rows, k * eb, lddx * eb, true},
                    offsets_view(g)});
  if (st != ANVIL_OK) return st;
  anvil::RowsProduct a{};
  // dx[r][c] = sum_d dz[r][d] w(d, c): w stored [n][k] runs down its rows with d = n
  a.a = dz; a.lda = lddz; a.b = w; a.b_kmajor = w_kn == 0;
  a.rows = rows; a.cols = static_cast<int>(k); a.depth = static_cast<int>(n);
  a.groups = groups_of(g, grouped);
  a.f16 = dtype == ANVIL_F16;
  a.gradient = true;
  a.act = act;
  a.aux = preact; a.ldaux = ldz;
  a.add = add; a.ldadd = ldadd;
  a.out = dx; a.ldout = lddx;
  return hip_status(anvil::launch_rows_product(a, static_cast<hipStream_t>(stream)));
}

anvil::WeightProduct weight_product(const void* dz, int64_t lddz, const void* x, int64_t ldx,
                                    int w_kn, const anvil::Groups& groups, int dtype, int64_t rows,
                                    int64_t n, int64_t k) {
  anvil::WeightProduct a{};
  a.rows = rows;
  a.groups = groups;
  a.f16 = dtype == ANVIL_F16;
  a.dz_is_q = w_kn != 0;
  if (w_kn) {   // dw [k][n] = x^T dz
    a.p = x; a.ldp = ldx; a.pi = static_cast<int>(k);
    a.q = dz; a.ldq = lddz; a.qj = static_cast<int>(n);
  } else {      // dw [n][k] = dz^T x
    a.p = dz; a.ldp = lddz; a.pi = static_cast<int>(n);
    a.q = x; a.ldq = ldx; a.qj = static_cast<int>(k);
  }
  return a;
}

size_t weight_workspace(int w_kn, int64_t rows, int64_t n, int64_t k, int64_t experts) {
  const GroupIn g{nullptr, 32, experts};
  if (check_sizes(ANVIL_BF16, g, false, rows, n, k) != ANVIL_OK || n == 0 || k == 0 || experts == 0)
    return 0;
  const anvil::Groups groups{nullptr, false, static_cast<int>(experts)};
  return anvil::weight_product_words(
             weight_product(nullptr, 0, nullptr, 0, w_kn, groups, ANVIL_BF16, rows, n, k)) * 4;
}

int weight_backward(const void* dz, int64_t lddz, const void* x, int64_t ldx, int w_kn,
                    const GroupIn& g, bool grouped, void* dw, int dw_dtype, float* dbias, int dtype,
                    int64_t rows, int64_t n, int64_t k, void* workspace, size_t workspace_bytes,
                    void* stream) {
  int st = check_sizes(dtype, g, grouped, rows, n, k);
  if (st != ANVIL_OK) return st;
  if (w_kn != 0 && w_kn != 1) return ANVIL_ERR_INVALID_ARG;
  if (dw_dtype != ANVIL_F32 && dw_dtype != dtype) return ANVIL_ERR_INVALID_ARG;
  const int64_t count = grouped ? g.count : 1;
  if (n == 0 || k == 0 || count == 0) return ANVIL_OK;
  if (grouped && !g.offsets) return ANVIL_ERR_INVALID_ARG;
  if (!dw || (rows > 0 && (!dz || !x))) return ANVIL_ERR_INVALID_ARG;
  if (!take_pitch(dz, &lddz, n, rows) || !take_pitch(x, &ldx, k, rows)) return ANVIL_ERR_UNSUPPORTED;
  const int eb = elem_bytes(dtype), wb = elem_bytes(dw_dtype);
  if (!aligned(dz, eb) || !aligned(x, eb) || !aligned(dw, wb) || !aligned(dbias, 4))
    return ANVIL_ERR_MISALIGNED;
  const size_t need = weight_workspace(w_kn, rows, n, k, count);
  if (need) {
    if (!workspace) return ANVIL_ERR_INVALID_ARG;
    if (workspace_bytes < need) return ANVIL_ERR_UNSUPPORTED;
    if (!aligned(workspace, 256)) return ANVIL_ERR_MISALIGNED;
  }
  st = check_views({{dz, rows, n * eb, lddz * eb, false},
                    {x, rows, k * eb, ldx * eb, false},
                    dense(dw, count * n * k * wb, true),
                    dense(dbias, dbias ? count * n * 4 : 0, true),
                    dense(need ? workspace : nullptr, need, true),
                    offsets_view(g)});
  if (st != ANVIL_OK) return st;
  anvil::WeightProduct a =
      weight_product(dz, lddz, x, ldx, w_kn, groups_of(g, grouped), dtype, rows, n, k);
  a.dw = dw;
  a.dw_f32 = dw_dtype == ANVIL_F32;
  a.db = dbias;
  return hip_status(anvil::launch_weight_product(a, static_cast<float*>(workspace),
                                                 static_cast<hipStream_t>(stream)));
}

// Gated linear layers: n columns of h, 2 n of the weight and of z.
int gated_forward(const void* x, int64_t ldx, const void* w, int w_kn, const GroupIn& g,
                  bool grouped, const void* bias, int bias_dtype, int act, void* y, int64_t ldy,
                  void* preact, int64_t ldz, int dtype, int64_t rows, int64_t n, int64_t k,
                  void* stream) {
  if (n > kMaxWidth / 2) return ANVIL_ERR_UNSUPPORTED;
  int st = check_sizes(dtype, g, grouped, rows, n < 0 ? n : 2 * n, k);
  if (st != ANVIL_OK) return st;
  if ((w_kn != 0 && w_kn != 1) || !act_known(act)) return ANVIL_ERR_INVALID_ARG;
  if (bias && bias_dtype != ANVIL_F32 && bias_dtype != dtype) return ANVIL_ERR_INVALID_ARG;
  if (rows == 0 || n == 0) return ANVIL_OK;
  const int64_t count = grouped ? g.count : 1;
  if (grouped && !g.offsets) return ANVIL_ERR_INVALID_ARG;
  if (!y || (k > 0 && !x) || (k > 0 && count > 0 && !w)) return ANVIL_ERR_INVALID_ARG;
  if (!take_pitch(x, &ldx, k, rows) || !take_pitch(y, &ldy, n, rows) ||
      !take_pitch(preact, &ldz, 2 * n, rows))
    return ANVIL_ERR_UNSUPPORTED;
  const int eb = elem_bytes(dtype);
  if (!aligned(x, eb) || !aligned(w, eb) || !aligned(y, eb) || !aligned(preact, eb) ||
      !aligned(bias, bias ? elem_bytes(bias_dtype) : 1))
    return ANVIL_ERR_MISALIGNED;
  st = check_views({{x, rows, k * eb, ldx * eb, false},
                    dense(w, count * 2 * n * k * eb, false),
                    dense(bias, bias ? count * 2 * n * elem_bytes(bias_dtype) : 0, false),
                    {y, rows, n * eb, ldy * eb, true},
                    {preact, rows, 2 * n * eb, ldz * eb, true},
                    offsets_view(g)});
  if (st != ANVIL_OK) return st;
  anvil::RowsProduct a{};
  a.a = x; a.lda = ldx; a.b = w; a.b_kmajor = w_kn != 0;
  a.rows = rows; a.cols = static_cast<int>(n); a.depth = static_cast<int>(k);
  a.groups = groups_of(g, grouped);
  a.f16 = dtype == ANVIL_F16;
  a.act = act;
  a.bias = bias; a.bias_f32 = bias && bias_dtype == ANVIL_F32;
  a.keep = preact; a.ldkeep = ldz;
  a.out = y; a.ldout = ldy;
  return hip_status(anvil::launch_gated_product(a, static_cast<hipStream_t>(stream)));
}

// dz [rows][2 k] from dy [rows][n] of the layer w that h [rows][k] feeds, or (no w) from dh itself.
int gated_backward(const void* dy, int64_t lddy, const void* w, bool has_w, int w_kn,
                   const GroupIn& g, bool grouped, const void* preact, int64_t ldz, int act,
                   void* dz, int64_t lddz, int dtype, int64_t rows, int64_t n, int64_t k,
                   void* stream) {
  if (k > kMaxWidth / 2) return ANVIL_ERR_UNSUPPORTED;
  int st = check_sizes(dtype, g, grouped, rows, has_w ? n : 0, k);
  if (st != ANVIL_OK) return st;
  if ((w_kn != 0 && w_kn != 1) || !act_known(act)) return ANVIL_ERR_INVALID_ARG;
  if (rows == 0 || k == 0) return ANVIL_OK;
  const int64_t count = grouped ? g.count : 1;
  if (grouped && !g.offsets) return ANVIL_ERR_INVALID_ARG;
  if (!dz || !preact || (n > 0 && !dy) || (has_w && n > 0 && count > 0 && !w))
    return ANVIL_ERR_INVALID_ARG;
  if (!take_pitch(dy, &lddy, n, rows) || !take_pitch(dz, &lddz, 2 * k, rows) ||
      !take_pitch(preact, &ldz, 2 * k, rows))
    return ANVIL_ERR_UNSUPPORTED;
  const int eb = elem_bytes(dtype);
  if (!aligned(dy, eb) || !aligned(w, eb) || !aligned(dz, eb) || !aligned(preact, eb))
    return ANVIL_ERR_MISALIGNED;
  st = check_views({{dy, rows, n * eb, lddy * eb, false},
                    dense(w, w ? count * n * k * eb : 0, false),
                    {preact, rows, 2 * k * eb, ldz * eb, false},
                    {dz, rows, 2 * k * eb, lddz * eb, true},
                    offsets_view(g)});
  if (st != ANVIL_OK) return st;
  anvil::RowsProduct a{};
  a.a = dy; a.lda = lddy; a.b = w; a.b_kmajor = w_kn == 0;   // as rows_backward
  a.rows = rows; a.cols = static_cast<int>(k); a.depth = static_cast<int>(n);
  a.groups = groups_of(g, grouped);
  a.f16 = dtype == ANVIL_F16;
  a.act = act;
  a.aux = preact; a.ldaux = ldz;
  a.out = dz; a.ldout = lddz;
  return hip_status(has_w ? anvil::launch_gated_grad(a, static_cast<hipStream_t>(stream))
                          : anvil::launch_gated_activation_grad(a, static_cast<hipStream_t>(stream)));
}

constexpr GroupIn kNoGroups{nullptr, 32, 1};

// ------------------------------------------------------------------------------------------
// Layer norm
// ------------------------------------------------------------------------------------------

int check_norm(int dtype, int param_dtype, bool params, int64_t rows, int64_t cols) {
  if (!elem_known(dtype) || (params && param_dtype != ANVIL_F32 && param_dtype != dtype))
    return ANVIL_ERR_INVALID_ARG;
  if (rows < 0 || cols < 0) return ANVIL_ERR_INVALID_ARG;
  if (rows >= kMaxRows || cols > kMaxWidth) return ANVIL_ERR_UNSUPPORTED;
  return ANVIL_OK;
}

}  // namespace

extern "C" {

int anvil_layer_norm(const void* x, int64_t ldx, const void* weight, const void* bias,
                     int param_dtype, float eps, void* y, int64_t ldy, float* mean, float* rstd,
                     int dtype, int64_t rows, int64_t cols, void* stream) {
  int st = check_norm(dtype, param_dtype, weight || bias, rows, cols);
  if (st != ANVIL_OK) return st;
  if (rows == 0 || cols == 0) return ANVIL_OK;
  if (!x || !y) return ANVIL_ERR_INVALID_ARG;
  if (!take_pitch(x, &ldx, cols, rows) || !take_pitch(y, &ldy, cols, rows)) return ANVIL_ERR_UNSUPPORTED;
  const int eb = elem_bytes(dtype), pb = weight || bias ? elem_bytes(param_dtype) : 1;
  if (!aligned(x, eb) || !aligned(y, eb) || !aligned(weight, pb) || !aligned(bias, pb) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return ANVIL_ERR_MISALIGNED;
  st = check_views({{x, rows, cols * eb, ldx * eb, false},
                    dense(weight, cols * pb, false),
                    dense(bias, cols * pb, false),
                    {y, rows, cols * eb, ldy * eb, true},
                    dense(mean, rows * 4, true),
                    dense(rstd, rows * 4, true)});
  if (st != ANVIL_OK) return st;
  anvil::NormArgs a{};
  a.x = x; a.ldx = ldx; a.weight = weight; a.bias = bias;
  a.param_f32 = param_dtype == ANVIL_F32;
  a.eps = eps; a.y = y; a.ldy = ldy; a.mean = mean; a.rstd = rstd;
  a.type = dtype; a.rows = rows; a.cols = static_cast<int>(cols);
  return hip_status(anvil::launch_norm(a, static_cast<hipStream_t>(stream)));
}

size_t anvil_layer_norm_grad_workspace(int64_t rows, int64_t cols) {
  if (check_norm(ANVIL_F32, ANVIL_F32, false, rows, cols) != ANVIL_OK || cols == 0) return 0;
  return static_cast<size_t>(anvil::norm_grad_blocks(rows, static_cast<int>(cols))) * 2 * cols * 4;
}

int anvil_layer_norm_grad(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                          const void* weight, int param_dtype, const float* mean,
                          const float* rstd, void* dx, int64_t lddx, float* dweight, float* dbias,
                          int dtype, int64_t rows, int64_t cols, void* workspace,
                          size_t workspace_bytes, void* stream) {
  int st = check_norm(dtype, param_dtype, weight != nullptr, rows, cols);
  if (st != ANVIL_OK) return st;
  if (cols == 0) return ANVIL_OK;
  const bool sums = dweight || dbias;
  if (rows == 0 && !sums) return ANVIL_OK;
  if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return ANVIL_ERR_INVALID_ARG;
  if (!take_pitch(dy, &lddy, cols, rows) || !take_pitch(x, &ldx, cols, rows) ||
      !take_pitch(dx, &lddx, cols, rows))
    return ANVIL_ERR_UNSUPPORTED;
  const int eb = elem_bytes(dtype), pb = weight ? elem_bytes(param_dtype) : 1;
  if (!aligned(dy, eb) || !aligned(x, eb) || !aligned(dx, eb) || !aligned(weight, pb) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4))
    return ANVIL_ERR_MISALIGNED;
  const size_t need = sums ? anvil_layer_norm_grad_workspace(rows, cols) : 0;
  if (need) {
    if (!workspace) return ANVIL_ERR_INVALID_ARG;
    if (workspace_bytes < need) return ANVIL_ERR_UNSUPPORTED;
    if (!aligned(workspace, 256)) return ANVIL_ERR_MISALIGNED;
  }
  st = check_views({{dy, rows, cols * eb, lddy * eb, false},
                    {x, rows, cols * eb, ldx * eb, false},
                    dense(weight, cols * pb, false),
                    dense(mean, rows * 4, false),
                    dense(rstd, rows * 4, false),
                    {dx, rows, cols * eb, lddx * eb, true},
                    dense(dweight, cols * 4, true),
                    dense(dbias, cols * 4, true),
                    dense(need ? workspace : nullptr, need, true)});
  if (st != ANVIL_OK) return st;
  anvil::NormArgs a{};
  a.x = x; a.ldx = ldx; a.weight = weight; a.param_f32 = param_dtype == ANVIL_F32;
  a.y = dx; a.ldy = lddx;
  a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
  a.type = dtype; a.rows = rows; a.cols = static_cast<int>(cols);
  return hip_status(anvil::launch_norm_grad(a, dy, lddy, dweight, dbias,
                                            static_cast<float*>(workspace),
                                            static_cast<hipStream_t>(stream)));
}

int anvil_linear(const void* x, int64_t ldx, const void* w, int w_kn, const void* bias,
                 int bias_dtype, int act, const void* residual, int64_t ldr, void* y, int64_t ldy,
                 void* preact, int64_t ldz, int dtype, int64_t rows, int64_t n, int64_t k,
                 void* stream) {
  return rows_forward(x, ldx, w, w_kn, kNoGroups, false, bias, bias_dtype, act, residual, ldr, y,
                      ldy, preact, ldz, dtype, rows, n, k, stream);
}

int anvil_linear_grad_input(const void* dz, int64_t lddz, const void* w, int w_kn,
                            const void* preact, int64_t ldz, int act, const void* add,
                            int64_t ldadd, void* dx, int64_t lddx, int dtype, int64_t rows,
                            int64_t n, int64_t k, void* stream) {
  return rows_backward(dz, lddz, w, w_kn, kNoGroups, false, preact, ldz, act, add, ldadd, dx, lddx,
                       dtype, rows, n, k, stream);
}

size_t anvil_linear_grad_weight_workspace(int w_kn, int64_t rows, int64_t n, int64_t k,
                                          int64_t experts) {
  return weight_workspace(w_kn, rows, n, k, experts);
}

int anvil_linear_grad_weight(const void* dz, int64_t lddz, const void* x, int64_t ldx, int w_kn,
                             void* dw, int dw_dtype, float* dbias, int dtype, int64_t rows,
                             int64_t n, int64_t k, void* workspace, size_t workspace_bytes,
                             void* stream) {
  return weight_backward(dz, lddz, x, ldx, w_kn, kNoGroups, false, dw, dw_dtype, dbias, dtype, rows,
                         n, k, workspace, workspace_bytes, stream);
}

int anvil_expert_linear(const void* x, int64_t ldx, const void* w, int w_kn, const void* offsets,
                        int offset_bits, int64_t experts, const void* bias, int bias_dtype, int act,
                        const void* residual, int64_t ldr, void* y, int64_t ldy, void* preact,
                        int64_t ldz, int dtype, int64_t rows, int64_t n, int64_t k, void* stream) {
  return rows_forward(x, ldx, w, w_kn, {offsets, offset_bits, experts}, true, bias, bias_dtype, act,
                      residual, ldr, y, ldy, preact, ldz, dtype, rows, n, k, stream);
}

int anvil_expert_grad_input(const void* dz, int64_t lddz, const void* w, int w_kn,
                            const void* offsets, int offset_bits, int64_t experts,
                            const void* preact, int64_t ldz, int act, const void* add,
                            int64_t ldadd, void* dx, int64_t lddx, int dtype, int64_t rows,
                            int64_t n, int64_t k, void* stream) {
  return rows_backward(dz, lddz, w, w_kn, {offsets, offset_bits, experts}, true, preact, ldz, act,
                       add, ldadd, dx, lddx, dtype, rows, n, k, stream);
}

int anvil_expert_grad_weight(const void* dz, int64_t lddz, const void* x, int64_t ldx, int w_kn,
                             const void* offsets, int offset_bits, int64_t experts, void* dw,
                             int dw_dtype, float* dbias, int dtype, int64_t rows, int64_t n,
                             int64_t k, void* workspace, size_t workspace_bytes, void* stream) {
  return weight_backward(dz, lddz, x, ldx, w_kn, {offsets, offset_bits, experts}, true, dw,
                         dw_dtype, dbias, dtype, rows, n, k, workspace, workspace_bytes, stream);
}

int anvil_activation_grad(const void* dy, int64_t lddy, const void* preact, int64_t ldz, int act,
                          void* dz, int64_t lddz, int dtype, int64_t rows, int64_t n,
                          void* stream) {
  int st = check_sizes(dtype, kNoGroups, false, rows, n, 0);
  if (st != ANVIL_OK) return st;
  if (!act_known(act)) return ANVIL_ERR_INVALID_ARG;
  if (rows == 0 || n == 0) return ANVIL_OK;
  if (!dy || !preact || !dz) return ANVIL_ERR_INVALID_ARG;
  if (!take_pitch(dy, &lddy, n, rows) || !take_pitch(preact, &ldz, n, rows) ||
      !take_pitch(dz, &lddz, n, rows))
    return ANVIL_ERR_UNSUPPORTED;
  const int eb = elem_bytes(dtype);
  if (!aligned(dy, eb) || !aligned(preact, eb) || !aligned(dz, eb)) return ANVIL_ERR_MISALIGNED;
  st = check_views({{dy, rows, n * eb, lddy * eb, false},
                    {preact, rows, n * eb, ldz * eb, false},
                    {dz, rows, n * eb, lddz * eb, true}});
  if (st != ANVIL_OK) return st;
  return hip_status(anvil::launch_activation_grad(dy, lddy, preact, ldz, act, dz, lddz,
                                                  dtype == ANVIL_F16, rows, static_cast<int>(n),
                                                  static_cast<hipStream_t>(stream)));
}

int anvil_gated_linear(const void* x, int64_t ldx, const void* w, int w_kn, const void* bias,
                       int bias_dtype, int act, void* y, int64_t ldy, void* preact, int64_t ldz,
                       int dtype, int64_t rows, int64_t n, int64_t k, void* stream) {
  return gated_forward(x, ldx, w, w_kn, kNoGroups, false, bias, bias_dtype, act, y, ldy, preact,
                       ldz, dtype, rows, n, k, stream);
}

int anvil_gated_grad_input(const void* dy, int64_t lddy, const void* w, int w_kn,
                           const void* preact, int64_t ldz, int act, void* dz, int64_t lddz,
                           int dtype, int64_t rows, int64_t n, int64_t k, void* stream) {
  return gated_backward(dy, lddy, w, true, w_kn, kNoGroups, false, preact, ldz, act, dz, lddz, dtype,
                        rows, n, k, stream);
}

int anvil_gated_activation_grad(const void* dh, int64_t lddh, const void* preact, int64_t ldz,
                                int act, void* dz, int64_t lddz, int dtype, int64_t rows, int64_t n,
                                void* stream) {
  return gated_backward(dh, lddh, nullptr, false, 0, kNoGroups, false, preact, ldz, act, dz, lddz,
                        dtype, rows, n, n, stream);
}

int anvil_expert_gated_linear(const void* x, int64_t ldx, const void* w, int w_kn,
                              const void* offsets, int offset_bits, int64_t experts,
                              const void* bias, int bias_dtype, int act, void* y, int64_t ldy,
                              void* preact, int64_t ldz, int dtype, int64_t rows, int64_t n,
                              int64_t k, void* stream) {
  return gated_forward(x, ldx, w, w_kn, {offsets, offset_bits, experts}, true, bias, bias_dtype, act,
                       y, ldy, preact, ldz, dtype, rows, n, k, stream);
}

int anvil_expert_gated_grad_input(const void* dy, int64_t lddy, const void* w, int w_kn,
                                  const void* offsets, int offset_bits, int64_t experts,
                                  const void* preact, int64_t ldz, int act, void* dz, int64_t lddz,
                                  int dtype, int64_t rows, int64_t n, int64_t k, void* stream) {
  return gated_backward(dy, lddy, w, true, w_kn, {offsets, offset_bits, experts}, true, preact, ldz,
                        act, dz, lddz, dtype, rows, n, k, stream);
}

}  // extern "C"
