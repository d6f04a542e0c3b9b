// Host-side launchers of the ANVIL kernels (internal to libanvil.so).  Arguments are checked by
// the C ABI layer before these are called; each returns the hipError_t of its launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace anvil {

// Fused twin-rail momentum + bf16 cast over `count` elements (count % 8 == 0).
hipError_t launch_momentum(const float* grad, float* v0, float* v1, uint16_t* x, int64_t count,
                           float momentum, float fast_beta, float fast_weight, hipStream_t stream);

// The same with the gradient fp32 or bf16 and (momentum, fast_beta, fast_weight) read from a
// device array when the kernel runs.
hipError_t launch_momentum_dev(const void* grad, bool grad_bf16, float* v0, float* v1,
                               uint16_t* x, int64_t count, const float* scalars,
                               hipStream_t stream);

// Geometry of one bank: stack g of m x n matrices.
struct Shape {
  int64_t g;
  int m, n;
  bool tall() const { return m > n; }
  int s() const { return m > n ? n : m; }
  int L() const { return m > n ? m : n; }
};

// Trace partials per matrix that launch_gram writes: one per 32-row diagonal block for wide or
// square shapes with s <= 256, else one per 128-row diagonal tile.
int gram_trace_slots(const Shape& sh);

hipError_t launch_gram(const uint16_t* x, uint16_t* a, float* trace_partials, const Shape& sh,
                       hipStream_t stream);
hipError_t launch_normalize(uint16_t* x, uint16_t* a, const float* trace_partials, float* d,
                            const Shape& sh, hipStream_t stream);
hipError_t launch_poly(const uint16_t* a, uint16_t* b, float coef_b, float coef_c, int64_t g,
                       int s, hipStream_t stream);
hipError_t launch_apply(const uint16_t* x, const uint16_t* b, uint16_t* c, float coef_a,
                        bool split, const Shape& sh, hipStream_t stream);
// Polynomial and apply of one map in a single launch (C = a X + B X with B = b A + c A·A formed
// per tile), for wide or square shapes with s <= 256 whose tiles of 32 rows by 1, 2, 3 or 6
// chunks of 128 columns fit one round on the CUs; the same arithmetic as launch_poly followed by
// launch_apply, element for element.
bool poly_apply_fused(const Shape& sh);
hipError_t launch_poly_apply(const uint16_t* a, const uint16_t* x, uint16_t* c, float coef_a,
                             float coef_b, float coef_c, const Shape& sh, hipStream_t stream);

// Equalizer lanes of an m x n matrix: rows when m >= n, else columns.
int equalizer_lanes(const Shape& sh);

// Equalizer on u (in place) with lane energies updated in place; scratch holds 2*g*lanes fp32.
// If param is not null, the same elementwise pass applies the sign-aligned decay to
// (param, mantissa) with the rescaled u, gate (the slow rail), per-matrix lr and wd (or wd read
// from the device at *wd_dev when that is not null).
hipError_t launch_equalize(uint16_t* u, float* lane_energy, double beta2, float* scratch,
                           const Shape& sh, hipStream_t stream, uint16_t* param,
                           uint16_t* mantissa, const float* gate, const float* lr, float wd,
                           const float* wd_dev = nullptr);

// The sign-aligned decay alone, with u as given.
hipError_t launch_decay(uint16_t* param, uint16_t* mantissa, const uint16_t* u, float wd,
                        const float* lr, const float* gate, const Shape& sh, hipStream_t stream);

// ---- training operators (norm.hip, linear.hip; checked by train_api.hip) ----

enum ElemType { kF32 = 0, kBf16 = 1, kF16 = 2 };

// Layer norm of `rows` rows; in the backward pass y / ldy are dx / lddx.
struct NormArgs {
  const void* x;
  int64_t ldx;
  const void* weight;
  const void* bias;
  bool param_f32;
  float eps;
  void* y;
  int64_t ldy;
  float* mean;
  float* rstd;
  int type;
  int64_t rows;
  int cols;
};
hipError_t launch_norm(const NormArgs& a, hipStream_t stream);
// Partial rows (of 2 * cols fp32) that launch_norm_grad leaves in `partial`.
int norm_grad_blocks(int64_t rows, int cols);
hipError_t launch_norm_grad(const NormArgs& a, const void* dy, int64_t lddy, float* dweight,
                            float* dbias, float* partial, hipStream_t stream);

// Rows in groups: group e owns rows [offsets[e], offsets[e + 1]) (device integers of 4 or 8
// bytes), and matrix e of a stack.  Without offsets all rows belong to one matrix.
struct Groups {
  const void* offsets;   // or null
  bool wide;             // 64-bit offsets
  int count;
};

// out[r][c] = epilogue(sum_d a[r][d] * b(c, d)), b of the row's group.
//   forward   z = sum + bias;  keep = z;  out = act(z) + add
//   gradient  out = sum * act'(aux) + add
struct RowsProduct {
  const void* a;
  int64_t lda;
  const void* b;
  bool b_kmajor;         // b stored [d][c] instead of [c][d]
  int64_t rows;
  int cols, depth;
  Groups groups;
  bool f16;
  bool gradient;
  int act;
  const void* bias;      // [groups][cols] or null
  bool bias_f32;
  const void* aux;       // gradient: preactivation, or null
  int64_t ldaux;
  const void* add;       // or null
  int64_t ldadd;
  void* keep;            // or null
  int64_t ldkeep;
  void* out;
  int64_t ldout;
};
hipError_t launch_rows_product(const RowsProduct& a, hipStream_t stream);

// Gated linear layer: the product has 2 cols columns, z = sum + bias, of which column c and column
// cols + c give out[r][c] = act(z[r][c]) * z[r][cols + c]; keep receives z [rows][2 cols].  (b is
// [groups][2 cols][depth], or [groups][depth][2 cols]; aux, add and gradient are not used.)
hipError_t launch_gated_product(const RowsProduct& a, hipStream_t stream);
// Its gradient through the layer that follows: with s = sum_d a[r][d] b(c, d) and z = aux [rows][2 cols],
// out[r][c] = s * z[r][cols + c] * act'(z[r][c]) and out[r][cols + c] = s * act(z[r][c]).
hipError_t launch_gated_grad(const RowsProduct& a, hipStream_t stream);
// The same with s = a [rows][cols].
hipError_t launch_gated_activation_grad(const RowsProduct& a, hipStream_t stream);

// dw[e][i][j] = sum over the rows r of group e of p[r][i] * q[r][j], and the column sums of
// whichever of the two is dz.
struct WeightProduct {
  const void* p;
  int64_t ldp;
  const void* q;
  int64_t ldq;
  int64_t rows;
  int pi, qj;
  bool dz_is_q;
  Groups groups;
  bool f16;
  void* dw;
  bool dw_f32;
  float* db;             // [groups][width of dz] or null
};
// Fp32 words of workspace for the product (0: none needed).
size_t weight_product_words(const WeightProduct& a);
hipError_t launch_weight_product(const WeightProduct& a, float* ws, hipStream_t stream);

// dz = dy * act'(z), elementwise.
hipError_t launch_activation_grad(const void* dy, int64_t lddy, const void* z, int64_t ldz, int act,
                                  void* dz, int64_t lddz, bool f16, int64_t rows, int cols,
                                  hipStream_t stream);

}  // namespace anvil
