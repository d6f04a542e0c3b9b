// The cross entropy of a linear head: what its two sources share.  Logits s = x W^T of `rows` tokens over
// `vocab` entries are formed tile by tile and never stored.
#pragma once

#include <hip/hip_runtime.h>

#include "launchers.h"

namespace anvil {

// Row r's target as a column of the whole vocabulary, -1 where it is outside (the row is ignored).
__device__ __forceinline__ int64_t target_of(const void* targets, bool wide, int64_t vocab, int64_t r) {
  const int64_t t = wide ? static_cast<const int64_t*>(targets)[r]
                         : (int64_t)static_cast<const int32_t*>(targets)[r];
  return t >= 0 && t < vocab ? t : -1;
}

// One product over columns [first, first + cols) of the vocabulary.  x [rows][depth] at pitch ldx and w
// ([vocab][depth], or [depth][vocab] where w_kn) at pitch ldw are ready for the copies: 16-byte aligned,
// pitches multiples of 8, the pieces of eight that reach past the depth zero.
struct HeadProduct {
  const void* x;
  int64_t ldx;
  const void* w;
  int64_t ldw;
  bool w_kn, f16;
  int64_t rows;
  int depth;
  int64_t vocab, first, cols;
  const void* targets;
  bool wide;             // 64-bit targets
  // statistics: part [rows][tiles_n] of (maximum, sum of exponentials above it), and loss[r] = the
  // target's logit
  float2* part;
  float* loss;
  // probabilities: p = (softmax - onehot) * dloss * (scale ? scale[0] : 1), rows without a target zeros,
  // in blocks of 64 columns, [ceil(cols / 64)][rows][64], zeros from cols to the next multiple of 8
  const float* lse;
  const float* dloss;
  const float* scale;
  void* p;
};

// The same for a caller's operands of any width, pitch and alignment: what of the workspace a call takes.
// Parts are 256-byte aligned; an offset of -1 means that the part is not needed.
struct HeadPlan {
  int64_t x, w, part;                    // packed operands, statistics
  int64_t scale, p, dx, dx_planes, planes;   // gradients
  int64_t ldx, ldw;                      // pitches of the packed operands
  int64_t piece;                         // columns of the vocabulary at a time
  size_t bytes;
};
HeadPlan head_plan(bool gradient, bool want_dx, bool want_dw, bool w_kn, bool f16, int in_place,
                   int64_t rows, int64_t vocab, int64_t depth);

struct HeadCall {
  const void* x;
  int64_t ldx;
  const void* w;                         // contiguous
  bool w_kn, f16;
  int in_place;                          // 1: x 16-byte aligned, ldx a multiple of 8; 2: w 16-byte aligned
  int64_t rows, vocab;
  int depth;
  const void* targets;
  bool wide;
  float* loss;                           // forward: out; gradient: not used
  float* lse;                            // forward: out; gradient: in
  const float* dloss;
  void* dx;                              // [rows][depth] or null
  int64_t lddx;
  void* dw;                              // as w, or null
  bool dw_f32;
};
hipError_t launch_cross_entropy(const HeadCall& a, char* ws, hipStream_t stream);
hipError_t launch_cross_entropy_grad(const HeadCall& a, char* ws, hipStream_t stream);

// Column tiles of the statistics (the second dimension of part).
int64_t head_stat_tiles(int64_t rows, int64_t vocab, int depth);
hipError_t launch_head_stats(const HeadProduct& a, float* lse, hipStream_t stream);
hipError_t launch_head_probabilities(const HeadProduct& a, hipStream_t stream);

}  // namespace anvil
