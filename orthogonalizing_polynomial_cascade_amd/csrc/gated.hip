// The gated linear layer, h = act(x W_g^T + b_g) * (x W_u^T + b_u), in one product of 2 n columns, and the
// gradient of z = [z_g, z_u] through the layer that h feeds, dh = dy W:
//   dz_g = dh z_u act'(z_g),   dz_u = dh act(z_g).
//
// Forward: a tile's columns are the same columns of both projections, half of each wave's fragments from
// either (Pipe's PAIR), so the two sums of an output element meet in one lane and the activation and the
// product are taken in registers, in fp32.  One read of x serves both projections, and h (and z, where the
// backward pass wants it) leave rounded once.  The gradient takes the linear layers' product as it is and
// reads z and writes both halves of dz in its epilogue, so that dh is never in memory.
// Everything else (slabs, fragments, tile order and choice, groups) is linear_tiles.hip's.
//
// Bound by the matrix cores and, one after the other on a CU, by the outgoing rows: 32768 rows, 768 -> 2 x
// 2816, silu: 258 us without z (1100 TFLOP/s; the library's plain product 250), 303-325 with z (553 MB leave);
// the gradient 242-256 us (141 GFLOP, 740 MB of z and dz).  256x256 tiles on four waves by two give a wave 64
// columns of either projection, so that rows leave as whole lines; rounded ahead of LDS they take
// half of its accesses (354 -> 322 us).  128x128 tiles, two workgroups a CU: 379 us with z, 261 the gradient.
// One row takes 6.6 us (six sets of waves over the depth).  Odd widths (any_gated_kernel): 517 rows, 1001 x 513 22.3 us
// forward and 20.3 the gradient in a trace; 16384 rows, 769 -> 2 x 2817 305, with z 382, the gradient 312.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "activation.h"
#include "any_pipe.h"
#include "tile_pipe.h"

namespace anvil {

namespace {

// The lane's four biases of columns c .. c + 3 (zeros past the width: cols is a multiple of 8).
template <typename T>
__device__ __forceinline__ void bias4(const RowsProduct& p, int64_t base, int c, float b[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = 0.0f;
  if (c >= p.cols) return;
  if (p.bias_f32) load_vec<float, 4>(static_cast<const float*>(p.bias) + base + c, b);
  else load_vec<T, 4>(static_cast<const T*>(p.bias) + base + c, b);
}

// Values leave rounded where a wave has 64 columns of them, which takes half of the LDS accesses.
template <typename T, typename C>
using GatedStage = std::conditional_t<C::kFN == 4, OutStage16<T>, OutStage<32>>;

// The outgoing rows of a wave's block: rows r0 .. of a group that ends at `end`, output columns c0 ..
template <typename T, typename C, int ACT>
__device__ __forceinline__ void gated_out(const RowsProduct& p, f32x16_t (&acc)[C::kFM][C::kFN],
                                          char* stage, int64_t r0, int64_t end, int group, int c0,
                                          int lane) {
  constexpr int F = C::kFN / 2;
  using S = GatedStage<T, C>;
  const int c = c0 + S::col(lane);
  const int64_t first = r0 + S::row(0, lane);
  const int rows = c < p.cols ? (int)min(end - first, (int64_t)C::kWTM) : 0;   // below: row inside
  T* out = static_cast<T*>(p.out) + first * p.ldout + c;
  T* keep = static_cast<T*>(p.keep) + first * p.ldkeep + c;
  auto leave = [&](const f32x16_t (&v)[F], int fm, T* to, int64_t ld) {
    S::put(stage, v, lane);
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) {
      const int r = fm * 32 + i * S::kRows;
      if constexpr (F == 2) {
        const u32x4_t w = S::get(stage, i, lane);
        if (r < rows) *reinterpret_cast<u32x4_t*>(to + r * ld) = w;
      } else {
        float w[8];
        S::get(stage, i, lane, w);
        if (r < rows) *reinterpret_cast<u32x4_t*>(to + r * ld) = pack8<T>(w);
      }
    }
  };
#pragma unroll
  for (int fm = 0; fm < C::kFM; ++fm) {
    f32x16_t gate[F], up[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
      gate[f] = acc[fm][f];
      up[f] = acc[fm][F + f];
    }
    if (p.bias && group >= 0) {
      const int64_t base = (int64_t)group * 2 * p.cols;
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int at = c0 + f * 32 + 8 * q + 4 * (lane >> 5);
          float bg[4], bu[4];
          bias4<T>(p, base, at, bg);
          bias4<T>(p, base + p.cols, at, bu);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            gate[f][4 * q + e] += bg[e];
            up[f][4 * q + e] += bu[e];
          }
        }
    }
    if (p.keep) {
      leave(gate, fm, keep, p.ldkeep);
      leave(up, fm, keep + p.cols, p.ldkeep);
    }
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int e = 0; e < 16; ++e) gate[f][e] = act_value(ACT, gate[f][e]) * up[f][e];
    leave(gate, fm, out, p.ldout);
  }
}

// Rows without an owner have zero sums and no bias: their z and h are zeros.
template <typename T, bool QT, int BM, int BN, int WM, int WN, int KS, int OCC>
__global__ __launch_bounds__(WM * WN * KS * 64)
__attribute__((amdgpu_waves_per_eu(OCC)))
void gated_tile_kernel(RowsProduct p, int tiles_n) {
  using C = Tile<BM, BN, WM, WN, KS>;
  using S = GatedStage<T, C>;
  static_assert(C::kWaves * S::kBytes <= C::kStage, "the outgoing rows fit one buffer");
  extern __shared__ __attribute__((aligned(1024))) char smem_all[];
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int kg = wave_all / C::kWaves;
  const int wave = wave_all % C::kWaves;
  char* smem = smem_all + kg * C::kRing;
  int64_t row0, end;
  int group, tj;
  if (!rows_place<BM>(p.groups, p.rows, tiles_n, &row0, &end, &group, &tj)) return;
  const int j0 = tj * (BN / 2);
  const uint16_t* b = static_cast<const uint16_t*>(p.b) +
                      (int64_t)(group < 0 ? 0 : group) * 2 * p.cols * p.depth +
                      (QT ? (int64_t)j0 : (int64_t)j0 * p.depth);

  f32x16_t acc[C::kFM][C::kFN];
#pragma unroll
  for (int fm = 0; fm < C::kFM; ++fm)
#pragma unroll
    for (int fn = 0; fn < C::kFN; ++fn) acc[fm][fn] = f32x16_t{};
  float none;
  Pipe<T, false, QT, BM, BN, WM, WN, KS, true> pipe(smem, wave);
  pipe.begin(static_cast<const uint16_t*>(p.a) + row0 * p.lda, p.lda, end - row0, b,
             QT ? 2 * (int64_t)p.cols : p.depth, p.cols - j0, group < 0 ? 0 : p.depth, kg,
             QT ? (int64_t)p.cols : (int64_t)p.cols * p.depth);
  const int wm = wave / WN, wn = wave % WN;
  const bool idle = row0 + wm * C::kWTM >= end;   // no row of the wave's block is there
  if (idle) pipe.attend();
  else pipe.template run<false>(acc, 0, none);
  if constexpr (KS > 1) {
    pipe.merge(kg, acc);
    if (kg > 0) return;
  }
  if (idle) return;
  char* stage = pipe.spare() + wave * S::kBytes;
  const int64_t r0 = row0 + wm * C::kWTM;
  const int c0 = j0 + wn * (C::kWTN / 2);
  switch (p.act) {
    case kActRelu: return gated_out<T, C, kActRelu>(p, acc, stage, r0, end, group, c0, lane);
    case kActRelu2: return gated_out<T, C, kActRelu2>(p, acc, stage, r0, end, group, c0, lane);
    case kActGelu: return gated_out<T, C, kActGelu>(p, acc, stage, r0, end, group, c0, lane);
    case kActSilu: return gated_out<T, C, kActSilu>(p, acc, stage, r0, end, group, c0, lane);
    default: return gated_out<T, C, kActNone>(p, acc, stage, r0, end, group, c0, lane);
  }
}

// dz of eight elements: d (dh in, dz_g out), gate in, up (z_u in, dz_u out).
template <int ACT, int N>
__device__ __forceinline__ void gated_slope(float (&d)[N], const float (&gate)[N], float (&up)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float dh = d[e];
    d[e] = dh * up[e] * act_slope(ACT, gate[e]);
    up[e] = dh * act_value(ACT, gate[e]);
  }
}

template <typename T, typename C, int ACT>
__device__ __forceinline__ void gated_grad_out(const RowsProduct& p,
                                               const f32x16_t (&acc)[C::kFM][C::kFN], char* stage,
                                               int64_t r0, int64_t end, int group, int c, int lane) {
  using S = OutStage<C::kWTN>;
  const int64_t first = r0 + S::row(0, lane);
  const int rows = c < p.cols ? (int)min(end - first, (int64_t)C::kWTM) : 0;   // below: row inside
  T* out = static_cast<T*>(p.out) + first * p.ldout + c;
  const T* z = static_cast<const T*>(p.aux) + first * p.ldaux + c;
  u32x4_t gate_next[S::kPasses], up_next[S::kPasses];   // 32 rows ahead
  auto fetch = [&](int fm) {
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) {
      const int r = fm * 32 + i * S::kRows;
      gate_next[i] = up_next[i] = u32x4_t{};
      if (r < rows) {
        gate_next[i] = *reinterpret_cast<const u32x4_t*>(z + r * p.ldaux);
        up_next[i] = *reinterpret_cast<const u32x4_t*>(z + r * p.ldaux + p.cols);
      }
    }
  };
  fetch(0);
#pragma unroll
  for (int fm = 0; fm < C::kFM; ++fm) {
    S::put(stage, acc[fm], lane);
    u32x4_t gate_now[S::kPasses], up_now[S::kPasses];
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) {
      gate_now[i] = gate_next[i];
      up_now[i] = up_next[i];
    }
    if (fm + 1 < C::kFM) fetch(fm + 1);
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) {
      const int r = fm * 32 + i * S::kRows;
      float d[8], gate[8], up[8];
      S::get(stage, i, lane, d);
      unpack8<T>(gate_now[i], gate);
      unpack8<T>(up_now[i], up);
      gated_slope<ACT>(d, gate, up);
      if (r < rows) {
        *reinterpret_cast<u32x4_t*>(out + r * p.ldout) = group < 0 ? u32x4_t{} : pack8<T>(d);
        *reinterpret_cast<u32x4_t*>(out + r * p.ldout + p.cols) = group < 0 ? u32x4_t{} : pack8<T>(up);
      }
    }
  }
}

template <typename T, bool QT, int BM, int BN, int WM, int WN, int KS, int OCC>
__global__ __launch_bounds__(WM * WN * KS * 64)
__attribute__((amdgpu_waves_per_eu(OCC)))
void gated_grad_kernel(RowsProduct p, int tiles_n) {
  using C = Tile<BM, BN, WM, WN, KS>;
  using S = OutStage<C::kWTN>;
  static_assert(C::kWaves * S::kBytes <= C::kStage, "the outgoing rows fit one buffer");
  extern __shared__ __attribute__((aligned(1024))) char smem_all[];
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int kg = wave_all / C::kWaves;
  const int wave = wave_all % C::kWaves;
  char* smem = smem_all + kg * C::kRing;
  int64_t row0, end;
  int group, tj;
  if (!rows_place<BM>(p.groups, p.rows, tiles_n, &row0, &end, &group, &tj)) return;
  const int j0 = tj * BN;
  const uint16_t* b = static_cast<const uint16_t*>(p.b) +
                      (int64_t)(group < 0 ? 0 : group) * p.cols * p.depth +
                      (QT ? (int64_t)j0 : (int64_t)j0 * p.depth);

  f32x16_t acc[C::kFM][C::kFN];
#pragma unroll
  for (int fm = 0; fm < C::kFM; ++fm)
#pragma unroll
    for (int fn = 0; fn < C::kFN; ++fn) acc[fm][fn] = f32x16_t{};
  float none;
  Pipe<T, false, QT, BM, BN, WM, WN, KS> pipe(smem, wave);
  pipe.begin(static_cast<const uint16_t*>(p.a) + row0 * p.lda, p.lda, end - row0, b,
             QT ? p.cols : p.depth, p.cols - j0, group < 0 ? 0 : p.depth, kg);
  const int wm = wave / WN, wn = wave % WN;
  const bool idle = row0 + wm * C::kWTM >= end;
  if (idle) pipe.attend();
  else pipe.template run<false>(acc, 0, none);
  if constexpr (KS > 1) {
    pipe.merge(kg, acc);
    if (kg > 0) return;
  }
  if (idle) return;
  char* stage = pipe.spare() + wave * S::kBytes;
  const int64_t r0 = row0 + wm * C::kWTM;
  const int c = j0 + wn * C::kWTN + S::col(lane);
  switch (p.act) {
    case kActRelu: return gated_grad_out<T, C, kActRelu>(p, acc, stage, r0, end, group, c, lane);
    case kActRelu2: return gated_grad_out<T, C, kActRelu2>(p, acc, stage, r0, end, group, c, lane);
    case kActGelu: return gated_grad_out<T, C, kActGelu>(p, acc, stage, r0, end, group, c, lane);
    case kActSilu: return gated_grad_out<T, C, kActSilu>(p, acc, stage, r0, end, group, c, lane);
    default: return gated_grad_out<T, C, kActNone>(p, acc, stage, r0, end, group, c, lane);
  }
}

// Eight elements at p, `there` of them in the row (zeros past it).
template <typename T>
__device__ __forceinline__ void load_there(const T* p, int there, float v[8]) {
  if (there >= 8) return load_vec<T, 8>(p, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e < there ? to_f32(p[e]) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void store_there(T* p, int there, const float v[8]) {
  if (there >= 8) return store_vec<T, 8>(p, v);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < there) p[e] = from_f32<T>(v[e]);
}

// The outgoing 32 x 32 fragments of a wave, through LDS so that a lane has eight columns of a row: rows r0 ..
// of a group that ends at `end`, columns c0 ..  (Element by element from the accumulators' layout, 32 rows an
// instruction, the gradient of 16384 x 2817 took 882 us for 312, the forward pass with z 550 for 382.)
template <typename T, int ACT, int F>
__device__ __forceinline__ void any_gated_out(const RowsProduct& p, const f32x16_t (&acc)[F][2],
                                              char* stage, int64_t r0, int64_t end, int group,
                                              int64_t c0, int lane) {
  using S = OutStage<32>;
  const int64_t c = c0 + S::col(lane);
  const int there = c < p.cols ? (int)min(p.cols - c, (int64_t)8) : 0;
  float bias[2][16];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t col = c0 + 8 * (i / 4) + 4 * (lane >> 5) + i % 4;
      bias[h][i] = 0.0f;
      if (p.bias && group >= 0 && col < p.cols) {
        const int64_t at = ((int64_t)group * 2 + h) * p.cols + col;
        bias[h][i] = p.bias_f32 ? static_cast<const float*>(p.bias)[at]
                                : to_f32(static_cast<const T*>(p.bias)[at]);
      }
    }
  auto leave = [&](const f32x16_t& v, int m, void* to, int64_t ld, int64_t shift) {
    const f32x16_t one[1] = {v};
    S::put(stage, one, lane);
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) {
      const int64_t r = r0 + m * 32 + S::row(i, lane);
      float w[8];
      S::get(stage, i, lane, w);
      if (r < end) store_there(static_cast<T*>(to) + r * ld + shift + c, there, w);
    }
  };
#pragma unroll
  for (int m = 0; m < F; ++m) {
    f32x16_t gate = acc[m][0], up = acc[m][1];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      gate[i] += bias[0][i];
      up[i] += bias[1][i];
    }
    if (p.keep) {
      leave(gate, m, p.keep, p.ldkeep, 0);
      leave(up, m, p.keep, p.ldkeep, p.cols);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) gate[i] = act_value(ACT, gate[i]) * up[i];
    leave(gate, m, p.out, p.ldout, 0);
  }
}

template <typename T, int ACT, int F>
__device__ __forceinline__ void any_grad_out(const RowsProduct& p, const f32x16_t (&acc)[F][F],
                                             char* stage, int64_t r0, int64_t end, int group,
                                             int64_t c0, int lane) {
  using S = OutStage<32>;
#pragma unroll
  for (int n = 0; n < F; ++n) {
    const int64_t c = c0 + n * 32 + S::col(lane);
    const int there = c < p.cols ? (int)min(p.cols - c, (int64_t)8) : 0;
#pragma unroll
    for (int m = 0; m < F; ++m) {
      const f32x16_t one[1] = {acc[m][n]};
      S::put(stage, one, lane);
#pragma unroll
      for (int i = 0; i < S::kPasses; ++i) {
        const int64_t r = r0 + m * 32 + S::row(i, lane);
        float d[8], gate[8], up[8];
        S::get(stage, i, lane, d);
        if (r >= end || there == 0) continue;
        const T* z = static_cast<const T*>(p.aux) + r * p.ldaux + c;
        load_there(z, there, gate);
        load_there(z + p.cols, there, up);
        gated_slope<ACT>(d, gate, up);
        if (group < 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = up[e] = 0.0f;
        }
        T* out = static_cast<T*>(p.out) + r * p.ldout + c;
        store_there(out, there, d);
        store_there(out + p.cols, there, up);
      }
    }
  }
}

// Any width, pitch and alignment: tiles of 64 or 128 rows through registers, the forward pass's by 64 columns
// of either projection, which meet in one lane as in the tiles above.  (In two passes over the depth, one for
// each projection, 128x128 tiles spilled 126 registers and 64x64 ones waited twice as long.)
template <typename T, bool QT, int SIDE, bool GRADIENT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2)))
void any_gated_kernel(RowsProduct p, int tiles_n) {
  constexpr int F = SIDE / 64;
  constexpr int kCols = GRADIENT ? SIDE : 64, FN = kCols / 64;   // columns of a tile, a wave's fragments of them
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t wide = GRADIENT ? p.cols : 2 * (int64_t)p.cols;   // columns of b
  __shared__ __attribute__((aligned(16))) char stage[4 * OutStage<32>::kBytes];
  RowTiles<SIDE> tiles(p.groups, p.rows);
  for (int64_t tile = blockIdx.x; tile < (int64_t)tiles.total * tiles_n; tile += gridDim.x) {
    int64_t row0, end;
    int group;
    tiles.find((int)(tile / tiles_n), &row0, &end, &group);
    const int64_t j0 = (tile % tiles_n) * kCols;
    const T* b = static_cast<const T*>(p.b) + (int64_t)(group < 0 ? 0 : group) * wide * p.depth;
    f32x16_t acc[F][GRADIENT ? FN : 2] = {};
    float none[F] = {};
    any_accumulate<T, false, QT, SIDE, !GRADIENT>(
        static_cast<const T*>(p.a), p.lda, row0, end, b, QT ? wide : p.depth, j0, p.cols, 0,
        group < 0 ? 0 : p.depth, acc, 0, none, QT ? (int64_t)p.cols : (int64_t)p.cols * p.depth);
    char* mine = stage + wave * OutStage<32>::kBytes;
    const int64_t r0 = row0 + (wave >> 1) * F * 32, c0 = j0 + (wave & 1) * FN * 32;
    auto out = [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      if constexpr (GRADIENT) any_grad_out<T, ACT, F>(p, acc, mine, r0, end, group, c0, lane);
      else any_gated_out<T, ACT, F>(p, acc, mine, r0, end, group, c0, lane);
    };
    switch (p.act) {
      case kActRelu: out(std::integral_constant<int, kActRelu>{}); break;
      case kActRelu2: out(std::integral_constant<int, kActRelu2>{}); break;
      case kActGelu: out(std::integral_constant<int, kActGelu>{}); break;
      case kActSilu: out(std::integral_constant<int, kActSilu>{}); break;
      default: out(std::integral_constant<int, kActNone>{}); break;
    }
  }
}

// dz from dh in memory, elementwise; bound by memory.
template <typename T, int ACT>
__global__ __launch_bounds__(256) void gated_activation_kernel(RowsProduct p) {
  const int pieces = (p.cols + 7) / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.rows * pieces;
       i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / pieces;
    const int c = (int)(i % pieces) * 8;
    const T* dh = static_cast<const T*>(p.a) + r * p.lda + c;
    const T* z = static_cast<const T*>(p.aux) + r * p.ldaux + c;
    T* out = static_cast<T*>(p.out) + r * p.ldout + c;
    if (c + 8 <= p.cols) {
      float d[8], gate[8], up[8];
      load_vec<T, 8>(dh, d);
      load_vec<T, 8>(z, gate);
      load_vec<T, 8>(z + p.cols, up);
      gated_slope<ACT>(d, gate, up);
      store_vec<T, 8>(out, d);
      store_vec<T, 8>(out + p.cols, up);
    } else {
      for (int e = 0; c + e < p.cols; ++e) {
        float d[1] = {to_f32(dh[e])}, gate[1] = {to_f32(z[e])}, up[1] = {to_f32(z[p.cols + e])};
        gated_slope<ACT>(d, gate, up);
        out[e] = from_f32<T>(d[0]);
        out[p.cols + e] = from_f32<T>(up[0]);
      }
    }
  }
}

// The product's shape as the tile choice sees it: a gated product has twice the output's columns.  The choice is
// the linear layers' fitted cost, which no sweep of the gated products' own tiles has been taken for; 32768 rows,
// 768 -> 2 x 2816 on either side of it stand at the head of this file.
RowsProduct as_rows(const RowsProduct& a, bool gradient) {
  RowsProduct r = a;
  r.cols = gradient ? a.cols : 2 * a.cols;
  return r;
}

template <typename T, bool QT, int BM, int BN, int WM, int WN, int KS, int OCC>
hipError_t gated_tiles(const RowsProduct& a, hipStream_t stream) {
  using C = Tile<BM, BN, WM, WN, KS>;
  static std::atomic<uint64_t> configured{0};
  const int64_t tiles_m = row_tiles(a, BM), tiles_n = ceil64(a.cols, BN / 2);
  return launch_lds(gated_tile_kernel<T, QT, BM, BN, WM, WN, KS, OCC>, configured,
                    ceil64(tiles_m * tiles_n, 8) * 8 + 8, C::kThreads, C::kLds, stream, a,
                    (int)tiles_n);
}

template <typename T, bool QT, int BM, int BN, int WM, int WN, int KS, int OCC>
hipError_t gated_grad_tiles(const RowsProduct& a, hipStream_t stream) {
  using C = Tile<BM, BN, WM, WN, KS>;
  static std::atomic<uint64_t> configured{0};
  const int64_t tiles_m = row_tiles(a, BM), tiles_n = ceil64(a.cols, BN);
  return launch_lds(gated_grad_kernel<T, QT, BM, BN, WM, WN, KS, OCC>, configured,
                    ceil64(tiles_m * tiles_n, 8) * 8 + 8, C::kThreads, C::kLds, stream, a,
                    (int)tiles_n);
}

// The tile shapes of the linear layers (rows_tile), with 64 columns of a pair where those have 32.
template <typename T, bool QT>
hipError_t gated_variant(const RowsProduct& a, hipStream_t stream) {
  switch (rows_tile(as_rows(a, false))) {
    case kRows32: return gated_tiles<T, QT, 32, 64, 1, 1, 6, 2>(a, stream);
    case kRows32x128: return gated_tiles<T, QT, 32, 128, 1, 2, 2, 2>(a, stream);
    case kRows64: return gated_tiles<T, QT, 64, 64, 2, 1, 4, 2>(a, stream);
    case kRows128: return gated_tiles<T, QT, 128, 128, 2, 2, 1, 2>(a, stream);
    default: return gated_tiles<T, QT, 256, 256, 4, 2, 1, 2>(a, stream);
  }
}

template <typename T, bool QT>
hipError_t gated_grad_variant(const RowsProduct& a, hipStream_t stream) {
  switch (rows_tile(as_rows(a, true))) {
    case kRows32: return gated_grad_tiles<T, QT, 32, 32, 1, 1, 8, 2>(a, stream);
    case kRows32x128: return gated_grad_tiles<T, QT, 32, 128, 1, 4, 2, 4>(a, stream);
    case kRows64: return gated_grad_tiles<T, QT, 64, 64, 2, 2, 4, 4>(a, stream);
    case kRows128: return gated_grad_tiles<T, QT, 128, 128, 2, 2, 1, 2>(a, stream);
    default: return gated_grad_tiles<T, QT, 256, 256, 2, 4, 1, 2>(a, stream);
  }
}

template <typename T, int SIDE, bool GRADIENT>
hipError_t any_gated_side(const RowsProduct& a, hipStream_t stream) {
  const int64_t tiles_m = ceil64(a.rows, SIDE) + (a.groups.offsets ? a.groups.count + 1 : 0);
  const int tiles_n = (int)ceil64(a.cols, GRADIENT ? SIDE : 64);
  if (a.b_kmajor)
    any_gated_kernel<T, true, SIDE, GRADIENT>
        <<<grid_for(tiles_m * tiles_n), 256, 0, stream>>>(a, tiles_n);
  else
    any_gated_kernel<T, false, SIDE, GRADIENT>
        <<<grid_for(tiles_m * tiles_n), 256, 0, stream>>>(a, tiles_n);
  return hipGetLastError();
}

template <typename T, bool GRADIENT>
hipError_t any_gated(const RowsProduct& a, hipStream_t stream) {
  return any_wide_tiles(as_rows(a, GRADIENT)) ? any_gated_side<T, 128, GRADIENT>(a, stream)
                           : any_gated_side<T, 64, GRADIENT>(a, stream);
}

bool tiles_take(const RowsProduct& a, bool gradient) {
  const RowsProduct r = as_rows(a, gradient);
  const RowsTile t = rows_tile(r);
  // the narrowest tile of a pair has 64 columns of it where the linear layers' has 32
  return row_tiles(a, kTileRows[t]) * ceil64(r.cols, kTileCols[t]) + 16 <= kMaxTileGrid &&
         a.depth > 0 && multiple8(a.depth) && multiple8(a.cols) && multiple8(a.lda) &&
         multiple8(a.ldout) && wide_aligned(a.a) && wide_aligned(a.b) && wide_aligned(a.out) &&
         (!a.aux || (multiple8(a.ldaux) && wide_aligned(a.aux))) &&
         (!a.keep || (multiple8(a.ldkeep) && wide_aligned(a.keep)));
}

template <typename T>
hipError_t activation_launch(const RowsProduct& a, hipStream_t stream) {
  const unsigned grid = (unsigned)std::min<int64_t>(ceil64(a.rows * ((a.cols + 7) / 8), 256), 16384);
  switch (a.act) {
    case kActRelu: gated_activation_kernel<T, kActRelu><<<grid, 256, 0, stream>>>(a); break;
    case kActRelu2: gated_activation_kernel<T, kActRelu2><<<grid, 256, 0, stream>>>(a); break;
    case kActGelu: gated_activation_kernel<T, kActGelu><<<grid, 256, 0, stream>>>(a); break;
    case kActSilu: gated_activation_kernel<T, kActSilu><<<grid, 256, 0, stream>>>(a); break;
    default: gated_activation_kernel<T, kActNone><<<grid, 256, 0, stream>>>(a); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_product(const RowsProduct& a, hipStream_t stream) {
  if (tiles_take(a, false)) {
    if (a.f16)
      return a.b_kmajor ? gated_variant<f16, true>(a, stream) : gated_variant<f16, false>(a, stream);
    return a.b_kmajor ? gated_variant<bf16, true>(a, stream) : gated_variant<bf16, false>(a, stream);
  }
  return a.f16 ? any_gated<f16, false>(a, stream) : any_gated<bf16, false>(a, stream);
}

hipError_t launch_gated_activation_grad(const RowsProduct& a, hipStream_t stream) {
  return a.f16 ? activation_launch<f16>(a, stream) : activation_launch<bf16>(a, stream);
}

hipError_t launch_gated_grad(const RowsProduct& a, hipStream_t stream) {
  if (tiles_take(a, true)) {
    if (a.f16)
      return a.b_kmajor ? gated_grad_variant<f16, true>(a, stream)
                        : gated_grad_variant<f16, false>(a, stream);
    return a.b_kmajor ? gated_grad_variant<bf16, true>(a, stream)
                      : gated_grad_variant<bf16, false>(a, stream);
  }
  return a.f16 ? any_gated<f16, true>(a, stream) : any_gated<bf16, true>(a, stream);
}

}  // namespace anvil
