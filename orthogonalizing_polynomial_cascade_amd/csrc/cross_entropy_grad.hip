// Gradients of the linear head's cross entropy, and the calls of both directions.
//
// With P = (softmax(x W^T) - onehot) dloss:  dx = P W,  dW = P^T x.  P is formed for a piece of the
// vocabulary at a time (cross_entropy.hip), rounded to the operands' type as the matrix cores take it, and
// both products read it: dW of the piece is complete, dx is summed over the pieces in fp32.  An fp16 P is
// scaled by a power of two so that the largest |dloss| of a row with a target comes to 2^14 (a mean over 16384 rows alone would push
// probabilities below 2^-10 under fp16's range); the products are scaled back in fp32, exactly.  P lies in
// blocks of 64 columns, so that the slabs of both products are contiguous.  The
// rounding of P is each element's own, at most half a step of its type: it adds to a sum of many of them
// what the roundings of the inputs already did.
//
// What bounds it: the matrix cores at the clock that they hold under load (a 64-deep slab of a 256x256 tile
// takes 1.7 us on all CUs, where its multiplies alone would take 0.9 at full clock).  16384 rows, 768 x
// 50304: loss and gradients 5.0-5.25 ms, 8 R V k operations (the logits twice) at 960-1010 TFLOP/s: the loss 1.15-1.2, P
// 1.5, dx 1.5, dW 1.1.  A piece of 21760 entries: P 670 us, dx 515 (1060 TFLOP/s; the library's product
// 468), dW 450 (1215; 553).  Rings of four and five 32-deep slabs for dW, which keep twice as much on its
// way, took the same time.
//
// Operands whose widths or addresses the copies into LDS cannot take (multiples of 8, 16 bytes) are packed
// into the workspace once, with zeros to the next multiple of 8.
#include <algorithm>
#include <atomic>

#include "cross_entropy.h"
#include "tile_pipe.h"

namespace anvil {

namespace {

int64_t ceil8(int64_t v) { return (v + 7) / 8 * 8; }

// What a call has to prepare, in one launch: copies [rows][width] -> [rows][pitch] of 16-bit elements
// with zeros from width to pitch, and the scale of P.
struct PackedCopy {
  const uint16_t* from;
  int64_t ld, rows, width;
  uint16_t* to;          // null: nothing to copy
  int64_t pitch;         // a multiple of 8
};
struct HeadReady {
  PackedCopy copy[2];
  const float* dloss;
  const void* targets;
  bool wide;
  int64_t vocab, rows;
  float* scale;          // {S, 1 / S}, or null
};
constexpr int kReadyThreads = 1024;

// S the power of two that takes the largest finite |dloss| to [2^14, 2^15).  Rows without a target do not
// count: they may hold anything.
__device__ __forceinline__ void find_scale(const HeadReady& p) {
  __shared__ float wave_top[kReadyThreads / 64];
  float top = 0.0f;
  for (int64_t r = threadIdx.x; r < p.rows; r += kReadyThreads) {
    const float v = fabsf(p.dloss[r]);
    if (v > top && v < INFINITY && target_of(p.targets, p.wide, p.vocab, r) >= 0) top = v;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  if ((threadIdx.x & 63) == 0) wave_top[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kReadyThreads / 64; ++i) top = fmaxf(top, wave_top[i]);
    int power = 0;
    if (top > 0.0f) {
      frexpf(top, &power);                       // top in [2^(power - 1), 2^power)
      power = min(max(15 - power, -120), 120);   // S and 1 / S stay normal numbers
    }
    p.scale[0] = ldexpf(1.0f, power);
    p.scale[1] = ldexpf(1.0f, -power);
  }
}

// Workgroup 0 finds the scale where there is one; the others copy.
__global__ __launch_bounds__(kReadyThreads) void head_ready_kernel(HeadReady p) {
  const int first = p.scale ? 1 : 0;
  if ((int)blockIdx.x < first) return find_scale(p);
  const int64_t me = (int64_t)(blockIdx.x - first) * kReadyThreads + threadIdx.x;
  const int64_t step = (int64_t)(gridDim.x - first) * kReadyThreads;
  for (int k = 0; k < 2; ++k) {
    const PackedCopy& c = p.copy[k];
    if (!c.to) continue;
    const int64_t pieces = c.pitch / 8;
    for (int64_t i = me; i < c.rows * pieces; i += step) {
      const int64_t r = i / pieces, at = i % pieces * 8;
      const uint16_t* from = c.from + r * c.ld + at;
      uint16_t v[8];
      if (at + 8 <= c.width) {
        __builtin_memcpy(v, from, 16);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = at + e < c.width ? from[e] : (uint16_t)0;
      }
      __builtin_memcpy(c.to + r * c.pitch + at, v, 16);
    }
  }
}

// v = the sum over the planes of their eight words at `from`, in order; four planes' loads at a time (one
// after the other they took 0.34 us each, 11 of a call of five rows).
__device__ __forceinline__ void sum_planes(const float* from, int64_t plane, int splits, float v[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.0f;
  for (int s = 0; s < splits; s += 4) {
    float t[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k) load_vec<float, 8>(from + min(s + k, splits - 1) * plane, t[k]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += s + k < splits ? t[k][e] : 0.0f;
  }
}

// One piece's part of dx.
struct InputGrad {
  const void* p;         // [ceil(depth / 64)][rows][64]
  const void* w;         // of the piece's first entry
  int64_t ldw;
  int64_t rows;
  int cols, depth;       // width of x, entries of the piece
  int splits;            // parts of the depth; with several, sums go to planes [splits][rows][ldsum]
  float* planes;
  float* sum;            // [rows][ldsum] fp32, when there are several pieces
  int64_t ldsum;         // a multiple of 8
  bool first, last;
  const float* scale;    // or null
  void* out;
  int64_t ldout;
};

// Eight sums (columns c .. c + 7 of row r) joined with those of the pieces before, and on to where they
// belong.
template <typename T>
__device__ __forceinline__ void input_out(const InputGrad& p, int64_t r, int c, float back, float v[8]) {
  float* sum = p.sum + r * p.ldsum + c;
  if (!p.first) {
    float before[8];
    load_vec<float, 8>(sum, before);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += before[e];
  }
  if (!p.last) {
    store_vec<float, 8>(sum, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= back;
  T* out = static_cast<T*>(p.out) + r * p.ldout + c;
  if (c + 8 <= p.cols) {
    store_vec<T, 8>(out, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < p.cols) out[e] = from_f32<T>(v[e]);
  }
}

template <typename T, bool QT, int BM, int BN, int WM, int WN, int KS, int OCC>
__global__ __launch_bounds__(WM * WN * KS * 64)
__attribute__((amdgpu_waves_per_eu(OCC)))
void head_input_kernel(InputGrad p, int tiles_m, int tiles_n) {
  using C = Tile<BM, BN, WM, WN, KS>;
  constexpr int kSide = C::kFN % 2 ? 1 : 2;   // fragments that leave side by side
  using S = OutStage<kSide * 32>;
  static_assert(C::kWaves * S::kBytes <= C::kStage, "the outgoing rows fit one buffer");
  extern __shared__ __attribute__((aligned(1024))) char smem_all[];
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int kg = wave_all / C::kWaves;
  const int wave = wave_all % C::kWaves;
  char* smem = smem_all + kg * C::kRing;
  const int unit = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  const int s = unit / (tiles_m * tiles_n);
  int ti, tj;
  banded(unit % (tiles_m * tiles_n), tiles_m, tiles_n, &ti, &tj);
  const int64_t row0 = (int64_t)ti * BM;
  const int j0 = tj * BN;
  const int part = ((p.depth + kBK - 1) / kBK + p.splits - 1) / p.splits * kBK;
  const int k0 = min(s * part, p.depth), k1 = min(k0 + part, p.depth);
  const uint16_t* w = static_cast<const uint16_t*>(p.w) + (QT ? j0 + k0 * p.ldw : j0 * p.ldw + k0);
  f32x16_t acc[C::kFM][C::kFN];
#pragma unroll
  for (int fm = 0; fm < C::kFM; ++fm)
#pragma unroll
    for (int fn = 0; fn < C::kFN; ++fn) acc[fm][fn] = f32x16_t{};
  float none;
  Pipe<T, false, QT, BM, BN, WM, WN, KS> pipe(smem, wave);
  const uint16_t* block0 = static_cast<const uint16_t*>(p.p);
  pipe.begin(block0, 64, 0, w, p.ldw, p.cols - j0, k1 - k0, kg);
  pipe.sp.init_blocks(block0 + ((k0 / 64 + (KS > 1 ? kg * pipe.KT : 0)) * p.rows + row0) * 64,
                      p.rows * 64, p.rows - row0, wave, lane);
  const int wm = wave / WN, wn = wave % WN;
  const bool idle = row0 + wm * C::kWTM >= p.rows;
  if (idle) pipe.attend();
  else pipe.template run<false>(acc, 0, none);
  if constexpr (KS > 1) {
    pipe.merge(kg, acc);
    if (kg > 0) return;
  }
  if (idle) return;
  char* stage = pipe.spare() + wave * S::kBytes;
  const float back = p.scale ? p.scale[1] : 1.0f;
#pragma unroll
  for (int fn = 0; fn < C::kFN; fn += kSide) {
    const int c = j0 + wn * C::kWTN + fn * 32 + S::col(lane);
#pragma unroll
    for (int fm = 0; fm < C::kFM; ++fm) {
      f32x16_t leaving[kSide];
#pragma unroll
      for (int f = 0; f < kSide; ++f) leaving[f] = acc[fm][fn + f];
      S::put(stage, leaving, lane);
#pragma unroll
      for (int i = 0; i < S::kPasses; ++i) {
        const int64_t r = row0 + wm * C::kWTM + fm * 32 + S::row(i, lane);
        float v[8];
        S::get(stage, i, lane, v);
        if (r >= p.rows || c >= p.cols) continue;
        if (p.splits > 1) store_vec<float, 8>(p.planes + (s * p.rows + r) * p.ldsum + c, v);
        else input_out<T>(p, r, c, back, v);
      }
    }
  }
}

// Adds the planes in order.
template <typename T>
__global__ __launch_bounds__(256) void input_planes_kernel(InputGrad p) {
  const int64_t pieces = p.ldsum / 8, plane = p.rows * p.ldsum;
  const float back = p.scale ? p.scale[1] : 1.0f;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < p.rows * pieces;
       u += (int64_t)gridDim.x * 256) {
    float v[8];
    sum_planes(p.planes + u * 8, plane, p.splits, v);
    input_out<T>(p, u / pieces, (int)(u % pieces) * 8, back, v);
  }
}

// dW of one piece: out[i][j] = the sum over the rows of P(r, i) x(r, j), or of x(r, i) P(r, j).
struct WeightGrad {
  const void* p;         // [ceil(entries / 64)][rows][64]
  const void* x;
  int64_t ldx;
  bool p_second;         // P(r, j)
  int64_t rows;
  int ni, nj;
  int splits;            // parts of the rows; with several, sums go to planes [splits][ni][ceil8(nj)]
  float* planes;
  const float* scale;
  void* out;
  int64_t ldout;
  bool out_f32;
};

// Eight sums (columns j .. j + 7) to the output, scaled back.
template <typename T>
__device__ __forceinline__ void weight_out(const WeightGrad& p, int64_t i, int j, float back,
                                           float v[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= back;
  const int64_t at = i * p.ldout + j;
  if (j + 8 <= p.nj) {
    if (p.out_f32) store_vec<float, 8>(static_cast<float*>(p.out) + at, v);
    else store_vec<T, 8>(static_cast<T*>(p.out) + at, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (j + e >= p.nj) break;
    if (p.out_f32) static_cast<float*>(p.out)[at + e] = v[e];
    else static_cast<T*>(p.out)[at + e] = from_f32<T>(v[e]);
  }
}

template <typename T, int BM, int BN, int WM, int WN, int OCC>
__global__ __launch_bounds__(WM * WN * 64)
__attribute__((amdgpu_waves_per_eu(OCC)))
void head_weight_kernel(WeightGrad p, int tiles_i, int tiles_j) {
  using C = Tile<BM, BN, WM, WN, 1>;
  using S = OutStage<C::kWTN>;
  static_assert(C::kWaves * S::kBytes <= C::kStage, "the outgoing rows fit one buffer");
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int unit = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  const int s = unit / (tiles_i * tiles_j);
  int ti, tj;
  banded(unit % (tiles_i * tiles_j), tiles_i, tiles_j, &ti, &tj);
  const int i0 = ti * BM, j0 = tj * BN;
  const int64_t part = ((p.rows + kBK - 1) / kBK + p.splits - 1) / p.splits * kBK;
  const int64_t k0 = min(s * part, p.rows), k1 = min(k0 + part, p.rows);
  f32x16_t acc[C::kFM][C::kFN];
#pragma unroll
  for (int fm = 0; fm < C::kFM; ++fm)
#pragma unroll
    for (int fn = 0; fn < C::kFN; ++fn) acc[fm][fn] = f32x16_t{};
  float none;
  Pipe<T, true, true, BM, BN, WM, WN, 1> pipe(smem, wave);
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + k0 * p.ldx;
  const uint16_t* blocks = static_cast<const uint16_t*>(p.p);
  const int64_t block = p.rows * 64;
  pipe.begin(x + i0, p.ldx, p.ni - i0, x + j0, p.ldx, p.nj - j0, k1 - k0, 0);
  // (tiles begin at multiples of 64)
  if (p.p_second) pipe.sq[0].init_blocks(blocks + j0 / 64 * block + k0 * 64, block, p.nj - j0, wave, lane);
  else pipe.sp.init_blocks(blocks + i0 / 64 * block + k0 * 64, block, p.ni - i0, wave, lane);
  pipe.template run<false>(acc, 0, none);
  const int wm = wave / WN, wn = wave % WN;
  char* stage = pipe.spare() + wave * S::kBytes;
  const int j = j0 + wn * C::kWTN + S::col(lane);
  const int64_t pitch = (p.nj + 7) / 8 * 8;
  const float back = p.scale ? p.scale[1] : 1.0f;
#pragma unroll
  for (int fm = 0; fm < C::kFM; ++fm) {
    S::put(stage, acc[fm], lane);
#pragma unroll
    for (int k = 0; k < S::kPasses; ++k) {
      const int i = i0 + wm * C::kWTM + fm * 32 + S::row(k, lane);
      float v[8];
      S::get(stage, k, lane, v);
      if (i >= p.ni || j >= p.nj) continue;
      if (p.splits > 1) store_vec<float, 8>(p.planes + ((int64_t)s * p.ni + i) * pitch + j, v);
      else weight_out<T>(p, i, j, back, v);
    }
  }
}

// Adds the planes in order.
template <typename T>
__global__ __launch_bounds__(256) void head_planes_kernel(WeightGrad p) {
  const int64_t pieces = (p.nj + 7) / 8, plane = p.ni * pieces * 8;
  const float back = p.scale ? p.scale[1] : 1.0f;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < p.ni * pieces;
       u += (int64_t)gridDim.x * 256) {
    float v[8];
    sum_planes(p.planes + u * 8, plane, p.splits, v);
    weight_out<T>(p, u / pieces, (int)(u % pieces) * 8, back, v);
  }
}

// Zeros of dW where there are no rows.
__global__ __launch_bounds__(256) void head_zero_kernel(uint16_t* to, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    to[i] = 0;
}

template <typename T, bool QT, int BM, int BN, int WM, int WN, int KS, int OCC>
hipError_t input_tiles(const InputGrad& a, hipStream_t stream) {
  using C = Tile<BM, BN, WM, WN, KS>;
  static std::atomic<uint64_t> configured{0};
  const int64_t tiles_m = ceil64(a.rows, BM), tiles_n = ceil64(a.cols, BN);
  hipError_t e = launch_lds(head_input_kernel<T, QT, BM, BN, WM, WN, KS, OCC>, configured,
                            tiles_m * tiles_n * a.splits, C::kThreads, C::kLds, stream, a,
                            (int)tiles_m, (int)tiles_n);
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t pieces = a.rows * (a.ldsum / 8);
  input_planes_kernel<T><<<dim3((unsigned)std::min<int64_t>(ceil64(pieces, 256), 8192)), 256, 0,
                           stream>>>(a);
  return hipGetLastError();
}

// Time in microseconds of a product of `groups` workgroups with `slabs` 64-deep slabs each, for depths of
// hundreds of slabs: a fixed part (first slab, outgoing rows) and one for each slab, which grows with the
// share of the CUs that multiply (256x256: 1.05 us with a few workgroups, 1.34 with 96, 1.6 with 192, 1.7
// with all).  The last, partial round counts with its own share.
double deep_cost(RowsTile tile, double groups, double slabs) {
  double slots = 256, fixed = 10.0, slab = 1.05, more = 0.65;   // 256x256
  switch (tile) {
    case kRows32: return rounds(groups, 256) * (4.5 + 0.7 * std::ceil(slabs / 8));
    case kRows32x128: return rounds(groups, 512) * (4.5 + 0.6 * std::ceil(slabs / 2));
    case kRows64: fixed = 2.2; slab = 0.22; more = 0.08; break;
    case kRows128: slots = 512; fixed = 4.0; slab = 0.6; more = 0.5; break;
    case kRows128x192: slots = 512; fixed = 5.0; slab = 0.75; more = 0.7; break;
    default: break;
  }
  const double whole = std::floor(groups / slots), rest = groups - whole * slots;
  return whole * (fixed + (slab + more) * slabs) +
         (rest > 0 ? fixed + (slab + more * rest / slots) * slabs : 0.0);
}

// Adding up `splits` planes of `bytes`: read in the join, written in the product, half of it hidden there.
double join_cost(int splits, double bytes) {
  return splits > 1 ? 5.0 + 1.5 * splits * bytes / 5.4e6 : 0.0;
}

// Tile and splits of dx's product: the least of these.  The depth is a piece of the vocabulary, so few rows
// leave most CUs idle for long without splits.  The planes of a split take at most 2.7e8 bytes, which bounds the
// workspace; the sweep went no further.  Us by tile/splits with the join, the choice first (rows x
// width, depth):
//    256 x  768, 16384   128/16        21   64/4  24   256/16 32   128/1 159   256/1  278
//    512 x  768, 50304   128/16        54   64/8  88   256/16 73   128/1 487   256/1  829
//   2048 x  768, 50304   128x192/8    165   128/4 196  256/8  183  128/1 565   256/1  943
//   8192 x 1024, 32768   256/2        450   128/1 556  128x192/4 584           256/1  760
//  16384 x  768, 21760   128x192/1    487   256/4 521  128/2  611  128/1 682   256/1  543
//  16384 x 1536, 16384   256/2        704   128x192/1 725          128/1 801   256/1  800
struct InputPlan {
  RowsTile tile;
  int splits;
};

InputPlan input_plan(int64_t rows, int64_t cols, int64_t depth) {
  const double slabs = (double)std::max<int64_t>(1, ceil64(depth, kBK));
  const double bytes = 4.0 * (double)rows * (double)cols;
  InputPlan best{kRows256, 1};
  double least = 0;
  for (RowsTile t : {kRows256, kRows128x192, kRows128, kRows64, kRows32x128, kRows32}) {
    const double tiles = (double)ceil64(rows, kTileRows[t]) * (double)ceil64(cols, kTileCols[t]);
    if (t != kRows256 && tiles > kMaxTileGrid) continue;
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
      const double each = std::ceil(slabs / splits), groups = tiles * splits;
      if (splits > 1 && (each < 8 || groups > kMaxTileGrid || splits * bytes > 2.7e8)) break;
      const double cost = deep_cost(t, groups, each) + join_cost(splits, bytes);
      if ((t == kRows256 && splits == 1) || cost < least) {
        best = {t, splits};
        least = cost;
      }
    }
  }
  return best;
}

template <typename T, bool QT>
hipError_t input_variant(const InputGrad& a, RowsTile tile, hipStream_t stream) {
  switch (tile) {
    case kRows32: return input_tiles<T, QT, 32, 32, 1, 1, 8, 2>(a, stream);
    case kRows32x128: return input_tiles<T, QT, 32, 128, 1, 4, 2, 4>(a, stream);
    case kRows64: return input_tiles<T, QT, 64, 64, 2, 2, 4, 4>(a, stream);
    case kRows128: return input_tiles<T, QT, 128, 128, 2, 2, 1, 2>(a, stream);
    case kRows128x192: return input_tiles<T, QT, 128, 192, 2, 2, 1, 2>(a, stream);
    default: return input_tiles<T, QT, 256, 256, 2, 4, 1, 2>(a, stream);
  }
}

template <typename T, int BM, int BN, int WM, int WN, int OCC>
hipError_t weight_side(const WeightGrad& a, hipStream_t stream) {
  using C = Tile<BM, BN, WM, WN, 1>;
  static std::atomic<uint64_t> configured{0};
  const int64_t tiles_i = ceil64(a.ni, BM), tiles_j = ceil64(a.nj, BN);
  hipError_t e = launch_lds(head_weight_kernel<T, BM, BN, WM, WN, OCC>, configured,
                            tiles_i * tiles_j * a.splits, C::kThreads, C::kLds, stream, a,
                            (int)tiles_i, (int)tiles_j);
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t pieces = a.ni * ceil64(a.nj, 8);
  head_planes_kernel<T><<<dim3((unsigned)std::min<int64_t>(ceil64(pieces, 256), 8192)), 256, 0,
                          stream>>>(a);
  return hipGetLastError();
}

// The same for dW, whose depth is the rows (at least 256 a split).  Its planes take at most 1.1e9 bytes, about what P
// does.
struct HeadWeightPlan {
  int side, splits;
};

HeadWeightPlan head_weight_plan(int64_t rows, int64_t entries, int64_t depth) {
  const double slabs = (double)std::max<int64_t>(1, ceil64(rows, kBK));
  const double bytes = 4.0 * (double)entries * (double)depth;
  HeadWeightPlan best{256, 1};
  double least = 0;
  for (RowsTile t : {kRows256, kRows128}) {
    const int side = kTileRows[t];
    const double tiles = (double)ceil64(entries, side) * (double)ceil64(depth, side);
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
      const double each = std::ceil(slabs / splits);
      if (splits > 1 && (each < 4 || splits * bytes > 1.1e9)) break;
      const double cost = deep_cost(t, tiles * splits, each) + join_cost(splits, bytes);
      if ((t == kRows256 && splits == 1) || cost < least) {
        best = {side, splits};
        least = cost;
      }
    }
  }
  return best;
}

// Columns of the vocabulary at a time: as many as give dW whole rounds of 256x256 tiles on the CUs, with
// up to 2^29 elements of P (1 GiB), but no fewer than 1024, since every piece reads and writes dx's sums: from 2^19
// rows on P has 1024 columns, 8 GiB at the most rows that a call takes.  Loss and gradients of 16384 rows, 768 x 50304, dx on 256x256 tiles: 5610 us by
// 21760 columns (255 tiles of dW), 5690 by 16384 (192), 5790 by 25344 (297).
int64_t piece_of(int64_t rows, int64_t vocab, int64_t depth) {
  const int64_t most =
      std::max<int64_t>(1024, (int64_t(1) << 29) / std::max<int64_t>(rows, 1) / 256 * 256);
  if (most >= vocab) return ceil8(vocab);
  const int64_t across = ceil64(depth, 256);
  for (int64_t m = most / 256 * across / 256; m >= 1; --m) {
    const int64_t cols = 256 * m / across * 256;
    if (cols <= most && cols >= 1024) return cols;
  }
  return most;
}

// The call's operands as the tiles read them, packed where that is needed, and P's scale.
hipError_t ready(const HeadCall& a, const HeadPlan& plan, char* ws, HeadProduct* p,
                 hipStream_t stream) {
  *p = HeadProduct{};
  p->x = a.x; p->ldx = a.ldx;
  p->w = a.w; p->ldw = a.w_kn ? a.vocab : a.depth;
  p->w_kn = a.w_kn; p->f16 = a.f16;
  p->rows = a.rows; p->depth = a.depth; p->vocab = a.vocab;
  p->targets = a.targets; p->wide = a.wide;
  HeadReady r{};
  int64_t pieces = 0;
  if (plan.x >= 0) {
    uint16_t* to = reinterpret_cast<uint16_t*>(ws + plan.x);
    r.copy[0] = {static_cast<const uint16_t*>(a.x), a.ldx, a.rows, a.depth, to, plan.ldx};
    p->x = to;
    p->ldx = plan.ldx;
    pieces += a.rows * (plan.ldx / 8);
  }
  if (plan.w >= 0) {
    uint16_t* to = reinterpret_cast<uint16_t*>(ws + plan.w);
    r.copy[1] = {static_cast<const uint16_t*>(a.w), p->ldw, a.w_kn ? a.depth : a.vocab, p->ldw, to,
                 plan.ldw};
    p->w = to;
    p->ldw = plan.ldw;
    pieces += r.copy[1].rows * (plan.ldw / 8);
  }
  if (plan.scale >= 0) {
    r.dloss = a.dloss;
    r.targets = a.targets; r.wide = a.wide; r.vocab = a.vocab;
    r.rows = a.rows;
    r.scale = reinterpret_cast<float*>(ws + plan.scale);
    p->scale = r.scale;
  }
  const int64_t grid = std::min<int64_t>(ceil64(pieces, kReadyThreads), 4096) + (r.scale ? 1 : 0);
  if (grid == 0) return hipSuccess;
  head_ready_kernel<<<dim3((unsigned)grid), kReadyThreads, 0, stream>>>(r);
  return hipGetLastError();
}

template <typename T>
hipError_t gradients(const HeadCall& a, const HeadPlan& plan, char* ws, hipStream_t stream) {
  HeadProduct p;
  hipError_t e = ready(a, plan, ws, &p, stream);
  if (e != hipSuccess) return e;
  p.lse = a.lse;
  p.dloss = a.dloss;
  p.p = ws + plan.p;
  for (int64_t v = 0; v < a.vocab; v += plan.piece) {
    const int64_t cols = std::min(plan.piece, a.vocab - v);
    p.first = v;
    p.cols = cols;
    e = launch_head_probabilities(p, stream);
    if (e != hipSuccess) return e;
    if (a.dx) {
      InputGrad g{};
      g.p = p.p;
      g.w = static_cast<const uint16_t*>(p.w) + (a.w_kn ? v : v * p.ldw);
      g.ldw = p.ldw;
      g.rows = a.rows; g.cols = a.depth; g.depth = (int)cols;
      g.sum = plan.dx >= 0 ? reinterpret_cast<float*>(ws + plan.dx) : nullptr;
      g.ldsum = ceil8(a.depth);
      const InputPlan tiles = input_plan(a.rows, a.depth, cols);
      g.splits = tiles.splits;
      g.planes = plan.dx_planes >= 0 ? reinterpret_cast<float*>(ws + plan.dx_planes) : nullptr;
      g.first = v == 0; g.last = v + cols == a.vocab;
      g.scale = p.scale;
      g.out = a.dx; g.ldout = a.lddx;
      e = a.w_kn ? input_variant<T, false>(g, tiles.tile, stream)
                 : input_variant<T, true>(g, tiles.tile, stream);
      if (e != hipSuccess) return e;
    }
    if (a.dw) {
      WeightGrad g{};
      const HeadWeightPlan tiles = head_weight_plan(a.rows, cols, a.depth);
      const int64_t at = a.w_kn ? v : v * a.depth;
      g.p = p.p;
      g.x = p.x; g.ldx = p.ldx;
      g.p_second = a.w_kn;
      g.ni = a.w_kn ? a.depth : (int)cols;
      g.nj = a.w_kn ? (int)cols : a.depth;
      g.rows = a.rows;
      g.splits = tiles.splits;
      g.planes = plan.planes >= 0 ? reinterpret_cast<float*>(ws + plan.planes) : nullptr;
      g.scale = p.scale;
      g.out = static_cast<char*>(a.dw) + at * (a.dw_f32 ? 4 : 2);
      g.ldout = a.w_kn ? a.vocab : a.depth;
      g.out_f32 = a.dw_f32;
      e = tiles.side == 256 ? weight_side<T, 256, 256, 2, 4, 2>(g, stream)
                            : weight_side<T, 128, 128, 2, 2, 2>(g, stream);
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace

HeadPlan head_plan(bool gradient, bool want_dx, bool want_dw, bool w_kn, bool f16, int in_place,
                   int64_t rows, int64_t vocab, int64_t depth) {
  HeadPlan plan{-1, -1, -1, -1, -1, -1, -1, -1, ceil8(depth), ceil8(w_kn ? vocab : depth), 0, 0};
  auto take = [&](int64_t bytes) {
    const int64_t at = (int64_t)plan.bytes;
    plan.bytes += (size_t)((bytes + 255) / 256 * 256);
    return at;
  };
  if (!(in_place & 1) || depth % 8) plan.x = take(rows * plan.ldx * 2);
  if (!(in_place & 2) || (w_kn ? vocab : depth) % 8) plan.w = take((w_kn ? depth : vocab) * plan.ldw * 2);
  if (!gradient) {
    plan.part = take(rows * head_stat_tiles(rows, vocab, (int)depth) * 8);
    return plan;
  }
  plan.piece = piece_of(rows, vocab, depth);
  if (f16) plan.scale = take(8);
  plan.p = take(rows * ceil64(plan.piece, 64) * 128);
  if (want_dx && plan.piece < vocab) plan.dx = take(rows * ceil8(depth) * 4);
  if (want_dx) {
    int splits = 1;
    for (int64_t cols : {std::min(plan.piece, vocab), vocab % plan.piece})   // and the last piece
      if (cols) splits = std::max(splits, input_plan(rows, depth, cols).splits);
    if (splits > 1) plan.dx_planes = take(splits * rows * ceil8(depth) * 4);
  }
  if (want_dw) {
    int64_t words = 0;
    for (int64_t cols : {std::min(plan.piece, vocab), vocab % plan.piece}) {   // and the last piece
      if (cols == 0) continue;
      const HeadWeightPlan t = head_weight_plan(rows, cols, depth);
      if (t.splits > 1)
        words = std::max(words, t.splits * (w_kn ? depth * ceil8(cols) : cols * ceil8(depth)));
    }
    if (words) plan.planes = take(words * 4);
  }
  return plan;
}

hipError_t launch_cross_entropy(const HeadCall& a, char* ws, hipStream_t stream) {
  const HeadPlan plan =
      head_plan(false, false, false, a.w_kn, a.f16, a.in_place, a.rows, a.vocab, a.depth);
  HeadProduct p;
  const hipError_t e = ready(a, plan, ws, &p, stream);
  if (e != hipSuccess) return e;
  p.cols = a.vocab;
  p.part = reinterpret_cast<float2*>(ws + plan.part);
  p.loss = a.loss;
  return launch_head_stats(p, a.lse, stream);
}

hipError_t launch_cross_entropy_grad(const HeadCall& a, char* ws, hipStream_t stream) {
  if (a.rows == 0) {
    const int64_t n = a.dw ? a.vocab * a.depth * (a.dw_f32 ? 2 : 1) : 0;   // in 16-bit words
    if (n == 0) return hipSuccess;
    head_zero_kernel<<<dim3((unsigned)std::min<int64_t>(ceil64(n, 256), 4096)), 256, 0, stream>>>(
        static_cast<uint16_t*>(a.dw), n);
    return hipGetLastError();
  }
  const HeadPlan plan = head_plan(true, a.dx != nullptr, a.dw != nullptr, a.w_kn, a.f16, a.in_place,
                                  a.rows, a.vocab, a.depth);
  return a.f16 ? gradients<f16>(a, plan, ws, stream) : gradients<bf16>(a, plan, ws, stream);
}

}  // namespace anvil
