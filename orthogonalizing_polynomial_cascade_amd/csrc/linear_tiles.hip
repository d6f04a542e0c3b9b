// The linear layers' products on LDS tiles (see linear.hip for what they compute): widths and pitches
// that are multiples of 8, 16-byte aligned pointers.
//
// Pipeline (gfx950):
//  * Slabs of BK = 64 k of both operands travel from memory straight into LDS (16 bytes a lane, no
//    registers in between) into two buffers.  Rows past the tile's group, columns past the width
//    and k past the depth get an offset outside the buffer's range, which loads zeros.
//  * A wave reads the fragments of one 16-deep k-step while the matrix cores work on the step
//    before it.  At the last step of a slab the waves meet: the next slab has landed (it was
//    requested a whole slab earlier), its first fragments are read, and among that step's
//    multiplies the slab after it is requested into the buffer just finished.
//  * K-contiguous operands are one ds_read_b128 per fragment and lane, K-major ones two transposing
//    reads; both layouts are swizzled against bank conflicts (mfma_slab.h).
//  * The multiplies take (Q, P), so a lane holds runs of four consecutive columns of one output row.
//    The rows leave through LDS (the buffer that is free by then), eight columns a lane, whole lines
//    an access, with bias, activation, derivative and residual applied on the way.
//  * What bounds it: the matrix cores are busy in 76% of the cycles at 8192^3 forward, 55% in the
//    weight gradient (1260 TFLOP/s with w [n, k], 1300 with w [k, n], 1100 in the weight gradient;
//    the barrier and the waits ahead of it take most of the rest, waves wait in 32% of their cycles),
//    LDS is busy in 29% and 21% of them and free of bank conflicts.  A slab of
//    64 k keeps the K-contiguous copies at whole 128-byte lines (rings of four 32-deep slabs were 8%
//    slower), and 256x256 tiles read 7.8 bytes a thousand operations where 128x128 ones read
//    15.6 (8192^3: 1080 TFLOP/s).  Copies placed between the multiplies of a slab's last k-step, all
//    without branches, gave 3-7% over copies ahead of them.
//  * KS > 1: KS sets of waves share a tile, each with its own part of the depth and its own buffers,
//    and the first set adds the others' sums in order: for calls with fewer tiles than CUs.
#include <algorithm>
#include <atomic>

#include "activation.h"
#include "tile_pipe.h"

namespace anvil {

namespace {

// The outgoing rows of a wave's block: rows r0 .. of a group that ends at `end`, the lane's columns
// c .. c + 7.  One copy of the code for each activation, so that what a launch runs of it stays
// within the instruction cache beside the multiplies (with the choice made at every element and
// everything unrolled it did not, and took longer than the multiplies of twelve slabs).
template <typename T, typename C, bool GRADIENT, int ACT>
__device__ __forceinline__ void rows_out(const RowsProduct& p,
                                         const f32x16_t (&acc)[C::kFM][C::kFN], char* stage,
                                         int64_t r0, int64_t end, int group, int c, int lane) {
  using S = OutStage<C::kWTN>;
  const bool inside_c = c < p.cols;
  float bias[8];
  if (!GRADIENT) {
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = 0.0f;
    if (p.bias && group >= 0 && inside_c) {
      const int64_t at = (int64_t)group * p.cols + c;
      if (p.bias_f32) load_vec<float, 8>(static_cast<const float*>(p.bias) + at, bias);
      else load_vec<T, 8>(static_cast<const T*>(p.bias) + at, bias);
    }
  }
  const int64_t first = r0 + S::row(0, lane);
  const int rows = inside_c ? (int)min(end - first, (int64_t)C::kWTM) : 0;   // below: row inside
  T* out = static_cast<T*>(p.out) + first * p.ldout + c;
  T* keep = static_cast<T*>(p.keep) + first * p.ldkeep + c;
  const T* aux = static_cast<const T*>(p.aux) + first * p.ldaux + c;
  const T* add = static_cast<const T*>(p.add) + first * p.ldadd + c;
  // the lane's pieces of the operands, 32 rows ahead
  u32x4_t aux_next[S::kPasses], add_next[S::kPasses];
  auto fetch = [&](int fm) {
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) {
      const int r = fm * 32 + i * S::kRows;
      if (GRADIENT) {
        aux_next[i] = u32x4_t{};
        if (r < rows) aux_next[i] = *reinterpret_cast<const u32x4_t*>(aux + r * p.ldaux);
      }
      if (p.add) {
        add_next[i] = u32x4_t{};
        if (r < rows) add_next[i] = *reinterpret_cast<const u32x4_t*>(add + r * p.ldadd);
      }
    }
  };
  fetch(0);
#pragma unroll
  for (int fm = 0; fm < C::kFM; ++fm) {
    S::put(stage, acc[fm], lane);
    u32x4_t aux_now[S::kPasses], add_now[S::kPasses];
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) {
      aux_now[i] = aux_next[i];
      add_now[i] = add_next[i];
    }
    if (fm + 1 < C::kFM) fetch(fm + 1);
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) {
      const int r = fm * 32 + i * S::kRows;
      const bool inside = r < rows;
      float v[8];
      S::get(stage, i, lane, v);
      if (GRADIENT) {
        float z[8];
        unpack8<T>(aux_now[i], z);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= act_slope(ACT, z[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += bias[e];
        if (p.keep && inside)
          *reinterpret_cast<u32x4_t*>(keep + r * p.ldkeep) = group < 0 ? u32x4_t{} : pack8<T>(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = act_value(ACT, v[e]);
      }
      if (p.add) {
        float a[8];
        unpack8<T>(add_now[i], a);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += a[e];
      }
      if (inside)
        *reinterpret_cast<u32x4_t*>(out + r * p.ldout) = group < 0 ? u32x4_t{} : pack8<T>(v);
    }
  }
}

template <typename T, typename C>
__device__ __forceinline__ void rows_epilogue(const RowsProduct& p,
                                              const f32x16_t (&acc)[C::kFM][C::kFN], char* stage,
                                              int64_t r0, int64_t end, int group, int c, int lane) {
  if (p.gradient && p.aux) {
    switch (p.act) {
      case kActRelu: return rows_out<T, C, true, kActRelu>(p, acc, stage, r0, end, group, c, lane);
      case kActRelu2: return rows_out<T, C, true, kActRelu2>(p, acc, stage, r0, end, group, c, lane);
      case kActGelu: return rows_out<T, C, true, kActGelu>(p, acc, stage, r0, end, group, c, lane);
      default: return rows_out<T, C, true, kActSilu>(p, acc, stage, r0, end, group, c, lane);
    }
  }
  // a gradient without an activation has neither bias nor kept preactivation
  switch (p.act) {
    case kActRelu: return rows_out<T, C, false, kActRelu>(p, acc, stage, r0, end, group, c, lane);
    case kActRelu2: return rows_out<T, C, false, kActRelu2>(p, acc, stage, r0, end, group, c, lane);
    case kActGelu: return rows_out<T, C, false, kActGelu>(p, acc, stage, r0, end, group, c, lane);
    case kActSilu: return rows_out<T, C, false, kActSilu>(p, acc, stage, r0, end, group, c, lane);
    default: return rows_out<T, C, false, kActNone>(p, acc, stage, r0, end, group, c, lane);
  }
}

template <typename T, bool QT, int BM, int BN, int WM, int WN, int KS, int OCC>
__global__ __launch_bounds__(WM * WN * KS * 64)
__attribute__((amdgpu_waves_per_eu(OCC)))
void rows_tile_kernel(RowsProduct p, int tiles_n) {
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
  const bool idle = row0 + wm * C::kWTM >= end;   // no row of the wave's block is there
  if (idle) pipe.attend();
  else pipe.template run<false>(acc, 0, none);
  if constexpr (KS > 1) {
    pipe.merge(kg, acc);
    if (kg > 0) return;
  }
  if (idle) return;
  rows_epilogue<T, C>(p, acc, pipe.spare() + wave * S::kBytes, row0 + wm * C::kWTM, end, group,
                      j0 + wn * C::kWTN + S::col(lane), lane);
}

// Split s of a group takes the s-th part of its
// rows (whole slabs).  Where a group's rows are split, its sums go as fp32 to plane s of the
// workspace: [splits][groups * pi * qj], then [splits][groups * width of dz].
template <typename T, int BM, int BN, int WM, int WN, int OCC>
__global__ __launch_bounds__(WM * WN * 64)
__attribute__((amdgpu_waves_per_eu(OCC)))
void weight_tile_kernel(WeightProduct p, float* ws, int splits, int tiles_i, int tiles_j) {
  using C = Tile<BM, BN, WM, WN, 1>;
  static_assert(C::kFM <= WN && C::kFN <= WM, "each wave sums one fragment at most");
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  // Each XCD takes an eighth of every group's tiles (not whole groups, which differ in length), the
  // longest group's first.
  const int tiles = tiles_i * tiles_j * splits;
  const int share = (tiles + 7) / 8;
  const int xcd = blockIdx.x % 8, at = blockIdx.x / 8;
  const int unit = xcd * share + at % share;
  if (unit >= tiles) return;
  int64_t begin, end;
  const int e = __builtin_amdgcn_readfirstlane(
      longest_first(p.groups, p.rows, at / share, &begin, &end));
  begin = uniform(begin);
  end = uniform(end);
  const int s = unit / (tiles_i * tiles_j);
  int ti, tj;
  banded(unit % (tiles_i * tiles_j), tiles_i, tiles_j, &ti, &tj);
  const int i0 = ti * BM, j0 = tj * BN;
  const int64_t part = ((end - begin + kBK - 1) / kBK + splits - 1) / splits * kBK;
  const int64_t k0 = min(begin + s * part, end), k1 = min(k0 + part, end);

  f32x16_t acc[C::kFM][C::kFN];
#pragma unroll
  for (int fm = 0; fm < C::kFM; ++fm)
#pragma unroll
    for (int fn = 0; fn < C::kFN; ++fn) acc[fm][fn] = f32x16_t{};
  float sums = 0.0f;
  const int sum = !p.db ? 0 : p.dz_is_q ? (ti == 0 ? 2 : 0) : (tj == 0 ? 1 : 0);
  Pipe<T, true, true, BM, BN, WM, WN, 1> pipe(smem, wave);
  pipe.begin(static_cast<const uint16_t*>(p.p) + k0 * p.ldp + i0, p.ldp, p.pi - i0,
             static_cast<const uint16_t*>(p.q) + k0 * p.ldq + j0, p.ldq, p.qj - j0, k1 - k0, 0);
  pipe.template run<true>(acc, sum, sums);

  const int wm = wave / WN, wn = wave % WN;
  const int width = p.dz_is_q ? p.qj : p.pi;
  const int64_t plane = (int64_t)p.groups.count * p.pi * p.qj;
  if (sum && (sum == 1 ? wn < C::kFM : wm < C::kFN)) {
    const int c = (sum == 1 ? i0 + wm * C::kWTM + wn * 32 : j0 + wn * C::kWTN + wm * 32) + lane;
    float* db = splits > 1 ? ws + splits * plane + (int64_t)s * p.groups.count * width : p.db;
    const float both = sums + __shfl_xor(sums, 32);
    if (lane < 32 && c < width) db[(int64_t)e * width + c] = both;
  }
  using S = OutStage<C::kWTN>;
  static_assert(C::kWaves * S::kBytes <= C::kStage, "the outgoing rows fit one buffer");
  char* stage = pipe.spare() + wave * S::kBytes;
  const int c = j0 + wn * C::kWTN + S::col(lane);
#pragma unroll
  for (int fm = 0; fm < C::kFM; ++fm) {
    S::put(stage, acc[fm], lane);
#pragma unroll
    for (int k = 0; k < S::kPasses; ++k) {
      const int i = i0 + wm * C::kWTM + fm * 32 + S::row(k, lane);
      float v[8];
      S::get(stage, k, lane, v);
      if (i >= p.pi || c >= p.qj) continue;
      const int64_t at = ((int64_t)e * p.pi + i) * p.qj + c;
      if (splits > 1) store_vec<float, 8>(ws + s * plane + at, v);
      else if (p.dw_f32) store_vec<float, 8>(static_cast<float*>(p.dw) + at, v);
      else *reinterpret_cast<u32x4_t*>(static_cast<T*>(p.dw) + at) = pack8<T>(v);
    }
  }
}

template <typename T, bool QT, int BM, int BN, int WM, int WN, int KS, int OCC>
hipError_t rows_tiles(const RowsProduct& a, hipStream_t stream) {
  using C = Tile<BM, BN, WM, WN, KS>;
  static std::atomic<uint64_t> configured{0};
  const int64_t tiles_m = row_tiles(a, BM), tiles_n = ceil64(a.cols, BN);
  // every XCD gets the same number of workgroups, whatever its share of partly filled tiles
  return launch_lds(rows_tile_kernel<T, QT, BM, BN, WM, WN, KS, OCC>, configured,
                    ceil64(tiles_m * tiles_n, 8) * 8 + 8,
                    C::kThreads, C::kLds, stream, a, (int)tiles_n);
}

template <typename T, bool QT>
hipError_t rows_variant(const RowsProduct& a, hipStream_t stream) {
  switch (rows_tile(a)) {
    case kRows32: return rows_tiles<T, QT, 32, 32, 1, 1, 8, 2>(a, stream);
    case kRows32x128: return rows_tiles<T, QT, 32, 128, 1, 4, 2, 4>(a, stream);
    case kRows64: return rows_tiles<T, QT, 64, 64, 2, 2, 4, 4>(a, stream);
    case kRows128: return rows_tiles<T, QT, 128, 128, 2, 2, 1, 2>(a, stream);
    default: return rows_tiles<T, QT, 256, 256, 2, 4, 1, 2>(a, stream);
  }
}

template <typename T, int BM, int BN, int WM, int WN, int OCC>
hipError_t weight_tiles(const WeightProduct& a, float* ws, int splits, hipStream_t stream) {
  using C = Tile<BM, BN, WM, WN, 1>;
  static std::atomic<uint64_t> configured{0};
  const int64_t tiles_i = ceil64(a.pi, BM), tiles_j = ceil64(a.qj, BN);
  return launch_lds(weight_tile_kernel<T, BM, BN, WM, WN, OCC>, configured,
                    ceil64(tiles_i * tiles_j * splits, 8) * 8 * a.groups.count, C::kThreads, C::kLds, stream, a, ws,
                    splits, (int)tiles_i, (int)tiles_j);
}

template <typename T>
hipError_t weight_variant(const WeightProduct& a, float* ws, int splits, hipStream_t stream) {
  if (weight_plan(a).side == 256) return weight_tiles<T, 256, 256, 2, 4, 2>(a, ws, splits, stream);
  return weight_tiles<T, 128, 128, 2, 2, 2>(a, ws, splits, stream);
}

}  // namespace

bool tiles_take_rows(const RowsProduct& a) {
  const RowsTile t = rows_tile(a);
  if (row_tiles(a, kTileRows[t]) * ceil64(a.cols, kTileCols[t]) + 16 > kMaxTileGrid) return false;
  return a.depth > 0 && multiple8(a.depth) && multiple8(a.cols) && multiple8(a.lda) &&
         multiple8(a.ldout) && wide_aligned(a.a) && wide_aligned(a.b) && wide_aligned(a.out) &&
         (!a.aux || (multiple8(a.ldaux) && wide_aligned(a.aux))) &&
         (!a.add || (multiple8(a.ldadd) && wide_aligned(a.add))) &&
         (!a.keep || (multiple8(a.ldkeep) && wide_aligned(a.keep)));
}

hipError_t launch_rows_tiles(const RowsProduct& a, hipStream_t stream) {
  if (a.f16)
    return a.b_kmajor ? rows_variant<f16, true>(a, stream) : rows_variant<f16, false>(a, stream);
  return a.b_kmajor ? rows_variant<bf16, true>(a, stream) : rows_variant<bf16, false>(a, stream);
}

bool tiles_take_weight(const WeightProduct& a) {
  const WeightPlan plan = weight_plan(a);
  if (ceil64(a.pi, plan.side) * ceil64(a.qj, plan.side) * a.groups.count * plan.splits + 8 * a.groups.count > kMaxTileGrid)
    return false;
  return multiple8(a.pi) && multiple8(a.qj) && multiple8(a.ldp) && multiple8(a.ldq) &&
         wide_aligned(a.p) && wide_aligned(a.q) && wide_aligned(a.dw);
}

int weight_tile_splits(const WeightProduct& a) { return weight_plan(a).splits; }

hipError_t launch_weight_tiles(const WeightProduct& a, float* ws, int splits, hipStream_t stream) {
  return a.f16 ? weight_variant<f16>(a, ws, splits, stream)
               : weight_variant<bf16>(a, ws, splits, stream);
}

}  // namespace anvil
