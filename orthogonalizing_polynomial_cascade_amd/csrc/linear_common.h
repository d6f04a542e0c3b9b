// Shared by the linear layers' kernels: the matrix instruction of each element type and the groups
// of rows.
#pragma once

#include "device_common.h"
#include "launchers.h"
#include "scalar_types.h"

namespace anvil {

template <typename T>
struct Mfma;
template <>
struct Mfma<bf16> {
  typedef bf16x8_t vec;
  __device__ static __forceinline__ f32x16_t run(vec a, vec b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  __device__ static __forceinline__ f32x4_t run16(vec a, vec b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mfma<f16> {
  typedef f16 vec __attribute__((ext_vector_type(8)));
  __device__ static __forceinline__ f32x16_t run(vec a, vec b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  __device__ static __forceinline__ f32x4_t run16(vec a, vec b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

// Sums over k of a 32-row fragment (lane l: row l % 32, k 8 (l / 32) .. + 7) by a 16x16x32 multiply,
// four registers instead of a fragment's sixteen.  That instruction takes the lane's column as
// l % 16 and its k group as l / 16, so rows r and r + 16 of the fragment meet in one column, in k
// groups of different parity: row 0 of the other operand holds ones for the even groups, row 1 for
// the odd ones.  Sums of rows r and 16 + r arrive in entries 0 and 1 of lane r < 16.
template <typename T>
__device__ __forceinline__ typename Mfma<T>::vec row_sum_selector(int lane) {
  typename Mfma<T>::vec v;
  const float x = lane % 16 == (lane / 16) % 2 ? 1.0f : 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = from_f32<T>(x);
  return v;
}

// Offset j of the groups, clamped to [0, rows] (not yet a running maximum).
__device__ __forceinline__ int64_t raw_offset(const Groups& g, int j, int64_t rows) {
  int64_t v = g.wide ? static_cast<const int64_t*>(g.offsets)[j]
                     : (int64_t)static_cast<const int32_t*>(g.offsets)[j];
  return v < 0 ? 0 : (v > rows ? rows : v);
}

__device__ __forceinline__ int64_t wave_max(int64_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const int64_t u = __shfl_xor(v, o);
    v = u > v ? u : v;
  }
  return v;
}

// Rows [*begin, *end) of group e: every wave looks at the offsets up to e + 1.
__device__ __forceinline__ void group_rows(const Groups& g, int64_t rows, int e, int64_t* begin,
                                           int64_t* end) {
  if (!g.offsets) {
    *begin = 0;
    *end = rows;
    return;
  }
  int64_t lo = 0;
  for (int j = threadIdx.x & 63; j <= e; j += 64) {
    const int64_t v = raw_offset(g, j, rows);
    lo = v > lo ? v : lo;
  }
  lo = wave_max(lo);
  const int64_t hi = raw_offset(g, e + 1, rows);
  *begin = lo;
  *end = hi > lo ? hi : lo;
}

__device__ __forceinline__ int scan_max(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o);
    if (lane >= o && u > v) v = u;
  }
  return v;
}
__device__ __forceinline__ int scan_sum(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The rows in tiles of TILE, group by group; rows without an owner form two groups of their own,
// before the first and after the last.  Segment s = 0 .. count + 1 spans bound(s) .. bound(s + 1):
// bound(0) = 0, bound(s) = the running maximum of the offsets up to s - 1, bound(count + 2) = rows.
// A wave looks at 64 segments at a time, one a lane.
template <int TILE>
struct RowTiles {
  const Groups& g;
  int rows, lane;
  int lo, hi, upto;   // the lane's segment of the current chunk, tiles up to and with it
  int start, done;    // bound at the next chunk's first segment, tiles before the next chunk
  int total;          // tiles in all

  __device__ __forceinline__ void chunk(int s0) {
    const int s = s0 + lane;
    int v = s <= g.count ? (int)raw_offset(g, s, rows) : rows;
    v = v > start ? v : start;
    hi = scan_max(v, lane);
    lo = __shfl_up(hi, 1);
    if (lane == 0) lo = start;
    upto = done + scan_sum((int)(((unsigned)(hi - lo) + TILE - 1) / TILE), lane);
    start = __shfl(hi, 63);
    done = __shfl(upto, 63);
  }
  __device__ __forceinline__ RowTiles(const Groups& g_, int64_t rows_)
      : g(g_), rows((int)rows_), lane((int)(threadIdx.x & 63)), start(0), done(0) {
    if (!g.offsets) {
      total = (int)(((unsigned)rows + TILE - 1) / TILE);
      return;
    }
    for (int s0 = 0; s0 < g.count + 2; s0 += 64) chunk(s0);
    total = done;
  }
  // Tile t < total: its first row, the end of its group's rows, its group (-1: no owner).
  __device__ __forceinline__ void find(int t, int64_t* row0, int64_t* end, int* group) {
    if (!g.offsets) {
      *row0 = (int64_t)t * TILE;
      *end = rows;
      *group = 0;
      return;
    }
    int s0 = 0;
    if (g.count + 2 > 64) {   // several chunks: walk over them again
      start = done = 0;
      for (;; s0 += 64) {
        chunk(s0);
        if (t < done) break;
      }
    }
    const int who = __ffsll((unsigned long long)__ballot(upto > t)) - 1;
    const int left = __shfl(upto, who) - t;    // tiles from t to the segment's end
    const int first = __shfl(lo, who), last = __shfl(hi, who);
    const int tiles = (int)(((unsigned)(last - first) + TILE - 1) / TILE);
    *row0 = first + (int64_t)(tiles - left) * TILE;
    *end = last;
    const int seg = s0 + who;
    *group = seg == 0 || seg > g.count ? -1 : seg - 1;
  }
};

// The group at place j when the groups are taken from the one with the most rows down (in their own
// order from 65 groups on).  Work on the long groups starts first, so that the short ones fill up
// the end.
__device__ __forceinline__ int longest_first(const Groups& g, int64_t rows, int j) {
  if (!g.offsets || g.count > 64) return j;
  const int lane = threadIdx.x & 63;
  const int mine = lane <= g.count ? (int)raw_offset(g, lane, rows) : 0;
  const int bound = scan_max(mine, lane);
  int next = __shfl_down(bound, 1);
  if (lane == 63) {   // the 64th group's end is the 65th offset
    const int v = g.count == 64 ? (int)raw_offset(g, 64, rows) : bound;
    next = v > bound ? v : bound;
  }
  const int size = lane < g.count ? next - bound : -1;
  int rank = 0;
  for (int f = 0; f < g.count; ++f) {
    const int other = __builtin_amdgcn_readlane(size, f);
    rank += other > size || (other == size && f < lane) ? 1 : 0;
  }
  return __ffsll((unsigned long long)__ballot(lane < g.count && rank == j)) - 1;
}

// linear_tiles.hip: the tiled kernels, for widths and pitches that are multiples of 8 and pointers
// of 16-byte alignment (tiles_take_*), with their launches.
bool tiles_take_rows(const RowsProduct& a);
hipError_t launch_rows_tiles(const RowsProduct& a, hipStream_t stream);
bool tiles_take_weight(const WeightProduct& a);
hipError_t launch_weight_tiles(const WeightProduct& a, float* ws, int splits, hipStream_t stream);
// Splits of each group's rows that the tiled weight product makes (by sizes alone).
int weight_tile_splits(const WeightProduct& a);

}  // namespace anvil
