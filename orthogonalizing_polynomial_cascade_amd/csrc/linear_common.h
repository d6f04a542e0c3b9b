// Shared by the linear layers' kernels: the matrix instruction of each element type and the groups
// of rows.
#pragma once

#include "activation.h"
#include "device_common.h"
#include "launchers.h"
#include "scalar_types.h"

namespace anvil {

inline int64_t ceil64(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename T>
struct Mfma;
template <>
struct Mfma<bf16> {
  typedef bf16x8_t vec;
  __device__ static __forceinline__ f32x16_t run(vec a, vec b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mfma<f16> {
  typedef f16 vec __attribute__((ext_vector_type(8)));
  __device__ static __forceinline__ f32x16_t run(vec a, vec b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};

// s plus a lane's eight elements of a 32-row fragment (lane l: row l % 32, k 8 (l / 32) .. + 7), by the
// two-element dot products of the vector unit with ones: lanes l and l + 32 together hold the row's
// sum over k.  Every lane adds its own row only.  A matrix instruction that sums two rows at once has
// to tell them apart by zeros, and 0 * inf is NaN: one infinite gradient would spoil another column.
// Weight gradients in us with that instruction and with these: 517 x 512 x 4096 fp16 13.8 and 13.6,
// 32768 x 768 x 2816 163 and 163, 4096^3 131 and 128, 4096 x 4097 x 4095 623 and 622.
__device__ __forceinline__ float add8(Mfma<bf16>::vec v, float s) {
  typedef bf16 pair_t __attribute__((ext_vector_type(2)));
  const pair_t one = {from_f32<bf16>(1.0f), from_f32<bf16>(1.0f)};
#pragma unroll
  for (int e = 0; e < 8; e += 2) s = __builtin_amdgcn_fdot2_f32_bf16(pair_t{v[e], v[e + 1]}, one, s, false);
  return s;
}
__device__ __forceinline__ float add8(Mfma<f16>::vec v, float s) {
  typedef f16 pair_t __attribute__((ext_vector_type(2)));
  const pair_t one = {from_f32<f16>(1.0f), from_f32<f16>(1.0f)};
#pragma unroll
  for (int e = 0; e < 8; e += 2) s = __builtin_amdgcn_fdot2(pair_t{v[e], v[e + 1]}, one, s, false);
  return s;
}

// add8 of one of several fragments between which a wave chooses; `which` is a constant (an unrolled
// loop's), another one for each.  The empty block keeps the choices apart: merged into one sum, the
// compiler moves the chosen fragment through other registers first, behind the multiplies that still
// read them.
template <typename V>
__device__ __forceinline__ void add8_of(int which, V v, float& s) {
  s = add8(v, s);
  asm volatile("" : "+v"(s) : "n"(which));
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
// Whole tiles come first, in the order of the rows; then the segments' last, partly filled ones
// (more than half full, then the others), whose shorter work evens out the end of a launch.  A
// wave looks at 64 segments at a time, one a lane; with more than 62 groups the tiles keep the
// order of the rows.
template <int TILE>
struct RowTiles {
  const Groups& g;
  int rows, lane;
  int lo, hi, upto;   // the lane's segment of the current chunk; tiles up to and with it (whole
                      // ones where the partly filled ones come last)
  int start, done;    // bound at the next chunk's first segment, tiles before the next chunk
  int whole, total;   // whole tiles, all tiles
  uint64_t large, small;   // segments whose last tile is more than half full, or less

  __device__ __forceinline__ bool sorted() const { return g.count + 2 <= 64; }

  __device__ __forceinline__ void chunk(int s0, bool round_up) {
    const int s = s0 + lane;
    int v = s <= g.count ? (int)raw_offset(g, s, rows) : rows;
    v = v > start ? v : start;
    hi = scan_max(v, lane);
    lo = __shfl_up(hi, 1);
    if (lane == 0) lo = start;
    upto = done + scan_sum((int)(((unsigned)(hi - lo) + (round_up ? TILE - 1 : 0)) / TILE), lane);
    start = __shfl(hi, 63);
    done = __shfl(upto, 63);
  }
  __device__ __forceinline__ RowTiles(const Groups& g_, int64_t rows_)
      : g(g_), rows((int)rows_), lane((int)(threadIdx.x & 63)), start(0), done(0), large(0), small(0) {
    if (!g.offsets) {
      whole = rows / TILE;
      total = whole + (rows % TILE ? 1 : 0);
    } else if (sorted()) {
      chunk(0, false);
      const int rest = (hi - lo) % TILE;
      large = __ballot(rest > TILE / 2);
      small = __ballot(rest > 0 && rest <= TILE / 2);
      whole = done;
      total = done + __popcll(large) + __popcll(small);
    } else {
      for (int s0 = 0; s0 < g.count + 2; s0 += 64) chunk(s0, true);
      whole = total = done;
    }
  }
  // Tile t < total: its first row, the end of its group's rows, its group (-1: no owner).
  __device__ __forceinline__ void find(int t, int64_t* row0, int64_t* end, int* group) {
    if (!g.offsets) {
      *row0 = (int64_t)t * TILE;
      *end = rows;
      *group = 0;
      return;
    }
    int s0 = 0, who;
    bool tail = false;
    if (sorted()) {
      if (t < whole) {
        who = __ffsll((unsigned long long)__ballot(upto > t)) - 1;
      } else {
        tail = true;
        int nth = t - whole;
        uint64_t in = large;
        if (nth >= __popcll(large)) {
          nth -= __popcll(large);
          in = small;
        }
        const uint64_t below = lane == 0 ? 0 : in << (64 - lane);
        who = __ffsll((unsigned long long)__ballot((in >> lane & 1) && __popcll(below) == nth)) - 1;
      }
    } else {   // several chunks: walk over them again
      start = done = 0;
      for (;; s0 += 64) {
        chunk(s0, true);
        if (t < done) break;
      }
      who = __ffsll((unsigned long long)__ballot(upto > t)) - 1;
    }
    const int first = __shfl(lo, who), last = __shfl(hi, who), through = __shfl(upto, who);
    const unsigned span = (unsigned)(last - first);
    const int tiles = (int)((span + (sorted() ? 0 : TILE - 1)) / TILE);
    *row0 = first + (int64_t)(tail ? tiles : tiles - (through - t)) * TILE;
    *end = last;
    const int seg = s0 + who;
    *group = seg == 0 || seg > g.count ? -1 : seg - 1;
  }
};

// The group at place j when the groups are taken from the one with the most rows down (in their own
// order from 65 groups on), and its rows.  Work on the long groups starts first, so that the short
// ones fill up the end.
__device__ __forceinline__ int longest_first(const Groups& g, int64_t rows, int j, int64_t* begin,
                                             int64_t* end) {
  if (!g.offsets || g.count > 64) {
    group_rows(g, rows, j, begin, end);
    return j;
  }
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
  const int e = __ffsll((unsigned long long)__ballot(lane < g.count && rank == j)) - 1;
  *begin = __shfl(bound, e);
  *end = __shfl(next, e);
  return e;
}

// Epilogue of one element: sum over the depth in, output (and kept preactivation) out.
template <typename T>
__device__ __forceinline__ void finish_element(const RowsProduct& p, int group, int64_t r, int64_t c,
                                               float z) {
  T* out = static_cast<T*>(p.out) + r * p.ldout + c;
  T* keep = static_cast<T*>(p.keep) + r * p.ldkeep + c;
  if (group < 0) {
    if (p.keep) *keep = from_f32<T>(0.0f);
    *out = from_f32<T>(0.0f);
    return;
  }
  if (p.gradient) {
    if (p.aux) z *= act_slope(p.act, to_f32(static_cast<const T*>(p.aux)[r * p.ldaux + c]));
  } else {
    if (p.bias) {
      const int64_t at = (int64_t)group * p.cols + c;
      z += p.bias_f32 ? static_cast<const float*>(p.bias)[at]
                      : to_f32(static_cast<const T*>(p.bias)[at]);
    }
    if (p.keep) *keep = from_f32<T>(z);
    z = act_value(p.act, z);
  }
  if (p.add) z += to_f32(static_cast<const T*>(p.add)[r * p.ldadd + c]);
  *out = from_f32<T>(z);
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
