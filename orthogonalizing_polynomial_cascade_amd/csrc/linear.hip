// The linear layers that a bank's matrices belong to: products of activations with a weight matrix
// (or a stack of them, one per expert) with their epilogue, and the two gradient products.
//
//   rows product    out[r][c] = epilogue(sum_d a[r][d] b(c, d))      forward and input gradient
//   weight product  dw[i][j]  = sum_r p[r][i] q[r][j]                weight gradient (a bank's grad)
//
// Both are  C[i][j] = sum_k P(i, k) Q(j, k)  with fp32 accumulation on the matrix cores and one
// rounding at the end; an operand is "K-contiguous" (k runs along its rows in memory) or "K-major"
// (k runs down its rows).
//
// Groups (experts): rows are sorted by expert and the kernels read the row offsets themselves.  The
// offsets are taken as a running maximum clamped to [0, rows], so that every row has at most one
// owner and no access leaves the buffers whatever they hold; a row without an owner (before the
// first offset or past the last) gets an output row of zeros.
#include <algorithm>

#include "activation.h"
#include "any_pipe.h"

namespace anvil {

namespace {

// ---------------------------------------------------------------------------------------------
// The kernels for any width, pitch and alignment: tiles of SIDE x SIDE (64, or 128 where there are
// enough of them), four waves of F x F 32x32 fragments, operands through registers into LDS (the
// copies of linear_tiles.hip need 16-byte alignment).  Bound by the two barriers a slab, by the
// two-byte LDS writes of K-major operands and by an epilogue of single elements: 441 TFLOP/s at 4096 x
// 4097 x 4095 with w [n, k] and 365 with w [k, n], 220 and 275 in their weight gradients.  128x128 tiles
// of a K-major weight spill 8 registers, those of the weight gradient 4.  Slabs of 32 k, which wait for memory twice as often, and guarded loads of
// single elements at the edges took 1247 us for the first of these instead of 310.
// ---------------------------------------------------------------------------------------------

template <typename T, bool QT, int SIDE>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2)))
void any_rows_kernel(RowsProduct p, int tiles_n) {
  constexpr int F = SIDE / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  RowTiles<SIDE> tiles(p.groups, p.rows);
  for (int64_t tile = blockIdx.x; tile < (int64_t)tiles.total * tiles_n; tile += gridDim.x) {
    int64_t row0, end;
    int group;
    tiles.find((int)(tile / tiles_n), &row0, &end, &group);
    const int64_t j0 = (tile % tiles_n) * SIDE;
    const T* b = static_cast<const T*>(p.b) + (int64_t)(group < 0 ? 0 : group) * p.cols * p.depth;
    f32x16_t acc[F][F] = {};
    float none[F] = {};
    any_accumulate<T, false, QT, SIDE>(static_cast<const T*>(p.a), p.lda, row0, end, b,
                                       QT ? p.cols : p.depth, j0, p.cols, 0,
                                       group < 0 ? 0 : p.depth, acc, 0, none);
#pragma unroll
    for (int m = 0; m < F; ++m) {
      const int64_t r = row0 + ((wave >> 1) * F + m) * 32 + (lane & 31);
      if (r >= end) continue;
#pragma unroll
      for (int n = 0; n < F; ++n) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int64_t c =
              j0 + ((wave & 1) * F + n) * 32 + 8 * (i / 4) + 4 * (lane >> 5) + i % 4;
          if (c < p.cols) finish_element<T>(p, group, r, c, acc[m][n][i]);
        }
      }
    }
  }
}

// Weight product, tile by tile of [groups][splits][tiles]: split s of a group takes the s-th part
// of its rows (a multiple of kAnyDepth).  With one split the tile goes to dw and db; with more, as
// fp32 to plane s of the workspace, [splits][groups * pi * qj] and then [splits][groups * width].
template <typename T, int SIDE>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2)))
void any_weight_kernel(WeightProduct p, float* ws, int splits, int tiles_i, int tiles_j) {
  constexpr int F = SIDE / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t tiles = (int64_t)tiles_i * tiles_j;
  const int groups = p.groups.count;
  const int width = p.dz_is_q ? p.qj : p.pi;
  const int64_t plane = (int64_t)groups * p.pi * p.qj;
  for (int64_t w = blockIdx.x; w < tiles * splits * groups; w += gridDim.x) {
    const int64_t t = w % tiles;
    const int s = (int)(w / tiles % splits);
    const int e = (int)(w / tiles / splits);
    const int64_t i0 = t / tiles_j * SIDE, j0 = t % tiles_j * SIDE;
    int64_t begin, end;
    group_rows(p.groups, p.rows, e, &begin, &end);
    const int64_t part =
        ((end - begin + splits - 1) / splits + kAnyDepth - 1) / kAnyDepth * kAnyDepth;
    const int64_t k0 = std::min(begin + s * part, end), k1 = std::min(k0 + part, end);
    const int sum = !p.db ? 0
                    : p.dz_is_q ? (i0 == 0 && wave < 2 ? 2 : 0)
                                : (j0 == 0 && (wave & 1) == 0 ? 1 : 0);
    f32x16_t acc[F][F] = {};
    float sums[F] = {};
    any_accumulate<T, true, true, SIDE>(static_cast<const T*>(p.p), p.ldp, i0, p.pi,
                                        static_cast<const T*>(p.q), p.ldq, j0, p.qj, k0, k1, acc,
                                        sum, sums);
    if (sum) {
      float* db = splits > 1 ? ws + splits * plane + (int64_t)s * groups * width : p.db;
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const float both = sums[f] + __shfl_xor(sums[f], 32);
        const int64_t c = (p.dz_is_q ? j0 + ((wave & 1) * F + f) * 32
                                     : i0 + ((wave >> 1) * F + f) * 32) + lane;
        if (lane < 32 && c < width) db[(int64_t)e * width + c] = both;
      }
    }
#pragma unroll
    for (int m = 0; m < F; ++m) {
      const int64_t i = i0 + ((wave >> 1) * F + m) * 32 + (lane & 31);
      if (i >= p.pi) continue;
#pragma unroll
      for (int n = 0; n < F; ++n) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int64_t j =
              j0 + ((wave & 1) * F + n) * 32 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
          if (j >= p.qj) continue;
          const int64_t at = ((int64_t)e * p.pi + i) * p.qj + j;
          if (splits > 1) ws[s * plane + at] = acc[m][n][r];
          else if (p.dw_f32) static_cast<float*>(p.dw)[at] = acc[m][n][r];
          else static_cast<T*>(p.dw)[at] = from_f32<T>(acc[m][n][r]);
        }
      }
    }
  }
}

// Adds the splits' planes in order: dw (n words, then the nb words of db, which has planes of its own
// behind dw's).  Bound by memory: four words a lane and access; seven planes of 2816 x 768 in 10.4 us
// (6.6 TB/s, mostly from the caches that the planes were just written to).
template <typename O>
__global__ __launch_bounds__(256) void join_kernel(const float* ws, int splits, int64_t n, O* dw,
                                                   int64_t nb, float* db) {
  const int64_t wide = n / 4;   // n is a multiple of 4, or the last words go one by one
  const int64_t step = (int64_t)gridDim.x * 256;
  const int64_t me = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (int64_t i = me; i < wide; i += step) {
    float s[4];
    load_vec<float, 4>(ws + i * 4, s);
#pragma unroll 2
    for (int k = 1; k < splits; ++k) {
      float v[4];
      load_vec<float, 4>(ws + k * n + i * 4, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += v[e];
    }
    store_vec<O, 4>(dw + i * 4, s);
  }
  for (int64_t i = wide * 4 + me; i < n; i += step) {
    float s = ws[i];
    for (int k = 1; k < splits; ++k) s += ws[k * n + i];
    dw[i] = from_f32<O>(s);
  }
  const float* wb = ws + splits * n;
  for (int64_t i = me; i < nb; i += step) {
    float s = wb[i];
    for (int k = 1; k < splits; ++k) s += wb[k * nb + i];
    db[i] = s;
  }
}


template <typename T, int SIDE>
hipError_t launch_rows_side(const RowsProduct& a, hipStream_t stream) {
  const int64_t tiles_m = ceil64(a.rows, SIDE) + (a.groups.offsets ? a.groups.count + 1 : 0);
  const int tiles_n = (int)ceil64(a.cols, SIDE);
  if (a.b_kmajor)
    any_rows_kernel<T, true, SIDE><<<grid_for(tiles_m * tiles_n), 256, 0, stream>>>(a, tiles_n);
  else
    any_rows_kernel<T, false, SIDE><<<grid_for(tiles_m * tiles_n), 256, 0, stream>>>(a, tiles_n);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_rows_t(const RowsProduct& a, hipStream_t stream) {
  return any_wide_tiles(a) ? launch_rows_side<T, 128>(a, stream) : launch_rows_side<T, 64>(a, stream);
}

struct AnyPlan {
  int side, splits;
};

// Splits of each group's rows: enough workgroups for two rounds of two (128x128) or four (64x64) a
// CU while a split keeps at least 512 rows on average.  Us by side/splits, the choice first:
//    600 rows,  131 x 333    64/1   17.3   64/2  12.9   128/2 21.4
//   2048 rows, 1031 x 769    64/4   38.0   64/1  45.9   64/2  37.4   128/4 35.9
//   4096 rows, 1031 x 769   128/8   56.2   128/4 49.8   128/1 140.1   64/4 59.3
//   4096 rows, 2049 x 769   128/8   93.2   128/4 73.3   128/2 80.7    64/4 92.4
//  32768 rows,  131 x 333   128/64  81.1   64/32 67.0   64/64 83.2   128/32 77.5
//   4096 rows, 4097 x 4095 128/1  643.9   128/2 584.0   64/1 732.2
// Half as many splits would serve most of these better, by a tenth to a quarter.
AnyPlan any_weight_plan(const WeightProduct& a) {
  const int64_t most = std::max<int64_t>(1, a.rows / a.groups.count / 512);
  auto splits = [&](int side, int64_t slots) {
    const int64_t tiles = ceil64(a.pi, side) * ceil64(a.qj, side) * a.groups.count;
    return std::min({std::max<int64_t>(1, slots / tiles), most, int64_t(64)});
  };
  const int64_t wide = splits(128, 1024);
  if (wide * ceil64(a.pi, 128) * ceil64(a.qj, 128) * a.groups.count >= kManyTiles)
    return {128, (int)wide};
  return {64, (int)splits(64, 2048)};
}

template <typename T, int SIDE>
hipError_t launch_weight_side(const WeightProduct& a, float* ws, int splits, hipStream_t stream) {
  const int tiles_i = (int)ceil64(a.pi, SIDE), tiles_j = (int)ceil64(a.qj, SIDE);
  const int64_t work = (int64_t)tiles_i * tiles_j * splits * a.groups.count;
  any_weight_kernel<T, SIDE><<<grid_for(work), 256, 0, stream>>>(a, ws, splits, tiles_i, tiles_j);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_weight_t(const WeightProduct& a, float* ws, hipStream_t stream) {
  const bool tiled = tiles_take_weight(a);
  const AnyPlan plan = any_weight_plan(a);
  const int splits = tiled ? weight_tile_splits(a) : plan.splits;
  hipError_t e;
  if (tiled) e = launch_weight_tiles(a, ws, splits, stream);
  else if (plan.side == 128) e = launch_weight_side<T, 128>(a, ws, splits, stream);
  else e = launch_weight_side<T, 64>(a, ws, splits, stream);
  if (e != hipSuccess || splits == 1) return e;
  const int64_t n = (int64_t)a.groups.count * a.pi * a.qj;
  const int64_t nb = a.db ? (int64_t)a.groups.count * (a.dz_is_q ? a.qj : a.pi) : 0;
  const unsigned grid = (unsigned)std::min<int64_t>(ceil64(n, 1024), 4096);
  if (a.dw_f32)
    join_kernel<float><<<grid, 256, 0, stream>>>(ws, splits, n, static_cast<float*>(a.dw), nb, a.db);
  else
    join_kernel<T><<<grid, 256, 0, stream>>>(ws, splits, n, static_cast<T*>(a.dw), nb, a.db);
  return hipGetLastError();
}

// Bound by memory: 32768 x 2816 bf16 in 99 us (5.6 TB/s), with gelu as with relu2.
template <typename T>
__global__ __launch_bounds__(256) void activation_grad_kernel(const T* dy, int64_t lddy, const T* z,
                                                              int64_t ldz, int act, T* dz,
                                                              int64_t lddz, int64_t rows, int cols) {
  const int pieces = (cols + 7) / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * pieces;
       i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / pieces;
    const int c = (int)(i % pieces) * 8;
    if (c + 8 <= cols) {
      float d[8], v[8];
      load_vec<T, 8>(dy + r * lddy + c, d);
      load_vec<T, 8>(z + r * ldz + c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] *= act_slope(act, v[e]);
      store_vec<T, 8>(dz + r * lddz + c, d);
    } else {
      for (int e = c; e < cols; ++e)
        dz[r * lddz + e] =
            from_f32<T>(to_f32(dy[r * lddy + e]) * act_slope(act, to_f32(z[r * ldz + e])));
    }
  }
}

}  // namespace

hipError_t launch_rows_product(const RowsProduct& a, hipStream_t stream) {
  if (tiles_take_rows(a)) return launch_rows_tiles(a, stream);
  return a.f16 ? launch_rows_t<f16>(a, stream) : launch_rows_t<bf16>(a, stream);
}

// The larger of what the two kinds of kernels need: which of them runs depends on alignment too.
size_t weight_product_words(const WeightProduct& a) {
  int splits = any_weight_plan(a).splits;
  if (a.pi % 8 == 0 && a.qj % 8 == 0) splits = std::max(splits, weight_tile_splits(a));
  if (splits == 1) return 0;
  return (size_t)splits * a.groups.count *
         ((size_t)a.pi * a.qj + (a.dz_is_q ? (size_t)a.qj : (size_t)a.pi));
}

hipError_t launch_weight_product(const WeightProduct& a, float* ws, hipStream_t stream) {
  return a.f16 ? launch_weight_t<f16>(a, ws, stream) : launch_weight_t<bf16>(a, ws, stream);
}

hipError_t launch_activation_grad(const void* dy, int64_t lddy, const void* z, int64_t ldz, int act,
                                  void* dz, int64_t lddz, bool f16_type, int64_t rows, int cols,
                                  hipStream_t stream) {
  const unsigned grid = (unsigned)std::min<int64_t>(ceil64(rows * ((cols + 7) / 8), 256), 16384);
  if (f16_type)
    activation_grad_kernel<f16><<<grid, 256, 0, stream>>>(
        static_cast<const f16*>(dy), lddy, static_cast<const f16*>(z), ldz, act,
        static_cast<f16*>(dz), lddz, rows, cols);
  else
    activation_grad_kernel<bf16><<<grid, 256, 0, stream>>>(
        static_cast<const bf16*>(dy), lddy, static_cast<const bf16*>(z), ldz, act,
        static_cast<bf16*>(dz), lddz, rows, cols);
  return hipGetLastError();
}

}  // namespace anvil
