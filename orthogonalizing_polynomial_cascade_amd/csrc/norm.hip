// Layer norm over the last axis and its backward pass.
//
//   forward    mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//              h = (x - mean) rstd,  y = h w + b
//   backward   g = dy w,  dx = rstd (g - mean(g) - h mean(g h))
//              dw = sum over rows of dy h,  db = sum over rows of dy
//
// All sums are fp32; the variance is taken about the mean in a second pass over the row's
// registers (the one-pass form sum x^2 - C mean^2 loses every digit when the mean is large beside
// the deviation).  Outputs of 16 bits are rounded once.
//
// Both passes are bound by memory: forward reads x and writes y, backward reads dy and x and
// writes dx, one pass each.  A row lives in the registers of one wave (up to 2048 columns) or of
// one workgroup of 256 lanes (up to 8192); longer rows are read again from memory for each step.
// A wave walks over rows with weight and bias in registers and the next row on its way while it
// works on this one.  In the backward pass it also keeps its columns' sums of dy h and dy; the
// workgroup (one or two to a CU, see norm_grad_blocks) joins its waves' sums in LDS and leaves one
// partial row, and a second launch adds the partial rows in a fixed order (no atomics: the same bits on
// every run).  Times with that launch, us:
//                     forward                backward
//   65536 x 768  bf16  35.5 (5.7 TB/s)         58 (5.2 TB/s; 78 with a row to each wave at a time and
//                                              1024 partial rows)
//   65536 x 768  fp32  81   (5.0)             120 (5.0)
//   16384 x 2048 bf16  23.4 (5.7)              42 (4.8)
//   16384 x 2048 fp32  43.5 (6.2)             107 (3.8)
//    4099 x 1601 fp16  13.1 (2.0)              31 (1.3)
//    4096 x 8192 bf16  23.7 (5.7)              56 (3.6)
//    4096 x 8192 fp32  43.7 (6.1)             138 (2.9)
//    1000 x 20000 bf16 44   (1.8)              80 (1.5)
// Four pieces of a row a lane (1025 to 2048 and 4097 to 8192 columns) are too many for the backward
// pass: x, dy, h, g, the weight, two sums and the next row do not fit 256 registers, and the compiler
// spills 22 to 167 of them with 16-bit types and 283 to 347 with fp32, which is what keeps these widths
// further from the memory's rate than the others.
#include <algorithm>

#include "device_common.h"
#include "launchers.h"
#include "scalar_types.h"

namespace anvil {

namespace {

constexpr int kVec = 8;   // consecutive columns of one lane

// Eight consecutive columns of a row as they lie in memory, read with wide accesses at whatever
// alignment the row starts; columns at or past the width are 0.
template <typename T>
struct Raw {
  T t[kVec];
  __device__ __forceinline__ void load(const T* row, int c, int cols) {
    if (c + kVec <= cols) {
      __builtin_memcpy(t, row + c, sizeof(t));
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) t[e] = c + e < cols ? row[c + e] : from_f32<T>(0.0f);
    }
  }
  // The width is a multiple of kVec: all of the columns are there or none.
  __device__ __forceinline__ void load_even(const T* row, int c, int cols) {
    if (c < cols) {
      __builtin_memcpy(t, row + c, sizeof(t));
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) t[e] = from_f32<T>(0.0f);
    }
  }
  __device__ __forceinline__ void get(float v[kVec]) const {
#pragma unroll
    for (int e = 0; e < kVec; ++e) v[e] = to_f32(t[e]);
  }
};

template <typename T>
__device__ __forceinline__ void load8(const T* row, int c, int cols, float v[kVec]) {
  Raw<T> r;
  r.load(row, c, cols);
  r.get(v);
}

template <typename T>
__device__ __forceinline__ void store8(T* row, int c, int cols, const float v[kVec]) {
  if (c + kVec <= cols) {
    store_vec<T, kVec>(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      if (c + e < cols) row[c + e] = from_f32<T>(v[e]);
  }
}

// Eight columns of the weight or bias (fp32 or T), or a constant where the pointer is null.
template <typename T>
__device__ __forceinline__ void load_param(const void* p, bool f32, int c, int cols, float fill,
                                           float v[kVec]) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) v[e] = fill;
  } else if (f32) {
    load8(static_cast<const float*>(p), c, cols, v);
  } else {
    load8(static_cast<const T*>(p), c, cols, v);
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Sum over the THREADS lanes that share a row (every lane gets it).  `red` is LDS of one float
// per wave; calls alternate between two such rows, so one barrier a call is enough.
template <int THREADS>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (THREADS > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) v += red[w];
  }
  return v;
}

struct NormParams {
  const void* x;
  int64_t ldx;
  const void* w;
  const void* b;
  bool param_f32;
  float eps;
  void* y;
  int64_t ldy;
  float* mean;
  float* rstd;
  int64_t rows;
  int cols;
  const void* dy;      // backward
  int64_t lddy;
  float* partial;      // backward: [blocks][2][cols] column sums, or null
};

// A row in pieces: THREADS lanes, CHUNKS pieces of eight columns each.  EVEN: the width is a multiple
// of eight.
template <typename T, int THREADS, int CHUNKS, bool EVEN>
struct Row {
  Raw<T> raw[CHUNKS];
  __device__ static __forceinline__ int col(int k) {
    return (k * THREADS + (int)threadIdx.x % THREADS) * kVec;
  }
  __device__ __forceinline__ void load(const void* base, int64_t at, int cols) {
    const T* row = static_cast<const T*>(base) + at;
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) {
      if (EVEN) raw[k].load_even(row, col(k), cols);
      else raw[k].load(row, col(k), cols);
    }
  }
};

template <typename T, bool EVEN>
__device__ __forceinline__ void store_row(T* row, int c, int cols, const float v[kVec]) {
  if (EVEN) {
    if (c < cols) store_vec<T, kVec>(row + c, v);
  } else {
    store8(row, c, cols, v);
  }
}

// A workgroup is 256 lanes: 256 / THREADS rows at a time, the groups of rows gridDim.x apart.
template <typename T, int THREADS, int CHUNKS, bool EVEN>
__global__ __launch_bounds__(256) void norm_kernel(NormParams p) {
  __shared__ float red[4][4];
  constexpr int kRows = 256 / THREADS;
  const int t = threadIdx.x % THREADS;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / THREADS;
  typedef Row<T, THREADS, CHUNKS, EVEN> R;
  R next;
  if (row < p.rows) next.load(p.x, row * p.ldx, p.cols);
  float w[CHUNKS][kVec], b[CHUNKS][kVec];
#pragma unroll
  for (int k = 0; k < CHUNKS; ++k) {
    load_param<T>(p.w, p.param_f32, R::col(k), p.cols, 1.0f, w[k]);
    load_param<T>(p.b, p.param_f32, R::col(k), p.cols, 0.0f, b[k]);
  }
  for (int turn = 0; row < p.rows; row += step, turn ^= 2) {
    float v[CHUNKS][kVec];
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) {
      next.raw[k].get(v[k]);
#pragma unroll
      for (int e = 0; e < kVec; ++e) sum += v[k][e];
    }
    if (row + step < p.rows) next.load(p.x, (row + step) * p.ldx, p.cols);
    const float mean = row_sum<THREADS>(sum, red[turn]) / (float)p.cols;
    float sq = 0.0f;
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) {
      const bool there = EVEN ? R::col(k) < p.cols : true;
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const float d = v[k][e] - mean;
        v[k][e] = d;
        if (EVEN ? there : R::col(k) + e < p.cols) sq = fmaf(d, d, sq);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<THREADS>(sq, red[turn + 1]) / (float)p.cols + p.eps);
    if (t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) {
      float o[kVec];
#pragma unroll
      for (int e = 0; e < kVec; ++e) o[e] = fmaf(v[k][e] * rstd, w[k][e], b[k][e]);
      store_row<T, EVEN>(y, R::col(k), p.cols, o);
    }
  }
}

// Rows longer than the registers take: one workgroup a row, the row read three times (its later
// reads come from L2).
template <typename T>
__global__ __launch_bounds__(256) void norm_long_kernel(NormParams p) {
  __shared__ float red[2][4];
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    float v[kVec];
    float sum = 0.0f;
    for (int c = threadIdx.x * kVec; c < p.cols; c += 256 * kVec) {
      load8(x, c, p.cols, v);
#pragma unroll
      for (int e = 0; e < kVec; ++e) sum += v[e];
    }
    const float mean = row_sum<256>(sum, red[0]) / (float)p.cols;
    float sq = 0.0f;
    for (int c = threadIdx.x * kVec; c < p.cols; c += 256 * kVec) {
      load8(x, c, p.cols, v);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const float d = v[e] - mean;
        if (c + e < p.cols) sq = fmaf(d, d, sq);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<256>(sq, red[1]) / (float)p.cols + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(p.y) + row * p.ldy;
    for (int c = threadIdx.x * kVec; c < p.cols; c += 256 * kVec) {
      float w[kVec], b[kVec], o[kVec];
      load8(x, c, p.cols, v);
      load_param<T>(p.w, p.param_f32, c, p.cols, 1.0f, w);
      load_param<T>(p.b, p.param_f32, c, p.cols, 0.0f, b);
#pragma unroll
      for (int e = 0; e < kVec; ++e) o[e] = fmaf((v[e] - mean) * rstd, w[e], b[e]);
      store8(y, c, p.cols, o);
    }
  }
}

// Backward pass in workgroups of LANES lanes, LANES / THREADS rows at a time; each workgroup leaves
// its column sums in its partial row.
// At least two waves a SIMD: with the 290 registers that the compiler takes for 2048 uneven columns
// only one fits, and the 4099 x 1601 fp16 pass took 34 us instead of 24 with 111 of them spilled.
template <typename T, int LANES, int THREADS, int CHUNKS, bool EVEN>
__global__ __launch_bounds__(LANES) __attribute__((amdgpu_waves_per_eu(2)))
void norm_grad_kernel(NormParams p) {
  constexpr int kRows = LANES / THREADS;
  __shared__ float red[4][4];                              // rows of 256 lanes: their sums
  __shared__ float cs[kRows > 1 ? kRows * THREADS * kVec : 1];   // the waves' column sums
  const int t = threadIdx.x % THREADS;
  const int sub = threadIdx.x / THREADS;
  typedef Row<T, THREADS, CHUNKS, EVEN> R;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + sub;
  R next_x, next_dy;
  float next_mean = 0.0f, next_rstd = 0.0f;
  auto fetch = [&](int64_t r) {
    next_x.load(p.x, r * p.ldx, p.cols);
    next_dy.load(p.dy, r * p.lddy, p.cols);
    next_mean = p.mean[r];
    next_rstd = p.rstd[r];
  };
  if (row < p.rows) fetch(row);
  float w[CHUNKS][kVec], sw[CHUNKS][kVec], sb[CHUNKS][kVec];
#pragma unroll
  for (int k = 0; k < CHUNKS; ++k) {
    load_param<T>(p.w, p.param_f32, R::col(k), p.cols, 1.0f, w[k]);
#pragma unroll
    for (int e = 0; e < kVec; ++e) sw[k][e] = sb[k][e] = 0.0f;
  }
  const float inv = 1.0f / (float)p.cols;
  for (int turn = 0; row < p.rows; row += step, turn ^= 2) {
    const float mean = next_mean, rstd = next_rstd;
    float h[CHUNKS][kVec], g[CHUNKS][kVec];
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) {
      next_x.raw[k].get(h[k]);
      next_dy.raw[k].get(g[k]);
    }
    if (row + step < p.rows) fetch(row + step);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k)
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        // a column past the end has dy = 0 and adds nothing to any sum, if its h is finite:
        // (0 - mean) rstd need not be.  Pieces of the first half are whole at every width of the
        // layout.
        const bool there = k < CHUNKS / 2 || R::col(k) + (EVEN ? 0 : e) < p.cols;
        const float hv = (h[k][e] - mean) * (there ? rstd : 0.0f);
        const float d = g[k][e];
        sb[k][e] += d;
        sw[k][e] = fmaf(d, hv, sw[k][e]);
        const float gv = d * w[k][e];
        s1 += gv;
        s2 = fmaf(gv, hv, s2);
        h[k][e] = hv;
        g[k][e] = gv;
      }
    s1 = row_sum<THREADS>(s1, red[turn]) * inv;
    s2 = row_sum<THREADS>(s2, red[turn + 1]) * inv;
    T* dx = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) {
      float o[kVec];
#pragma unroll
      for (int e = 0; e < kVec; ++e) o[e] = rstd * (g[k][e] - s1 - h[k][e] * s2);
      store_row<T, EVEN>(dx, R::col(k), p.cols, o);
    }
  }
  if (!p.partial) return;
  float* out = p.partial + (int64_t)blockIdx.x * 2 * p.cols;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k) {
      store8(out, R::col(k), p.cols, sw[k]);
      store8(out + p.cols, R::col(k), p.cols, sb[k]);
    }
  } else {
    // piece by piece: every wave lays its sums down, then each lane adds one or more columns over
    // the waves in order
#pragma unroll
    for (int pass = 0; pass < 2; ++pass)
#pragma unroll
      for (int k = 0; k < CHUNKS; ++k) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          cs[(sub * kVec + e) * THREADS + t] = pass ? sb[k][e] : sw[k][e];
        __syncthreads();
        for (int j = threadIdx.x; j < THREADS * kVec; j += LANES) {
          const int c = (k * THREADS + j / kVec) * kVec + j % kVec;
          if (c >= p.cols) continue;
          float s = 0.0f;
#pragma unroll
          for (int r = 0; r < kRows; ++r) s += cs[(r * kVec + j % kVec) * THREADS + j / kVec];
          out[pass * p.cols + c] = s;
        }
      }
  }
}

// Long rows: dx by one workgroup a row ...
template <typename T>
__global__ __launch_bounds__(256) void norm_grad_long_kernel(NormParams p) {
  __shared__ float red[2][4];
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float xv[kVec], g[kVec], w[kVec];
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x * kVec; c < p.cols; c += 256 * kVec) {
      load8(x, c, p.cols, xv);
      load8(dy, c, p.cols, g);
      load_param<T>(p.w, p.param_f32, c, p.cols, 1.0f, w);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        if (c + e < p.cols) {
          const float gv = g[e] * w[e];
          s1 += gv;
          s2 = fmaf(gv, (xv[e] - mean) * rstd, s2);
        }
      }
    }
    s1 = row_sum<256>(s1, red[0]) / (float)p.cols;
    s2 = row_sum<256>(s2, red[1]) / (float)p.cols;
    T* dx = static_cast<T*>(p.y) + row * p.ldy;
    for (int c = threadIdx.x * kVec; c < p.cols; c += 256 * kVec) {
      load8(x, c, p.cols, xv);
      load8(dy, c, p.cols, g);
      load_param<T>(p.w, p.param_f32, c, p.cols, 1.0f, w);
      float o[kVec];
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        o[e] = rstd * (g[e] * w[e] - s1 - (xv[e] - mean) * rstd * s2);
      store8(dx, c, p.cols, o);
    }
  }
}

// ... and the column sums by workgroups of 512 columns (blockIdx.y) that take rows blockIdx.x,
// blockIdx.x + gridDim.x, .. in four waves.
template <typename T>
__global__ __launch_bounds__(256) void norm_columns_kernel(NormParams p) {
  __shared__ float cs[2][3][kVec][64];
  const int t = threadIdx.x & 63, sub = threadIdx.x >> 6;
  const int c = blockIdx.y * 512 + t * kVec;
  float sw[kVec], sb[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) sw[e] = sb[e] = 0.0f;
  if (c < p.cols) {
    for (int64_t row = (int64_t)blockIdx.x * 4 + sub; row < p.rows; row += (int64_t)gridDim.x * 4) {
      float xv[kVec], g[kVec];
      const float mean = p.mean[row], rstd = p.rstd[row];
      load8(static_cast<const T*>(p.x) + row * p.ldx, c, p.cols, xv);
      load8(static_cast<const T*>(p.dy) + row * p.lddy, c, p.cols, g);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        sb[e] += g[e];
        sw[e] = fmaf(g[e], (xv[e] - mean) * rstd, sw[e]);
      }
    }
  }
  if (sub > 0) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      cs[0][sub - 1][e][t] = sw[e];
      cs[1][sub - 1][e][t] = sb[e];
    }
  }
  __syncthreads();
  if (sub == 0 && c < p.cols) {
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        sw[e] += cs[0][s][e][t];
        sb[e] += cs[1][s][e][t];
      }
    float* out = p.partial + (int64_t)blockIdx.x * 2 * p.cols;
    store8(out, c, p.cols, sw);
    store8(out + p.cols, c, p.cols, sb);
  }
}

// dw and db from the partial rows, added in order by 16 lanes a column, then across the lanes.
// A workgroup takes 16 columns of the 2 * cols sums.
__global__ __launch_bounds__(256) void norm_join_kernel(const float* partial, int blocks, int cols,
                                                        float* dw, float* db) {
  __shared__ float cs[16][17];
  const int j = threadIdx.x & 15, i = threadIdx.x >> 4;
  const int64_t width = 2 * (int64_t)cols;
  const int64_t c = (int64_t)blockIdx.x * 16 + j;
  float s = 0.0f;
  if (c < width) {
#pragma unroll 8
    for (int r = i; r < blocks; r += 16) s += partial[r * width + c];
  }
  cs[i][j] = s;
  __syncthreads();
  if (i == 0 && c < width) {
#pragma unroll
    for (int k = 1; k < 16; ++k) s += cs[k][j];
    if (c < cols) {
      if (dw) dw[c] = s;
    } else if (db) {
      db[c - cols] = s;
    }
  }
}

constexpr int64_t kMaxGrid = 1 << 22;

int64_t ceil64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Workgroups of the kernels whose waves walk over rows: enough to fill the chip with what its
// registers hold (eight workgroups of 256 lanes a CU), each then takes further rows.
constexpr int64_t kWalkers = 2048;

template <typename T, bool EVEN>
hipError_t launch_norm_rows(const NormParams& p, hipStream_t stream) {
  const int c = p.cols;
  const dim3 rows4((unsigned)std::min(ceil64(p.rows, 4), kWalkers));
  const dim3 rows1((unsigned)std::min(p.rows, kWalkers));
  if (c <= 512) norm_kernel<T, 64, 1, EVEN><<<rows4, 256, 0, stream>>>(p);
  else if (c <= 1024) norm_kernel<T, 64, 2, EVEN><<<rows4, 256, 0, stream>>>(p);
  else if (c <= 2048) norm_kernel<T, 64, 4, EVEN><<<rows4, 256, 0, stream>>>(p);
  else if (c <= 4096) norm_kernel<T, 256, 2, EVEN><<<rows1, 256, 0, stream>>>(p);
  else norm_kernel<T, 256, 4, EVEN><<<rows1, 256, 0, stream>>>(p);
  return hipGetLastError();
}

template <typename T, bool EVEN>
hipError_t launch_norm_grad_rows(const NormParams& p, int blocks, hipStream_t stream) {
  const int c = p.cols;
  const dim3 grid(blocks);
  if (c <= 512) norm_grad_kernel<T, 1024, 64, 1, EVEN><<<grid, 1024, 0, stream>>>(p);
  else if (c <= 1024) norm_grad_kernel<T, 512, 64, 2, EVEN><<<grid, 512, 0, stream>>>(p);
  else if (c <= 2048) norm_grad_kernel<T, 256, 64, 4, EVEN><<<grid, 256, 0, stream>>>(p);
  else if (c <= 4096) norm_grad_kernel<T, 256, 256, 2, EVEN><<<grid, 256, 0, stream>>>(p);
  else norm_grad_kernel<T, 256, 256, 4, EVEN><<<grid, 256, 0, stream>>>(p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_norm_t(const NormParams& p, hipStream_t stream) {
  const int c = p.cols;
  // a launch counts its work-items in 32 bits: past kMaxGrid workgroups each takes further rows
  const dim3 rows1((unsigned)std::min(p.rows, kMaxGrid));
  if (c <= 8192) {
    const bool even = c % kVec == 0;
    return even ? launch_norm_rows<T, true>(p, stream) : launch_norm_rows<T, false>(p, stream);
  }
  norm_long_kernel<T><<<rows1, 256, 0, stream>>>(p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_norm_grad_t(const NormParams& p, int blocks, hipStream_t stream) {
  const int c = p.cols;
  if (c <= 8192) {
    const bool even = c % kVec == 0;
    return even ? launch_norm_grad_rows<T, true>(p, blocks, stream)
                : launch_norm_grad_rows<T, false>(p, blocks, stream);
  }
  hipError_t e = hipSuccess;
  if (p.rows > 0) {
    norm_grad_long_kernel<T><<<dim3((unsigned)std::min(p.rows, kMaxGrid)), 256, 0, stream>>>(p);
    e = hipGetLastError();
  }
  if (e != hipSuccess || !p.partial) return e;
  norm_columns_kernel<T><<<dim3(blocks, (unsigned)ceil64(c, 512)), 256, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

int norm_grad_blocks(int64_t rows, int cols) {
  // rows a workgroup holds at once, and the workgroups that fill the chip (sixteen waves to a CU up
  // to 1024 columns, then eight); a row too long for registers has its own column workgroups
  const int at_once = cols <= 512 ? 16 : cols <= 1024 ? 8 : cols <= 2048 ? 4 : cols <= 8192 ? 1 : 4;
  const int64_t most = cols <= 512 ? 256 : cols <= 8192 ? 512 : 64;
  return (int)std::min(most, std::max<int64_t>(1, ceil64(rows, at_once)));
}

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  NormParams p{};
  p.x = a.x; p.ldx = a.ldx; p.w = a.weight; p.b = a.bias; p.param_f32 = a.param_f32;
  p.eps = a.eps; p.y = a.y; p.ldy = a.ldy; p.mean = a.mean; p.rstd = a.rstd;
  p.rows = a.rows; p.cols = a.cols;
  switch (a.type) {
    case kBf16: return launch_norm_t<bf16>(p, stream);
    case kF16: return launch_norm_t<f16>(p, stream);
    default: return launch_norm_t<float>(p, stream);
  }
}

hipError_t launch_norm_grad(const NormArgs& a, const void* dy, int64_t lddy, float* dweight,
                            float* dbias, float* partial, hipStream_t stream) {
  NormParams p{};
  p.x = a.x; p.ldx = a.ldx; p.w = a.weight; p.param_f32 = a.param_f32;
  p.y = a.y; p.ldy = a.ldy; p.mean = a.mean; p.rstd = a.rstd;
  p.rows = a.rows; p.cols = a.cols; p.dy = dy; p.lddy = lddy;
  p.partial = dweight || dbias ? partial : nullptr;
  const int blocks = norm_grad_blocks(a.rows, a.cols);
  hipError_t e = hipSuccess;
  switch (a.type) {
    case kBf16: e = launch_norm_grad_t<bf16>(p, blocks, stream); break;
    case kF16: e = launch_norm_grad_t<f16>(p, blocks, stream); break;
    default: e = launch_norm_grad_t<float>(p, blocks, stream); break;
  }
  if (e != hipSuccess || !p.partial) return e;
  norm_join_kernel<<<dim3((unsigned)ceil64(2 * (int64_t)a.cols, 16)), 256, 0, stream>>>(
      partial, blocks, a.cols, dweight, dbias);
  return hipGetLastError();
}

}  // namespace anvil
