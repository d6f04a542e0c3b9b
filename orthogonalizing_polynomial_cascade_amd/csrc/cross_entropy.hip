// Cross entropy of a linear head over a large vocabulary, s = x W^T:
//   lse[r] = log sum_v exp s[r][v],   loss[r] = lse[r] - s[r][target[r]]
// and, for the gradients, the probabilities P[r][v] = (exp(s[r][v] - lse[r]) - [v = target[r]]) dloss[r]
// of a piece of the vocabulary.
//
// The logits are a product of the linear layers' pipeline (tile_pipe.h) whose accumulators never leave the
// registers as they are: a lane holds runs of columns of one row, so a row's maximum and sum of
// exponentials over the tile are taken within the lane and joined with one exchange between the wave's
// halves and one through LDS between the waves of a row.  A tile leaves eight bytes a row; a second
// launch joins a row's tiles (maximum first, then the sums scaled to it).  For the gradients the logits are
// formed again, which costs a third of their products, where keeping them would cost 16384 x 50304 x 4 bytes
// written and read.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "cross_entropy.h"
#include "tile_pipe.h"

namespace anvil {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// (m, s) and (m2, s2) as one: s e^m + s2 e^m2 with the larger m.  Without columns m is -inf and s 0.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float top = m2 > m ? m2 : m;
  const float ref = top == -INFINITY ? 0.0f : top;
  s = s * __builtin_amdgcn_exp2f((m - ref) * kLog2e) + s2 * __builtin_amdgcn_exp2f((m2 - ref) * kLog2e);
  m = top;
}

// What the rows of a lane's fragments (row lane % 32 of each) have to do with a tile: read ahead of the
// tile's end.
template <int FM>
struct RowData {
  int target[FM];      // -1: ignored
  float ref[FM];       // -lse log2(e)
  float weight[FM];    // dloss times the scale
  template <bool STATS>
  __device__ __forceinline__ void load(const HeadProduct& p, int64_t r0, int lane) {
    const float scale = !STATS && p.scale ? p.scale[0] : 1.0f;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
      const int64_t r = r0 + fm * 32 + (lane & 31);
      target[fm] = -1;
      ref[fm] = weight[fm] = 0.0f;
      if (r >= p.rows) continue;
      target[fm] = (int)target_of(p.targets, p.wide, p.vocab, r);
      if (!STATS) {
        ref[fm] = -p.lse[r] * kLog2e;
        weight[fm] = p.dloss[r] * scale;
      }
    }
  }
};

// Columns past the lane's first `left` of the block count as logits of -inf.
template <int FM, int FN>
__device__ __forceinline__ void mask_columns(f32x16_t (&acc)[FM][FN], int left) {
#pragma unroll
  for (int fm = 0; fm < FM; ++fm)
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (fn * 32 + 8 * (e / 4) + e % 4 >= left) acc[fm][fn][e] = -INFINITY;
}

// The lane's place (0 .. FN * 32 - 1) of the row's target in a block whose columns begin at c0, -1 where
// another lane or block has it.
template <int FN>
__device__ __forceinline__ int target_place(int target, int64_t c0, int lane) {
  const int64_t d = target - c0 - 4 * (lane >> 5);
  return d >= 0 && d < FN * 32 && (d & 4) == 0 ? (int)d : -1;
}

// Statistics of a wave's block (rows r0 .., columns c0 ..) into stat[row of the block].  The choice of the
// target's logit is a row of comparisons that only the few blocks with a target run.
template <int FM, int FN>
__device__ __forceinline__ void block_stats(const HeadProduct& p, f32x16_t (&acc)[FM][FN],
                                            const RowData<FM>& rows, float2* stat, int64_t r0,
                                            int64_t c0, int lane) {
  if (c0 + FN * 32 > p.cols) mask_columns(acc, (int)(p.cols - c0) - 4 * (lane >> 5));
#pragma unroll
  for (int fm = 0; fm < FM; ++fm) {
    const int d = target_place<FN>(rows.target[fm], c0, lane);
    if (__any(d >= 0)) {
      float z = 0.0f;
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          z = d == fn * 32 + 8 * (e / 4) + e % 4 ? acc[fm][fn][e] : z;
      if (d >= 0) p.loss[r0 + fm * 32 + (lane & 31)] = z;
    }
    float m = -INFINITY, s = 0.0f;
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
      for (int e = 0; e < 16; ++e) m = __builtin_fmaxf(m, acc[fm][fn][e]);   // NaN stays out
    m = __builtin_fmaxf(m, __shfl_xor(m, 32));
    const float ref = m == -INFINITY ? 0.0f : -m * kLog2e;
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        s += __builtin_amdgcn_exp2f(fmaf(acc[fm][fn][e], kLog2e, ref));
    s += __shfl_xor(s, 32);
    if (lane < 32) stat[fm * 32 + lane] = make_float2(m, s);
  }
}

// P of one fragment row of a wave's block in place of the logits; rows without a target are left for
// the store to clear.
template <int FN>
__device__ __forceinline__ void row_probabilities(f32x16_t (&z)[FN], int d, float ref, float weight) {
  const bool any = __any(d >= 0);
#pragma unroll
  for (int fn = 0; fn < FN; ++fn)
#pragma unroll
    for (int e = 0; e < 16; ++e)
      z[fn][e] = __builtin_amdgcn_exp2f(fmaf(z[fn][e], kLog2e, ref));
  if (any) {
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        z[fn][e] -= d == fn * 32 + 8 * (e / 4) + e % 4 ? 1.0f : 0.0f;
  }
#pragma unroll
  for (int fn = 0; fn < FN; ++fn)
#pragma unroll
    for (int e = 0; e < 16; ++e) z[fn][e] *= weight;
}

// The waves' statistics stat[WN][BM] of a tile's rows, joined, to part.
template <int BM, int WN, int WAVES>
__device__ __forceinline__ void tile_stats(const HeadProduct& p, const float2* stat, int64_t row0,
                                           int64_t end, int tj, int tiles_n, int wave, int lane) {
  for (int at = wave * 64 + lane; at < BM && row0 + at < end; at += WAVES * 64) {
    float m = -INFINITY, s = 0.0f;
#pragma unroll
    for (int i = 0; i < WN; ++i) join(m, s, stat[i * BM + at].x, stat[i * BM + at].y);
    p.part[(row0 + at) * tiles_n + tj] = make_float2(m, s);
  }
}

template <typename T, bool STATS, bool QT, int BM, int BN, int WM, int WN, int KS, int OCC>
__global__ __launch_bounds__(WM * WN * KS * 64)
__attribute__((amdgpu_waves_per_eu(OCC)))
void head_kernel(HeadProduct p, int tiles_n) {
  using C = Tile<BM, BN, WM, WN, KS>;
  // P leaves rounded where a wave has 64 columns, which takes half of the LDS accesses
  constexpr bool kRounded = C::kWTN == 64;
  using S = std::conditional_t<kRounded, OutStage16<T>, OutStage<32>>;
  static_assert(C::kWaves * S::kBytes <= C::kStage, "the outgoing rows fit one buffer");
  static_assert(WN * BM * 8 <= C::kStage, "the statistics fit one buffer");
  extern __shared__ __attribute__((aligned(1024))) char smem_all[];
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int kg = wave_all / C::kWaves;
  const int wave = wave_all % C::kWaves;
  char* smem = smem_all + kg * C::kRing;
  int64_t row0, end;
  int group, tj;
  if (!rows_place<BM>(Groups{nullptr, false, 1}, p.rows, tiles_n, &row0, &end, &group, &tj)) return;
  const int64_t j0 = (int64_t)tj * BN;
  const uint16_t* w = static_cast<const uint16_t*>(p.w) +
                      (QT ? p.first + j0 : (p.first + j0) * p.ldw);

  f32x16_t acc[C::kFM][C::kFN];
#pragma unroll
  for (int fm = 0; fm < C::kFM; ++fm)
#pragma unroll
    for (int fn = 0; fn < C::kFN; ++fn) acc[fm][fn] = f32x16_t{};
  float none;
  Pipe<T, false, QT, BM, BN, WM, WN, KS> pipe(smem, wave);
  pipe.begin(static_cast<const uint16_t*>(p.x) + row0 * p.ldx, p.ldx, end - row0, w, p.ldw,
             p.cols - j0, p.depth, kg);
  const int wm = wave / WN, wn = wave % WN;
  const bool idle = row0 + wm * C::kWTM >= end;   // no row of the wave's block is there
  if (idle) pipe.attend();
  else pipe.template run<false>(acc, 0, none);
  if constexpr (KS > 1) pipe.merge(kg, acc);
  const int64_t c0 = j0 + wn * C::kWTN, r0 = row0 + wm * C::kWTM;
  RowData<C::kFM> rows;
  if (kg == 0 && !idle) rows.template load<STATS>(p, r0, lane);
  if constexpr (STATS) {
    // the first set's spare buffer; the other sets only meet at the barrier
    float2* stat = reinterpret_cast<float2*>(pipe.spare());
    if (kg == 0 && !idle) block_stats(p, acc, rows, stat + wn * BM + wm * C::kWTM, r0, c0, lane);
    __syncthreads();
    if (kg == 0) tile_stats<BM, WN, C::kWaves>(p, stat, row0, end, tj, tiles_n, wave, lane);
  } else {
    if (kg > 0 || idle) return;
    char* stage = pipe.spare() + wave * S::kBytes;
    const int64_t c = c0 + S::col(lane), first = r0 + S::row(0, lane);
    const int inside = c < p.cols ? (int)min(p.rows - first, (int64_t)C::kWTM) : 0;
    T* out = static_cast<T*>(p.p) + (c / 64 * p.rows + first) * 64 + c % 64;
    if (c0 + C::kWTN > p.cols) mask_columns(acc, (int)(p.cols - c0) - 4 * (lane >> 5));
#pragma unroll
    for (int fm = 0; fm < C::kFM; ++fm) {
      row_probabilities(acc[fm], target_place<C::kFN>(rows.target[fm], p.first + c0, lane),
                        rows.ref[fm], rows.weight[fm]);
      const uint64_t counts = __ballot(rows.target[fm] >= 0);
      S::put(stage, acc[fm], lane);
#pragma unroll
      for (int i = 0; i < S::kPasses; ++i) {
        const int r = fm * 32 + i * S::kRows;
        u32x4_t w;
        if constexpr (kRounded) {
          w = S::get(stage, i, lane);
        } else {
          float v[8];
          S::get(stage, i, lane, v);
          w = pack8<T>(v);
        }
        if (r < inside)
          *reinterpret_cast<u32x4_t*>(out + r * 64) =
              counts >> S::row(i, lane) & 1 ? w : u32x4_t{};
      }
    }
  }
}

// The statistics of large products: 256 workgroups that walk over the 256x256 tiles, the next tile's
// slabs on their way while a tile is finished (Pipe::walk); the waves' statistics lie beside the two
// buffers.  16384 x 50304, depth 768: 1482 us with a workgroup for each tile, 1208 in the walk, 1146 (1100
// TFLOP/s) with an epilogue whose rare parts are behind ballots.  The
// probabilities do not gain: vector memory operations end in order, so a walk's copies wait for the
// last tile's 128 KB of stores, which a workgroup of its own leaves behind when it ends (16384 x 16384: 560 us,
// 483 with a workgroup for each tile, 484 in a walk whose stores are left out).
template <typename T, bool QT>
__global__ __launch_bounds__(512)
__attribute__((amdgpu_waves_per_eu(2)))
void head_walk_kernel(HeadProduct p, int tiles_n) {
  constexpr int BM = 256, BN = 256, WM = 2, WN = 4;
  using C = Tile<BM, BN, WM, WN, 1>;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wm = wave / WN, wn = wave % WN;
  TileOrder<BM> order(Groups{nullptr, false, 1}, p.rows, tiles_n);
  const int me = blockIdx.x / 8, step = gridDim.x / 8;
  const int tiles = (order.count() - me + step - 1) / step;
  int64_t row0, end;   // of the tile that is being finished
  int group, tj;

  f32x16_t acc[C::kFM][C::kFN];
#pragma unroll
  for (int fm = 0; fm < C::kFM; ++fm)
#pragma unroll
    for (int fn = 0; fn < C::kFN; ++fn) acc[fm][fn] = f32x16_t{};
  Pipe<T, false, QT, BM, BN, WM, WN, 1> pipe(smem, wave);
  pipe.KT = (p.depth + kBK - 1) / kBK;
  RowData<C::kFM> rows;
  pipe.walk(
      acc, tiles,
      [&](int i) {
        int64_t first, last;
        int none, column;
        order.place(me + i * step, &first, &last, &none, &column);
        const int64_t j0 = (int64_t)column * BN;
        pipe.begin(static_cast<const uint16_t*>(p.x) + first * p.ldx, p.ldx, last - first,
                   static_cast<const uint16_t*>(p.w) + (QT ? j0 : j0 * p.ldw), p.ldw, p.cols - j0,
                   p.depth, 0);
      },
      [&](int i) {
        order.place(me + i * step, &row0, &end, &group, &tj);
        rows.template load<true>(p, row0 + wm * C::kWTM, lane);
      },
      [&](int) {
        float2* stat = reinterpret_cast<float2*>(smem + C::kRing);
        block_stats(p, acc, rows, stat + wn * BM + wm * C::kWTM, row0 + wm * C::kWTM,
                    (int64_t)tj * BN + wn * C::kWTN, lane);
        wait_vmcnt<0>();
        __syncthreads();
        tile_stats<BM, WN, C::kWaves>(p, stat, row0, end, tj, tiles_n, wave, lane);
      });
}

// A wave for each row: its tiles' statistics, 64 at a time, then the wave's halves pairwise.
__global__ __launch_bounds__(256) void head_join_kernel(HeadProduct p, int tiles_n, float* lse) {
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= p.rows) return;
  const int lane = threadIdx.x & 63;
  const float2* part = p.part + r * tiles_n;
  float m = -INFINITY, s = 0.0f;
  for (int i = lane; i < tiles_n; i += 64) join(m, s, part[i].x, part[i].y);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) join(m, s, __shfl_xor(m, o), __shfl_xor(s, o));
  if (lane == 0) {
    const float l = m + logf(s);
    lse[r] = l;
    p.loss[r] = target_of(p.targets, p.wide, p.vocab, r) >= 0 ? l - p.loss[r] : 0.0f;
  }
}

RowsTile head_tile(int64_t rows, int64_t cols, int depth) {
  RowsProduct a{};
  a.rows = rows;
  a.cols = (int)cols;
  a.depth = depth;
  a.groups = Groups{nullptr, false, 1};
  a.act = kActSilu;   // an epilogue of exponentials
  const RowsTile t = rows_tile_that_fits(a);
  return depth == 0 && t == kRows256 ? kRows128 : t;   // the walk begins with a slab
}

template <typename T, bool STATS, bool QT, int BM, int BN, int WM, int WN, int KS, int OCC>
hipError_t head_tiles(const HeadProduct& a, hipStream_t stream) {
  using C = Tile<BM, BN, WM, WN, KS>;
  static std::atomic<uint64_t> configured{0};
  const int64_t tiles_m = ceil64(a.rows, BM), tiles_n = ceil64(a.cols, BN);
  return launch_lds(head_kernel<T, STATS, QT, BM, BN, WM, WN, KS, OCC>, configured,
                    ceil64(tiles_m * tiles_n, 8) * 8 + 8, C::kThreads, C::kLds, stream, a,
                    (int)tiles_n);
}

template <typename T, bool QT>
hipError_t head_walk(const HeadProduct& a, hipStream_t stream) {
  using C = Tile<256, 256, 2, 4, 1>;
  static std::atomic<uint64_t> configured{0};
  return launch_lds(head_walk_kernel<T, QT>, configured, 256, C::kThreads, C::kRing + 4 * 256 * 8,
                    stream, a, (int)ceil64(a.cols, 256));
}

template <typename T, bool STATS, bool QT>
hipError_t head_variant(const HeadProduct& a, hipStream_t stream) {
  switch (head_tile(a.rows, a.cols, a.depth)) {
    case kRows32: return head_tiles<T, STATS, QT, 32, 32, 1, 1, 8, 2>(a, stream);
    case kRows32x128: return head_tiles<T, STATS, QT, 32, 128, 1, 4, 2, 4>(a, stream);
    case kRows64: return head_tiles<T, STATS, QT, 64, 64, 2, 2, 4, 4>(a, stream);
    case kRows128: return head_tiles<T, STATS, QT, 128, 128, 2, 2, 1, 2>(a, stream);
    default:
      if constexpr (STATS) return head_walk<T, QT>(a, stream);
      else return head_tiles<T, STATS, QT, 256, 256, 2, 4, 1, 2>(a, stream);
  }
}

template <bool STATS>
hipError_t head_launch(const HeadProduct& a, hipStream_t stream) {
  if (a.f16)
    return a.w_kn ? head_variant<f16, STATS, true>(a, stream)
                  : head_variant<f16, STATS, false>(a, stream);
  return a.w_kn ? head_variant<bf16, STATS, true>(a, stream)
                : head_variant<bf16, STATS, false>(a, stream);
}

}  // namespace

int64_t head_stat_tiles(int64_t rows, int64_t vocab, int depth) {
  return ceil64(vocab, kTileCols[head_tile(rows, vocab, depth)]);
}

hipError_t launch_head_stats(const HeadProduct& a, float* lse, hipStream_t stream) {
  const hipError_t e = head_launch<true>(a, stream);
  if (e != hipSuccess) return e;
  head_join_kernel<<<dim3((unsigned)ceil64(a.rows, 4)), 256, 0, stream>>>(
      a, (int)head_stat_tiles(a.rows, a.cols, a.depth), lse);
  return hipGetLastError();
}

hipError_t launch_head_probabilities(const HeadProduct& a, hipStream_t stream) {
  return head_launch<false>(a, stream);
}

}  // namespace anvil
