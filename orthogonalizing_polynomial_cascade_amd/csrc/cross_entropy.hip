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

#include "cross_entropy.h"
#include "tile_pipe.h"

namespace anvil {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// The row's target as a column of the whole vocabulary, -1 where it is outside (the row is ignored).
__device__ __forceinline__ int64_t target_of(const HeadProduct& p, int64_t r) {
  const int64_t t = p.wide ? static_cast<const int64_t*>(p.targets)[r]
                           : (int64_t)static_cast<const int32_t*>(p.targets)[r];
  return t >= 0 && t < p.vocab ? t : -1;
}

// (m, s) and (m2, s2) as one: s e^m + s2 e^m2 with the larger m.  Without columns m is -inf and s 0.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float top = m2 > m ? m2 : m;
  const float ref = top == -INFINITY ? 0.0f : top;
  s = s * __builtin_amdgcn_exp2f((m - ref) * kLog2e) + s2 * __builtin_amdgcn_exp2f((m2 - ref) * kLog2e);
  m = top;
}

// Statistics of a wave's block (rows r0 .., columns c0 .. of the piece) into stat[wn][row of the tile].
template <typename C, int BM>
__device__ __forceinline__ void block_stats(const HeadProduct& p,
                                            const f32x16_t (&acc)[C::kFM][C::kFN], float2* stat,
                                            int64_t row0, int wm, int64_t c0, int lane) {
  const int half = 4 * (lane >> 5);
  const bool edge = c0 + C::kWTN > p.cols;
  const int left = (int)min(p.cols - c0, (int64_t)C::kWTN) - half;   // the lane's valid columns
#pragma unroll
  for (int fm = 0; fm < C::kFM; ++fm) {
    const int at = wm * C::kWTM + fm * 32 + (lane & 31);
    const int64_t r = row0 + at;
    float m = -INFINITY, s = 0.0f;
#pragma unroll
    for (int fn = 0; fn < C::kFN; ++fn)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float z = acc[fm][fn][e];
        const bool in = !edge || fn * 32 + 8 * (e / 4) + e % 4 < left;
        if (in && z > m) m = z;
      }
    const float other = __shfl_xor(m, 32);
    m = other > m ? other : m;
    const float ref = m == -INFINITY ? 0.0f : -m * kLog2e;
#pragma unroll
    for (int fn = 0; fn < C::kFN; ++fn)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float x = __builtin_amdgcn_exp2f(fmaf(acc[fm][fn][e], kLog2e, ref));
        const bool in = !edge || fn * 32 + 8 * (e / 4) + e % 4 < left;
        s += in ? x : 0.0f;
      }
    s += __shfl_xor(s, 32);
    if (lane < 32) stat[at] = make_float2(m, s);
    if (r < p.rows) {
      const int64_t column = target_of(p, r) - c0 - half;   // the lane's own column of the block
      const int d = column >= 0 && column < C::kWTN ? (int)column : -1;
      if (d >= 0 && (d & 4) == 0) {
#pragma unroll
        for (int fn = 0; fn < C::kFN; ++fn)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (d == fn * 32 + 8 * (e / 4) + e % 4) p.loss[r] = acc[fm][fn][e];
      }
    }
  }
}

// P of a wave's block, through LDS into whole lines.
template <typename T, typename C>
__device__ __forceinline__ void block_probabilities(const HeadProduct& p,
                                                    f32x16_t (&acc)[C::kFM][C::kFN], char* stage,
                                                    int64_t r0, int64_t c0, int lane) {
  using S = OutStage<C::kWTN>;
  const int64_t c = c0 + S::col(lane);
  const int64_t first = r0 + S::row(0, lane);
  const int rows = c < p.ldp ? (int)min(p.rows - first, (int64_t)C::kWTM) : 0;
  T* out = static_cast<T*>(p.p) + first * p.ldp + c;
  const int half = 4 * (lane >> 5);
  const bool edge = c0 + C::kWTN > p.cols;
  const int left = (int)(p.cols - c0) - half;   // vocabularies fit an int
  const float scale = p.scale ? p.scale[0] : 1.0f;
#pragma unroll
  for (int fm = 0; fm < C::kFM; ++fm) {
    const int64_t r = r0 + fm * 32 + (lane & 31);
    float ref = 0.0f, weight = 0.0f;
    int d = -1;
    bool counts = false;
    if (r < p.rows) {
      const int64_t t = target_of(p, r);
      counts = t >= 0;
      ref = -p.lse[r] * kLog2e;
      weight = p.dloss[r] * scale;
      const int64_t column = t - p.first - c0 - half;   // the lane's own column of the block
      if (column >= 0 && column < C::kWTN) d = (int)column;
    }
#pragma unroll
    for (int fn = 0; fn < C::kFN; ++fn)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int at = fn * 32 + 8 * (e / 4) + e % 4;
        float x = __builtin_amdgcn_exp2f(fmaf(acc[fm][fn][e], kLog2e, ref));
        x = (d == at ? x - 1.0f : x) * weight;
        acc[fm][fn][e] = counts && (!edge || at < left) ? x : 0.0f;
      }
    S::put(stage, acc[fm], lane);
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) {
      const int rr = fm * 32 + i * S::kRows;
      float v[8];
      S::get(stage, i, lane, v);
      if (rr < rows) *reinterpret_cast<u32x4_t*>(out + rr * p.ldp) = pack8<T>(v);
    }
  }
}

template <typename T, bool STATS, bool QT, int BM, int BN, int WM, int WN, int KS, int OCC>
__global__ __launch_bounds__(WM * WN * KS * 64)
__attribute__((amdgpu_waves_per_eu(OCC)))
void head_kernel(HeadProduct p, int tiles_n) {
  using C = Tile<BM, BN, WM, WN, KS>;
  using S = OutStage<C::kWTN>;
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
  const int64_t c0 = j0 + wn * C::kWTN;
  if constexpr (STATS) {
    // the first set's spare buffer; the other sets only meet at the barrier
    float2* stat = reinterpret_cast<float2*>(pipe.spare());
    if (kg == 0 && !idle) block_stats<C, BM>(p, acc, stat + wn * BM, row0, wm, c0, lane);
    __syncthreads();
    if (kg == 0) {
      for (int at = wave * 64 + lane; at < BM && row0 + at < end; at += C::kWaves * 64) {
        float m = -INFINITY, s = 0.0f;
#pragma unroll
        for (int i = 0; i < WN; ++i) join(m, s, stat[i * BM + at].x, stat[i * BM + at].y);
        p.part[(row0 + at) * tiles_n + tj] = make_float2(m, s);
      }
    }
  } else {
    if (kg > 0 || idle) return;
    block_probabilities<T, C>(p, acc, pipe.spare() + wave * S::kBytes, row0 + wm * C::kWTM, c0, lane);
  }
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
    p.loss[r] = target_of(p, r) >= 0 ? l - p.loss[r] : 0.0f;
  }
}

RowsTile head_tile(int64_t rows, int64_t cols, int depth) {
  RowsProduct a{};
  a.rows = rows;
  a.cols = (int)cols;
  a.depth = depth;
  a.groups = Groups{nullptr, false, 1};
  a.act = kActSilu;   // an epilogue of exponentials
  return rows_tile_that_fits(a);
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

template <typename T, bool STATS, bool QT>
hipError_t head_variant(const HeadProduct& a, hipStream_t stream) {
  switch (head_tile(a.rows, a.cols, a.depth)) {
    case kRows32: return head_tiles<T, STATS, QT, 32, 32, 1, 1, 8, 2>(a, stream);
    case kRows32x128: return head_tiles<T, STATS, QT, 32, 128, 1, 4, 2, 4>(a, stream);
    case kRows64: return head_tiles<T, STATS, QT, 64, 64, 2, 2, 4, 4>(a, stream);
    case kRows128: return head_tiles<T, STATS, QT, 128, 128, 2, 2, 1, 2>(a, stream);
    default: return head_tiles<T, STATS, QT, 256, 256, 2, 4, 1, 2>(a, stream);
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
