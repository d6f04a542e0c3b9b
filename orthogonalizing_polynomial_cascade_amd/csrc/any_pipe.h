// The products for any width, pitch and alignment: operands through registers into LDS, one slab at a
// time (linear.hip describes them and what they measure).
#pragma once

#include <algorithm>

#include "device_common.h"
#include "linear_common.h"

namespace anvil {

constexpr int64_t kMaxGrid = 1 << 22;   // a launch counts its work-items in 32 bits
inline unsigned grid_for(int64_t n) { return (unsigned)std::max<int64_t>(1, std::min(n, kMaxGrid)); }

constexpr int kAnyDepth = 64;
constexpr int kAnyPitch = kAnyDepth + 8;   // elements per LDS row: 16-byte slots, spread banks

// One operand of the tile: SIDE rows by 64 k, SIDE / 32 pieces of eight elements a lane.
// K-contiguous: element (i, k) at base[i * ld + k], eight lanes to a row; K-major: at
// base[k * ld + i], four lanes to a k-row's 64 bytes and 16 k-rows to a wave, so that the two-byte
// writes of a wave fall on different banks.
template <typename T, bool KMAJOR, int SIDE>
struct AnySlab {
  static constexpr int kPieces = SIDE / 32;
  uint32_t v[kPieces][4];   // two elements each
  // Strided and contiguous index of the lane's piece i within the slab.
  __device__ static __forceinline__ int major(int i) {
    const int at = (int)threadIdx.x + i * 256;
    return KMAJOR ? (at >> 2) % kAnyDepth : at / 8;
  }
  __device__ static __forceinline__ int minor(int i) {
    const int at = (int)threadIdx.x + i * 256;
    return (KMAJOR ? (at & 3) + 4 * ((at >> 2) / kAnyDepth) : at % 8) * 8;
  }
  // The piece of `there` >= 1 elements at p, which lies in a row of `row` elements that ends with it
  // where there < 8: read as the row's last eight elements and moved down (or one by one in a row
  // of fewer than eight).
  __device__ static __forceinline__ void edge(const T* p, int there, int64_t row, uint32_t w[4]) {
    if (row >= 8) {
      const int back = there < 8 ? 8 - there : 0;
      uint32_t u[5] = {0, 0, 0, 0, 0};
      __builtin_memcpy(u, p - back, 16);
#pragma unroll
      for (int s = 2; s >= 1; --s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t from = i + s < 4 ? u[i + s] : 0u;
          u[i] = (back >> s) & 1 ? from : u[i];   // back = 4 b2 + 2 b1 + b0: two words, one word
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t moved = (u[i] >> 16) | (u[i + 1] << 16);
        w[i] = back & 1 ? moved : u[i];
      }
    } else {
#pragma unroll 1
      for (int e = 0; e < there; ++e) {
        const uint32_t x = (uint32_t)__builtin_bit_cast(uint16_t, p[e]) << (16 * (e & 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] |= e / 2 == i ? x : 0u;
      }
    }
  }
  __device__ __forceinline__ void load(const T* base, int64_t ld, int64_t i0, int64_t ni,
                                       int64_t k0, int64_t nk) {
    const T* at = base + (KMAJOR ? k0 : i0) * ld + (KMAJOR ? i0 : k0);
    if (i0 + SIDE <= ni && k0 + kAnyDepth <= nk) {   // no edge in the slab: loads back to back
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        __builtin_memcpy(v[i], at + major(i) * ld + minor(i), 16);
      return;
    }
    const int64_t nmaj = KMAJOR ? nk - k0 : ni - i0, nmin = KMAJOR ? ni - i0 : nk - k0;
    const int64_t row = KMAJOR ? ni : nk;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      uint32_t w[4] = {0, 0, 0, 0};
      const int there = (int)(nmin - minor(i) < 8 ? nmin - minor(i) : 8);
      if (major(i) < nmaj && there > 0) edge(at + major(i) * ld + minor(i), there, row, w);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[i][q] = w[q];
    }
  }
  __device__ __forceinline__ void store(T (*lds)[kAnyPitch]) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if constexpr (KMAJOR) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          lds[minor(i) + e][major(i)] =
              __builtin_bit_cast(T, (uint16_t)(v[i][e / 2] >> (16 * (e & 1))));
      } else {
        __builtin_memcpy(&lds[major(i)][minor(i)], v[i], 16);
      }
    }
  }
};

// A slab with an edge is what odd widths wait for: edge() shifts a piece right behind its load and in a branch of its
// own, so the compiler waits for each such load before it issues the next, two an operand and slab in tiles of 64
// rows and four in those of 128.  A second slab on its way in tiles of 64 rows gained nothing while that is so (517
// rows, 2002 x 513: 14.1 us as it is, 16.3 with it; its input gradient 35.6 and 36.8).
//
// acc (the wave's fragments, C transposed: register r of lane l is row l%32, column
// 8(r/4) + 4(l/32) + r%4 of a fragment) of the tile's k range [k0, k1).  `sum`: 1 the wave also adds
// up its P fragments over k into `sums`, 2 its Q fragments (see add8).
// PAIR: SIDE rows by the same 64 columns of two Qs, `second` elements apart; a wave has 32 columns, acc[m][0] of
// the first and acc[m][1] of the second, and no sums.
template <typename T, bool PT, bool QT, int SIDE, bool PAIR = false>
__device__ __forceinline__ void any_accumulate(const T* P, int64_t ldp, int64_t i0, int64_t ni,
                                               const T* Q, int64_t ldq, int64_t j0, int64_t nj,
                                               int64_t k0, int64_t k1,
                                               f32x16_t (&acc)[SIDE / 64][PAIR ? 2 : SIDE / 64], int sum,
                                               float (&sums)[SIDE / 64], int64_t second = 0) {
  constexpr int kQs = PAIR ? 2 : 1, kCols = PAIR ? 64 : SIDE;   // Qs, columns of each
  __shared__ __attribute__((aligned(16))) T lp[SIDE][kAnyPitch];
  __shared__ __attribute__((aligned(16))) T lq[kQs * kCols][kAnyPitch];
  typedef typename Mfma<T>::vec vec;
  constexpr int F = SIDE / 64, FN = PAIR ? 2 : F;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  AnySlab<T, PT, SIDE> sp;
  AnySlab<T, QT, kCols> sq[kQs];
  auto load = [&](int64_t k) {
    sp.load(P, ldp, i0, ni, k, k1);
#pragma unroll
    for (int q = 0; q < kQs; ++q) sq[q].load(Q + q * second, ldq, j0, nj, k, k1);
  };
  if (k0 < k1) load(k0);
  for (int64_t k = k0; k < k1; k += kAnyDepth) {
    __syncthreads();   // the previous slab's reads are done
    sp.store(lp);
#pragma unroll
    for (int q = 0; q < kQs; ++q) sq[q].store(lq + q * kCols);
    __syncthreads();
    if (k + kAnyDepth < k1) load(k + kAnyDepth);
#pragma unroll
    for (int ks = 0; ks < kAnyDepth / 16; ++ks) {
      const int kk = ks * 16 + 8 * (lane >> 5);
      vec fp[F], fq[FN];
#pragma unroll
      for (int f = 0; f < F; ++f)
        fp[f] = *reinterpret_cast<const vec*>(&lp[((wave >> 1) * F + f) * 32 + (lane & 31)][kk]);
#pragma unroll
      for (int f = 0; f < FN; ++f) {
        const int row = PAIR ? f * kCols + (wave & 1) * 32 : ((wave & 1) * F + f) * 32;
        fq[f] = *reinterpret_cast<const vec*>(&lq[row + (lane & 31)][kk]);
      }
#pragma unroll
      for (int m = 0; m < F; ++m)
#pragma unroll
        for (int n = 0; n < FN; ++n) acc[m][n] = Mfma<T>::run(fq[n], fp[m], acc[m][n]);
      if constexpr (PAIR) continue;
      if (sum) {   // one branch for the waves that have none
        if (sum == 1) {
#pragma unroll
          for (int f = 0; f < F; ++f) add8_of(f, fp[f], sums[f]);
        } else {
#pragma unroll
          for (int f = 0; f < F; ++f) add8_of(F + f, fq[f], sums[f]);
        }
      }
    }
  }
}

// 128x128 tiles once they give every CU one.  Us of the forward product with 64x64 and 128x128 tiles, by
// the number of the latter:
//    72 tiles, depth 769   20.1   39.5      288 tiles, depth 769    38.7   41.7
//   144 tiles, depth 769   23.7   37.0      544 tiles, depth 769    64.2   73.2
//   272 tiles, depth 513   31.8   33.3     1056 tiles, depth 4095  439.9  308.9
// and of the weight gradient with its best splits, by rows x columns of the weight:
//    600 rows,  131 x 333   12.9  21.4      2048 rows, 1031 x 769   37.4   35.9
//   4096 rows, 2049 x 769   92.4  73.3      4096 rows, 4097 x 4095 732.2  584.0
// The larger tiles pay with the depth: short of about a thousand, 64x64 would be 5 to 15% faster past
// the threshold too.
constexpr int64_t kManyTiles = 256;
inline bool any_wide_tiles(const RowsProduct& a) {
  const int64_t stack = a.groups.offsets ? std::max(1, a.groups.count) : 1;
  const int64_t height = ceil64(a.rows, stack);
  return height > 64 && stack * ceil64(height, 128) * ceil64(a.cols, 128) >= kManyTiles;
}

}  // namespace anvil
