// The pipeline of the products on LDS tiles (gfx950): slabs of both operands copied into LDS, fragments
// read ahead of the multiplies, outgoing rows through LDS, and the tiles' order, choice and launch.
// linear_tiles.hip describes it and what it measures; the products that end in something else than a
// linear layer's epilogue (gated.hip, cross_entropy.hip) run on it too.
#pragma once

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "device_common.h"
#include "launchers.h"
#include "linear_common.h"
#include "mfma_slab.h"
#include "scalar_types.h"

namespace anvil {

constexpr int kBK = 64;   // k of one slab

// The copies of one operand's slabs.  `base` is the address of the next slab's origin (row 0 of the
// tile, its first k), uniform over the wave and advanced slab by slab, so that offsets within it
// stay small however long the depth is; `off` are the lane's byte offsets from it.
template <bool KMAJOR, int ROWS, int NW>
struct SlabStream {
  static constexpr int kInsts = ROWS * kBK / 512 / NW;
  static_assert(ROWS * kBK / 512 % NW == 0 && kInsts >= 1, "instructions split over the waves");
  // From one instruction of a wave to its next: rows (K-contiguous) or k (K-major).  A lane keeps its
  // slot where that is a whole period of the slot swizzle; eight rows are half a period of the
  // K-contiguous one, which exchanges the halves of the slab's k.
  static constexpr int kStep = KMAJOR ? NW * (512 / ROWS) : NW * (512 / kBK);
  static constexpr bool kHalf = !KMAJOR && kStep == 8;
  // K-major instructions differ by a uniform offset (soff); K-contiguous ones by rows that have to
  // be checked against the edge one by one; K-major ones of 192 rows begin anywhere in a k-row
  static constexpr bool kAny = KMAJOR && 512 % ROWS != 0;
  static_assert(kInsts == 1 || kHalf || kAny || kStep % (KMAJOR ? 4 : 16) == 0, "slot swizzle period");
  uint32_t off[KMAJOR && !kAny ? 1 : kInsts];
  int kin[kAny ? kInsts : 1];   // the lane's k within the slab (of its first instruction)
  uint32_t soff;           // K-major: bytes from one instruction to the next
  uint64_t base, step;

  __device__ static __forceinline__ void piece(int i, int wave, int lane, int* row, int* c) {
    const int u = wave + i * NW;
    if constexpr (!KMAJOR) {
      constexpr int kSlots = kBK / 8;
      *row = (64 / kSlots) * u + lane / kSlots;
      *c = (lane % kSlots) ^ KContig<ROWS, kBK>::swz(*row);
    } else if constexpr (kAny) {
      constexpr int kSlots = ROWS / 8;
      *row = (u * 64 + lane) / kSlots;
      *c = ((u * 64 + lane) % kSlots) ^ KMajor<ROWS>::swz(*row);
    } else {
      constexpr int kSlots = ROWS / 8;
      *row = u * (512 / ROWS) + lane / kSlots;
      *c = (lane % kSlots) ^ KMajor<ROWS>::swz(*row);
    }
  }

  // origin: the element of tile row 0 at the first k; rows: valid rows from there
  __device__ __forceinline__ void init(const uint16_t* origin, int64_t ld, int64_t rows, int wave,
                                       int lane) {
    base = reinterpret_cast<uint64_t>(origin);
    step = KMAJOR ? (uint64_t)ld * (2 * kBK) : 2 * kBK;
    soff = KMAJOR && !kAny ? (uint32_t)ld * (2 * kStep) : 0;
    int row, c;
    piece(0, wave, lane, &row, &c);
    kin[0] = KMAJOR ? row : c * 8;
#pragma unroll
    for (int i = 0; i < (KMAJOR && !kAny ? 1 : kInsts); ++i) {
      piece(i, wave, lane, &row, &c);
      if constexpr (kAny) kin[i] = row;
      off[i] = (KMAJOR ? c * 8 : row) < rows
                   ? ((uint32_t)row * (uint32_t)ld + (uint32_t)c * 8) * 2u
                   : kOOB;
    }
  }

  // The same for a matrix in blocks of 64 columns, [columns / 64][matrix rows][64] with `block` elements
  // from one to the next, so that a slab is contiguous.  origin: in the block of the tile's first column
  // (K-contiguous: of its first k), the tile's first row (K-major: the first k).
  __device__ __forceinline__ void init_blocks(const uint16_t* origin, int64_t block, int64_t rows,
                                              int wave, int lane) {
    static_assert(!kAny, "blocks for power-of-two rows");
    init(origin, 64, rows, wave, lane);
    if constexpr (!KMAJOR) {
      step = (uint64_t)block * 2;
    } else {
      int row, c;
      piece(0, wave, lane, &row, &c);
      if (off[0] != kOOB)
        off[0] = ((uint32_t)row * 64u + (uint32_t)(c / 8) * (uint32_t)block + (uint32_t)(c % 8) * 8u) * 2u;
    }
  }

  // Instruction i of the slab at `base` into LDS address dst; left: depth from its first k on, at
  // most kBK (no branch, so that the copies can stand among the multiplies).
  __device__ __forceinline__ void issue(int i, uint32_t dst, int left, int wave) const {
    const i32x4_t rsrc = make_rsrc(reinterpret_cast<const uint16_t*>(base), 0x80000000u);
    const uint32_t to = dst + (uint32_t)(wave + i * NW) * 1024u;
    if constexpr (kAny) {
      dma16(rsrc, to, kin[i] < left ? off[i] : kOOB);
    } else if constexpr (KMAJOR) {
      dma16(rsrc, to, kin[0] < left - i * kStep ? off[0] : kOOB,
            (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)i * soff)));
    } else {
      const int k = kHalf && (i & 1) ? kin[0] ^ (kBK / 2) : kin[0];
      dma16(rsrc, to, k < left ? off[i] : kOOB);
    }
  }
  __device__ __forceinline__ void advance() { base += step; }
};

template <int BM, int BN, int WM, int WN, int KS>
struct Tile {
  static constexpr int kWaves = WM * WN;             // of one set
  static constexpr int kThreads = kWaves * KS * 64;
  static constexpr int kWTM = BM / WM, kWTN = BN / WN;
  static constexpr int kFM = kWTM / 32, kFN = kWTN / 32;
  static constexpr int kStage = (BM + BN) * kBK * 2;
  static constexpr int kQ = BM * kBK * 2;            // Q's part of a stage
  static constexpr int kRing = 2 * kStage;
  static constexpr int kLds = KS * kRing;
  static_assert(kWTM % 32 == 0 && kWTN % 32 == 0, "whole fragments");
  static_assert(KS == 1 || kWaves * kFM * kFN * 4096 <= kRing, "a set's sums fit its buffers");
};

// The multiplies of one tile: acc += the wave's block of the sum over `depth` k of P(i, k) Q(j, k).
// PAIR: the tile's columns are BN / 2 of one Q and the same BN / 2 of a second one, half of each wave's
// fragments from either, so that a lane holds both sums of an output element.
template <typename T, bool PT, bool QT, int BM, int BN, int WM, int WN, int KS, bool PAIR = false>
struct Pipe {
  using C = Tile<BM, BN, WM, WN, KS>;
  typedef typename Mfma<T>::vec vec;
  typedef SlabStream<PT, BM, C::kWaves> StreamP;
  static constexpr int kQs = PAIR ? 2 : 1;
  static constexpr int kRowsQ = BN / kQs;            // LDS rows of one Q
  static constexpr int kFQ = C::kFN / kQs;           // a wave's fragments of one Q
  typedef SlabStream<QT, kRowsQ, C::kWaves> StreamQ;
  static constexpr int kSteps = kBK / 16;
  static constexpr int kCopies = StreamP::kInsts + kQs * StreamQ::kInsts;
  static_assert(C::kFN % kQs == 0, "whole fragments of either Q");
  static_assert(kSteps % 2 == 0, "the first k-step of a slab uses the first fragment buffer");

  char* smem;        // this set's two buffers
  uint32_t lds;
  int wave, lane, wm, wn;
  StreamP sp;
  StreamQ sq[kQs];
  int64_t left;      // depth from the next slab to request on
  int KT;            // slabs

  __device__ __forceinline__ Pipe(char* smem_, int wave_)
      : smem(smem_), lds(lds_addr(smem_)), wave(wave_), lane((int)(threadIdx.x & 63)),
        wm(wave_ / WN), wn(wave_ % WN) {}

  // With KS sets (this is number kg) every set runs the same number of slabs; slabs past the depth
  // are zeros.  `second`: elements from the first Q to the second.
  __device__ __forceinline__ void begin(const uint16_t* P, int64_t ldp, int64_t rows_p,
                                        const uint16_t* Q, int64_t ldq, int64_t rows_q,
                                        int64_t depth, int kg, int64_t second = 0) {
    const int64_t slabs = (depth + kBK - 1) / kBK;
    KT = (int)(KS > 1 ? (slabs + KS - 1) / KS : slabs);
    const int64_t k0 = KS > 1 ? (int64_t)kg * KT * kBK : 0;
    left = depth - k0;
    sp.init(P + k0 * (PT ? ldp : 1), ldp, rows_p, wave, lane);
#pragma unroll
    for (int q = 0; q < kQs; ++q)
      sq[q].init(Q + q * second + k0 * (QT ? ldq : 1), ldq, rows_q, wave, lane);
  }

  // Instruction i of the next slab's copies into buffer `stage`.
  __device__ __forceinline__ void copy(int i, int stage) const {
    const uint32_t to = lds + (uint32_t)(stage * C::kStage);
    const int here = (int)(left < kBK ? left : kBK);
    if (i < StreamP::kInsts) {
      sp.issue(i, to, here, wave);
    } else {
      const int q = (i - StreamP::kInsts) / StreamQ::kInsts;
      sq[q].issue((i - StreamP::kInsts) % StreamQ::kInsts, to + C::kQ + q * (kRowsQ * kBK * 2), here,
                  wave);
    }
  }
  __device__ __forceinline__ void advance() {
    sp.advance();
#pragma unroll
    for (int q = 0; q < kQs; ++q) sq[q].advance();
    left -= kBK;
  }
  __device__ __forceinline__ void request(int stage) {
#pragma unroll
    for (int i = 0; i < kCopies; ++i) copy(i, stage);
    advance();
  }

  // The buffer that no wave reads any more after run(): the one before the last slab's.
  __device__ __forceinline__ char* spare() const { return smem + (KT & 1) * C::kStage; }

  // The wave's fragments of k-step ks of a buffer.
  __device__ __forceinline__ void read(int stage, int ks, int buf, vec (&fa)[2][C::kFM],
                                       vec (&fb)[2][C::kFN]) const {
    const char* tp = smem + stage * C::kStage;
    const char* tq = tp + C::kQ;
#pragma unroll
    for (int f = 0; f < C::kFM; ++f)
      fa[buf][f] = __builtin_bit_cast(
          vec, (read_frag<PT, BM, kBK>(tp, wm * C::kWTM + f * 32, ks, lane)));
#pragma unroll
    for (int f = 0; f < C::kFN; ++f)
      fb[buf][f] = __builtin_bit_cast(
          vec, (read_frag<QT, kRowsQ, kBK>(tq + f / kFQ * (kRowsQ * kBK * 2),
                                           (wn * kFQ + f % kFQ) * 32, ks, lane)));
  }

  // All slabs.  `sum`: 0 none, 1 also the sums over k of the wave's P fragment `wn`, 2 of its Q
  // fragment `wm` into `sums` (see add8).
  template <bool SUMS>
  __device__ __forceinline__ void run(f32x16_t (&acc)[C::kFM][C::kFN], int sum, float& sums) {
    if (KT == 0) return;
    vec fa[2][C::kFM], fb[2][C::kFN];
    auto read = [&](int stage, int ks, int buf) { this->read(stage, ks, buf, fa, fb); };

    // Slab kt from buffer `stage`.  MORE: there is a slab after it; REQUEST: and one after that,
    // whose copies go out among the last step's multiplies.
    auto slab = [&](int stage, auto more, auto req) {
      constexpr bool MORE = decltype(more)::value, REQUEST = decltype(req)::value;
      constexpr int kMults = C::kFM * C::kFN;
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        const bool last = ks + 1 == kSteps;
        if (!last) {
          read(stage, ks + 1, (ks + 1) & 1);
        } else {
          // this wave's reads of the slab are done and its part of the next one has landed; past
          // the barrier that holds for every wave
          wait_lds();
          if (MORE) {
            wait_vmcnt<0>();
            __syncthreads();
            read(stage ^ 1, 0, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);   // the reads stay ahead of the multiplies
#pragma unroll
        for (int m = 0; m < kMults; ++m) {
          const int fm = m / C::kFN, fn = m % C::kFN;
          acc[fm][fn] = Mfma<T>::run(fb[ks & 1][fn], fa[ks & 1][fm], acc[fm][fn]);
          if (last && REQUEST) {
#pragma unroll
            for (int i = m * kCopies / kMults; i < (m + 1) * kCopies / kMults; ++i) copy(i, stage);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        if constexpr (SUMS) {
          if (sum == 1) {
#pragma unroll
            for (int f = 0; f < C::kFM; ++f)
              if (f == wn) add8_of(f, fa[ks & 1][f], sums);
          } else if (sum == 2) {
#pragma unroll
            for (int f = 0; f < C::kFN; ++f)
              if (f == wm) add8_of(C::kFM + f, fb[ks & 1][f], sums);
          }
        }
        if (last && REQUEST) advance();
      }
    };

    constexpr std::integral_constant<bool, true> yes{};
    constexpr std::integral_constant<bool, false> no{};
    request(0);
    wait_vmcnt<0>();
    __syncthreads();
    if (KT > 1) request(1);
    read(0, 0, 0);
    int kt = 0;
    for (; kt + 2 < KT; ++kt) slab(kt & 1, yes, yes);
    if (kt + 1 < KT) slab(kt++ & 1, yes, no);
    slab(kt & 1, no, no);
  }

  // The slabs of `tiles` tiles one after the other, as one stream: while a tile's sums are finished, the
  // first slabs of the next one are on their way.  place(i) calls begin() for tile i (all of the same
  // depth, at least 1, which KT is set to before); before(i) runs ahead of the last slab's multiplies, done(i) after them, with
  // the tile's sums in acc, which are zero again for the next.  done() may use LDS outside the two
  // buffers; a barrier lies between any two calls of it.  It has to wait for all copies (wait_vmcnt<0>)
  // ahead of its first store to memory, and the slab after it does not wait again: it would wait for
  // those stores.  Past the last tile the copies load zeros.
  template <typename Place, typename Before, typename Done>
  __device__ __forceinline__ void walk(f32x16_t (&acc)[C::kFM][C::kFN], int tiles, Place place,
                                       Before before, Done done) {
    static_assert(KS == 1, "one set of waves");
    if (tiles <= 0) return;
    vec fa[2][C::kFM], fb[2][C::kFN];
    place(0);
    request(0);
    wait_vmcnt<0>();
    __syncthreads();
    int ahead = 0, asked = 1;   // the tile that is being copied, slabs requested of it
    auto turn = [&] {
      if (asked == KT) {
        asked = 0;
        if (++ahead < tiles) place(ahead);
        else left = 0;
      }
      ++asked;
    };
    turn();
    request(1);
    read(0, 0, 0, fa, fb);
    int at = 0, kt = 0;
    bool landed = false;
    const int total = tiles * KT;
    constexpr int kMults = C::kFM * C::kFN;
    for (int s = 0; s < total; ++s) {
      const int stage = s & 1;
      const bool last_slab = kt + 1 == KT;
      if (last_slab) before(at);
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        const bool last = ks + 1 == kSteps;
        if (!last) {
          read(stage, ks + 1, (ks + 1) & 1, fa, fb);
        } else {
          turn();
          wait_lds();
          if (!landed) wait_vmcnt<0>();
          __syncthreads();
          read(stage ^ 1, 0, 0, fa, fb);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < kMults; ++m) {
          const int fm = m / C::kFN, fn = m % C::kFN;
          acc[fm][fn] = Mfma<T>::run(fb[ks & 1][fn], fa[ks & 1][fm], acc[fm][fn]);
          if (last) {
#pragma unroll
            for (int i = m * kCopies / kMults; i < (m + 1) * kCopies / kMults; ++i) copy(i, stage);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      advance();
      ++kt;
      landed = last_slab;
      if (last_slab) {
        done(at);
#pragma unroll
        for (int fm = 0; fm < C::kFM; ++fm)
#pragma unroll
          for (int fn = 0; fn < C::kFN; ++fn) acc[fm][fn] = f32x16_t{};
        kt = 0;
        ++at;
      }
    }
    wait_vmcnt<0>();   // no copy may land after the workgroup's end
  }

  // run() of a wave without multiplies: its share of the copies, and every barrier.
  __device__ __forceinline__ void attend() {
    if (KT == 0) return;
    request(0);
    wait_vmcnt<0>();
    __syncthreads();
    if (KT > 1) request(1);
    for (int kt = 0; kt + 1 < KT; ++kt) {
      wait_vmcnt<0>();
      __syncthreads();
      if (kt + 2 < KT) request(kt & 1);
    }
  }

  // KS > 1: each set's sums go through its own buffers; the first set adds them in order.
  __device__ __forceinline__ void merge(int kg, f32x16_t (&acc)[C::kFM][C::kFN]) {
    if (KT == 0) return;
    __syncthreads();
    char* mine = smem + wave * (C::kFM * C::kFN * 4096) + lane * 16;
    if (kg > 0) {
#pragma unroll
      for (int fm = 0; fm < C::kFM; ++fm)
#pragma unroll
        for (int fn = 0; fn < C::kFN; ++fn)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4_t*>(mine + ((fm * C::kFN + fn) * 4 + q) * 1024) =
                f32x4_t{acc[fm][fn][4 * q], acc[fm][fn][4 * q + 1], acc[fm][fn][4 * q + 2],
                        acc[fm][fn][4 * q + 3]};
    }
    __syncthreads();
    if (kg == 0) {
#pragma unroll
      for (int s = 1; s < KS; ++s)
#pragma unroll
        for (int fm = 0; fm < C::kFM; ++fm)
#pragma unroll
          for (int fn = 0; fn < C::kFN; ++fn)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x4_t v = *reinterpret_cast<const f32x4_t*>(
                  mine + s * C::kRing + ((fm * C::kFN + fn) * 4 + q) * 1024);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[fm][fn][4 * q + e] += v[e];
            }
    }
  }
};

// Eight 16-bit values of type T as they lie in memory, to fp32 and back.
template <typename T>
__device__ __forceinline__ void unpack8(u32x4_t w, float v[8]) {
  T t[8];
  __builtin_memcpy(t, &w, 16);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = to_f32(t[e]);
}
template <typename T>
__device__ __forceinline__ u32x4_t pack8(const float v[8]) {
  T t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = from_f32<T>(v[e]);
  u32x4_t w;
  __builtin_memcpy(&w, t, 16);
  return w;
}

// A wave's 32 rows of its block on their way out: the accumulators (a lane holds runs of four columns
// of one row) go to LDS as fp32 and come back with eight consecutive columns a lane, lanes
// side by side along the rows, so that every access to memory is whole 128-byte lines.  (Stored
// from the accumulators' layout, 32 bytes of 32 rows an instruction, the lines left L2 half
// written: 392 us against 273 for the 32768 x 2816 product of depth 768 with two outputs.)  Slots
// of 16 bytes are swizzled by row: both sides are free of bank conflicts.
template <int WTN>
struct OutStage {
  static constexpr int kLanes = WTN / 8;        // lanes of a row
  static constexpr int kRows = 64 / kLanes;     // rows of one pass
  static constexpr int kPasses = 32 / kRows;
  static constexpr int kBytes = 32 * WTN * 4;
  static constexpr int kPer256 = 64 / WTN;      // rows in the 256 bytes that the banks span
  static_assert(WTN == 32 || WTN == 64, "rows of 128 or 256 bytes");
  __device__ static __forceinline__ char* at(char* base, int row, int slot) {
    return base + row * (WTN * 4) + ((slot ^ ((row / kPer256) & (WTN / 4 - 1))) << 4);
  }
  template <int FN>
  __device__ static __forceinline__ void put(char* base, const f32x16_t (&acc)[FN], int lane) {
    // the previous rows have been read: LDS accesses of one wave complete in order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4_t*>(at(base, lane & 31, fn * 8 + 2 * q + (lane >> 5))) =
            f32x4_t{acc[fn][4 * q], acc[fn][4 * q + 1], acc[fn][4 * q + 2], acc[fn][4 * q + 3]};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  // Row (of 32) and first column (of WTN) of the lane's piece in a pass.
  __device__ static __forceinline__ int row(int pass, int lane) { return pass * kRows + lane / kLanes; }
  __device__ static __forceinline__ int col(int lane) { return lane % kLanes * 8; }
  __device__ static __forceinline__ void get(char* base, int pass, int lane, float v[8]) {
    const int r = row(pass, lane), slot = lane % kLanes * 2;
    const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(at(base, r, slot));
    const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(at(base, r, slot + 1));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = lo[e];
      v[4 + e] = hi[e];
    }
  }
};

// The same for values that are rounded first: a wave's 32 rows of 64 columns in 16 bits, 4 KB.  A row is
// 128 bytes = eight slots of 16; slot c of row r lies at c ^ (r / 2 % 8), so that the 16 rows that are read
// or written together fall on all banks.
template <typename T>
struct OutStage16 {
  static constexpr int kBytes = 32 * 64 * 2;
  static constexpr int kRows = 8;               // rows of one pass, eight lanes each
  static constexpr int kPasses = 4;
  __device__ static __forceinline__ char* at(char* base, int row, int slot) {
    return base + row * 128 + ((slot ^ ((row >> 1) & 7)) << 4);
  }
  __device__ static __forceinline__ void put(char* base, const f32x16_t (&v)[2], int lane) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int fn = 0; fn < 2; ++fn)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const T t[4] = {from_f32<T>(v[fn][4 * q]), from_f32<T>(v[fn][4 * q + 1]),
                        from_f32<T>(v[fn][4 * q + 2]), from_f32<T>(v[fn][4 * q + 3])};
        u32x2_t w;
        __builtin_memcpy(&w, t, 8);
        *reinterpret_cast<u32x2_t*>(at(base, lane & 31, fn * 4 + q) + 8 * (lane >> 5)) = w;
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  __device__ static __forceinline__ int row(int pass, int lane) { return pass * kRows + lane / 8; }
  __device__ static __forceinline__ int col(int lane) { return lane % 8 * 8; }
  __device__ static __forceinline__ u32x4_t get(char* base, int pass, int lane) {
    return *reinterpret_cast<const u32x4_t*>(at(base, row(pass, lane), lane % 8));
  }
};

// Tiles of one launch in an order that lets the workgroups that run together on an XCD share their
// operands: consecutive ids go down kBand row tiles before they step to the next column tile.
constexpr int kBand = 4;
__device__ __forceinline__ void banded(int t, int tiles_m, int tiles_n, int* ti, int* tj) {
  const int band = t / (kBand * tiles_n);
  const int rest = t - band * kBand * tiles_n;
  const int high = min(kBand, tiles_m - band * kBand);
  *ti = band * kBand + rest % high;
  *tj = rest / high;
}

// A value that all lanes share, into scalar registers.  The tile's place comes out of wave shuffles; the
// copies' descriptors follow from it, and from vector registers every slab would move them over
// again, word by word, ahead of each copy (weight gradient 32768 x 768 x 2816: 167.6 us, so 163.6).
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// The tiles of the rows product as the workgroups of one XCD take them: an eighth of the whole tiles
// and then an eighth of the partly filled ones, numbered from 0 in the order in which neighbours share
// operands.
template <int BM>
struct TileOrder {
  RowTiles<BM> rows;
  int tiles_n, xcd;
  int whole, parts, mine;   // all whole tiles, all partly filled ones, this XCD's whole ones

  __device__ __forceinline__ TileOrder(const Groups& groups, int64_t n_rows, int tiles_n_)
      : rows(groups, n_rows), tiles_n(tiles_n_), xcd(blockIdx.x % 8) {
    whole = rows.whole * tiles_n;
    parts = (rows.total - rows.whole) * tiles_n;
    mine = whole / 8 + (xcd < whole % 8 ? 1 : 0);
  }
  // This XCD's tiles.  The XCDs that have one whole tile less come first among the partly filled ones.
  __device__ __forceinline__ int count() const { return mine + (parts + xcd) / 8; }
  // Tile at < count(): its first row, the end of its group's rows, its group, its column tile.
  __device__ __forceinline__ void place(int at, int64_t* row0, int64_t* end, int* group, int* tj) {
    int ti;
    if (at < mine) {
      banded(xcd * (whole / 8) + min(xcd, whole % 8) + at, rows.whole, tiles_n, &ti, tj);
    } else {
      at = (at - mine) * 8 + (7 - xcd);
      ti = rows.whole + at / tiles_n;
      *tj = at % tiles_n;
    }
    rows.find(ti, row0, end, group);
    *row0 = uniform(*row0);
    *end = uniform(*end);
    *group = __builtin_amdgcn_readfirstlane(*group);
  }
};

// The tile of this workgroup, where a workgroup has one.  False where there is none: the launch counts one
// row tile more for each group than there may be.
template <int BM>
__device__ __forceinline__ bool rows_place(const Groups& groups, int64_t n_rows, int tiles_n,
                                           int64_t* row0, int64_t* end, int* group, int* tj) {
  TileOrder<BM> order(groups, n_rows, tiles_n);
  const int at = blockIdx.x / 8;
  if (at >= order.count()) return false;
  order.place(at, row0, end, group, tj);
  return true;
}

// Workgroups of one launch, which counts its work-items (at most 1024 a workgroup) in 32 bits;
// larger calls take the kernels of linear.hip, whose workgroups walk over tiles.
constexpr int64_t kMaxTileGrid = (int64_t(1) << 22) - 1;

// Launches a kernel of more than 64 KB of LDS (its limit raised once per device).
template <typename K, typename... A>
hipError_t launch_lds(K kern, std::atomic<uint64_t>& configured, int64_t grid, int threads, int lds,
                      hipStream_t stream, A... args) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (bit == 0 || !(configured.load(std::memory_order_acquire) & bit)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                            hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    configured.fetch_or(bit, std::memory_order_release);
  }
  kern<<<dim3((unsigned)grid), threads, lds, stream>>>(args...);
  return hipGetLastError();
}

// Tile shapes of the rows product: 32x32 with eight sets of one wave, 32x128 with two sets of four
// (two workgroups a CU), 64x64 with four sets of four, 128x128 of four waves (two workgroups a CU),
// 256x256 of eight.  (128x192 of four waves, two workgroups a CU, is not among rows_tile's choices.)
enum RowsTile { kRows32, kRows32x128, kRows64, kRows128, kRows256, kRows128x192 };
constexpr int kTileRows[] = {32, 32, 64, 128, 256, 128};
constexpr int kTileCols[] = {32, 128, 64, 128, 256, 192};

inline int64_t row_tiles(const RowsProduct& a, int side) {
  return ceil64(a.rows, side) + (a.groups.offsets ? a.groups.count + 1 : 0);
}

// Time of one launch in microseconds, from a fit of measured calls (32 .. 32768 rows, 256 .. 4096
// columns, depths 512 .. 4096): rounds of workgroups, each a fixed part (first slab, epilogue) and
// one for each 64-deep slab.  128x128 tiles run two to a CU; where one round leaves CUs with one,
// that one is faster.  GELU and SiLU lengthen the epilogue by what their instructions take on the
// rows one CU finishes at once.  Examples, us measured with 64 / 128 / 256 rows and columns:
//   4096 x 768, depth 2816      42.9 / 36.3 / 56.9        2048 x 2816, depth 768  35.9 / 17.4 / 23.4
//   16384 x 768, depth 2816    161.2 / 79.9 / 65.8        4096 x 2816, depth 768  63.5 / 28.6 / 25.8
//   2048 x 512, depth 4096      20.0 / 44.0 / 76.6        with gelu               70.0 / 33.3 / 34.2
inline double rounds(double workgroups, double slots) { return std::ceil(workgroups / slots); }

inline double tile_cost(int side, double tiles, double slabs, bool heavy) {
  switch (side) {
    case 64: return rounds(tiles, 256) * (2.2 + 0.25 * slabs + (heavy ? 0.6 : 0.0));
    case 128: {
      const double pair = 4.0 + 0.9 * slabs + (heavy ? 4.0 : 0.0);
      const double one = 5.0 + 0.6 * slabs + (heavy ? 2.0 : 0.0);
      const double whole = std::floor(tiles / 512), rest = tiles - whole * 512;
      return whole * pair + (rest == 0 ? 0.0 : rest <= 256 ? one : pair);
    }
    default: return rounds(tiles, 256) * (10.0 + 1.2 * slabs + (heavy ? 8.0 : 0.0));
  }
}

inline RowsTile rows_tile(const RowsProduct& a) {
  const int64_t stack = a.groups.offsets ? std::max(1, a.groups.count) : 1;
  const int64_t height = ceil64(a.rows, stack);   // rows of a typical group
  // Up to 32 rows a taller tile only adds work on rows that are not there: us with 32x32 / 32x128 /
  // 64x64 tiles, the first or second taken by the same kind of fit (rounds of workgroups, slabs of
  // one set of waves):
  //   1 row, 768 columns, depth 2816   7.2 / 12.8 / 10.3    64 rows over 8, 2816, depth 768    17.1 /  9.8 / 13.8
  //   1 row, 4096, depth 4096         10.4 / 24.7 / 16.7    64 over 8, 512, depth 4096         12.9 / 27.1 / 19.0
  //   32 rows, 4096, depth 512         4.7 /  5.4 /  5.3    1000 over 32, 2816, depth 768      90.6 / 39.7 / 49.3
  //   32 rows, 512, depth 4096         8.7 / 17.7 / 13.5    768 over 24, 512, depth 4096       38.3 / 32.1 / 28.4
  // The last is one of two measured calls where 64x64 tiles, which share the depth among four sets,
  // are faster (by a tenth).
  if (height <= 32) {
    const double tiles_m = a.groups.offsets ? (double)a.rows / 32 + 0.5 * (double)stack : 1.0;
    const double slabs = (double)ceil64(a.depth, kBK);
    const double narrow = rounds(tiles_m * (double)ceil64(a.cols, 32), 256) * (4.5 + 0.7 * std::ceil(slabs / 8));
    const double wide = rounds(tiles_m * (double)ceil64(a.cols, 128), 512) * (4.5 + 0.6 * std::ceil(slabs / 2));
    return narrow <= wide ? kRows32 : kRows32x128;
  }
  const bool heavy = a.act == kActGelu || a.act == kActSilu;
  const double slabs = (double)ceil64(a.depth, kBK);
  RowsTile best = kRows64;
  double least = 0;
  for (RowsTile t : {kRows64, kRows128, kRows256}) {
    const int side = kTileRows[t];
    double cost;
    if (a.groups.offsets) {
      // A group's last tile is half full on average and comes at the end, where it fills up what a
      // round leaves over: 0.2 of a tile for each group, no whole rounds.  Us with 64 / 128 / 256 rows
      // and columns, equal groups and then groups as a router leaves them, the rule's choice last:
      //   4096 rows over  8,  512, depth 4096   43 /  45 /  76    59 /  47 /  77   64
      //   4096 rows over  8, 2816, depth  768   76 /  30 /  26    79 /  37 /  29   128
      //   4096 rows over 32, 2816, depth  768   80 /  36 /  46    99 /  52 /  46   256
      //   8192 rows over 32,  512, depth 4096   83 /  51 /  78   104 /  58 /  79   128
      //  32768 rows over 24,  768, depth 2816  397 / 194 / 163   403 / 198 / 174   256
      //  32768 rows over 32,  512, depth 4096  414 / 173 / 138   434 / 211 / 221   256
      // The host does not see the groups, so the choice is the average group's.  All 1024 rows at one
      // of 32 experts (2816, depth 768) run on 32x128 tiles in 18.1 us, where 128x128 takes 11.8; half
      // of 32768 rows at one of 32 (512, depth 4096) in 201 (equal groups 138).
      const double tiles_m = (double)a.rows / side + 0.2 * (double)stack;
      const double slots = side == 128 ? 512 : 256;
      const double share = std::max(1.0, tiles_m * (double)ceil64(a.cols, side) / slots);
      cost = share * tile_cost(side, slots, slabs, heavy);
    } else {
      cost = tile_cost(side, (double)(ceil64(a.rows, side) * ceil64(a.cols, side)), slabs, heavy);
    }
    if (t == kRows64 || cost < least) {
      best = t;
      least = cost;
    }
  }
  return best;
}

// rows_tile, or the largest tile where that one's number would not fit a launch.
inline RowsTile rows_tile_that_fits(const RowsProduct& a) {
  const RowsTile t = rows_tile(a);
  return row_tiles(a, kTileRows[t]) * ceil64(a.cols, kTileCols[t]) + 16 > kMaxTileGrid ? kRows256 : t;
}

inline bool multiple8(int64_t v) { return v % 8 == 0; }
inline bool wide_aligned(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Tile side and splits of each group's rows: the least of the tiles' time (as above; the K-major
// operands' slabs take 1.25 and 0.95 us, 0.62 where a CU has one 128x128 tile) and the join's, which
// writes and reads each split's sums.  Us by side/splits, bias gradient included, the choice first:
//     517 rows,  512 x 4096         128/1   13.3   256/1  22.8   128/2  18.1
//    4096 rows,  768 x 2816         128/3   40.8   128/1  59.8   128/2  43.3   256/4 46.9   256/7 44.1
//    4096 rows, 4096 x 4096         256/1  140.8   128/1 165.9   256/2 174.9
//   32768 rows,  256 x 768          128/21  39.6   128/8  64.3   128/32 39.7   256/32 50.2
//   32768 rows,  768 x 2816         256/7  167.3   128/7 201.2   256/4 224.8   256/8 229.1
//   32768 rows,  512 x 4096         256/8  164.8   128/4 178.0   256/7 174.6   256/16 183.2
//   32768 over 24, 768 x 2816       256/1  206.0   128/1 223.3   256/2 355.4
//   32768 over 32, 512 x 4096       256/1  201.9   128/1 233.5   256/2 414.9
//   32768 over  8, 256 x 768        128/5   39.2   128/1 113.5   128/4 42.1   256/4 67.7
// Experts are split alike, by the average group's rows: with half of the 32768 rows at one expert the
// two cases of 24 and 32 take 459 and 471, with all of them there 859 and 878.
struct WeightPlan {
  int side, splits;
};

inline WeightPlan weight_plan(const WeightProduct& a) {
  const double slabs = std::max(1.0, (double)a.rows / a.groups.count / kBK);
  const double bytes = 4.0 * a.groups.count * a.pi * a.qj;
  WeightPlan best{128, 1};
  double least = 0;
  for (int side : {128, 256}) {
    const double tiles =
        (double)ceil64(a.pi, side) * (double)ceil64(a.qj, side) * (double)a.groups.count;
    for (int splits = 1; splits <= 64; ++splits) {
      const double each = std::ceil(slabs / splits);
      if (splits > 1 && each < 4) break;   // at least 256 rows a split
      const double workgroups = tiles * splits;
      double cost = side == 256 ? rounds(workgroups, 256) * (10.0 + 1.25 * each)
                                : rounds(workgroups, 512) * (4.0 + 0.95 * each);
      if (side == 128 && workgroups <= 256) cost = 5.0 + 0.62 * each;
      if (splits > 1) cost += 5.0 + (2 * splits + 1) * bytes / 5e6;
      if ((side == 128 && splits == 1) || cost < least) {
        best = {side, splits};
        least = cost;
      }
    }
  }
  return best;
}

}  // namespace anvil
