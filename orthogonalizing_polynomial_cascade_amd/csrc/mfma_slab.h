// LDS operand slabs of the MFMA kernels (gfx950): their layouts, the copy instruction that fills
// them, the fragment reads, and the waits and workgroup placement that go with them.
#pragma once

#include "device_common.h"

// m0 is written by the DMA inline assembly; the kernels have no other use of it (no indirect
// register indexing), which is what the compiler's reserved-register warning is about.
#pragma clang diagnostic ignored "-Winline-asm"

namespace anvil {

constexpr uint32_t kOOB = 0x80000000u;   // buffer offset past any range: the load returns 0

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_void_ptr;
typedef __attribute__((address_space(3))) s16x4_t* lds_s16x4_ptr;
typedef int i32x4_t __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------------------------
// LDS slab layouts
// ---------------------------------------------------------------------------------------------

// [ROWS][BK] bf16: a row is BK*2 bytes = BK/8 slots of 16 bytes (8 k each), and 256 bytes of LDS
// (one pass over the 64 banks) hold 16/(BK/8) rows, or one row spans BK/128 such passes.
// Logical slot c of row r sits at slot c ^ ((r / rows_per_256B) % min(slots, 16)): 16
// consecutive rows read at one logical slot hit 16 distinct 16-byte bank groups.
template <int ROWS, int BK>
struct KContig {
  static constexpr int kSlots = BK / 8;
  static constexpr int kRowsPer256 = kSlots >= 16 ? 1 : 16 / kSlots;
  static constexpr int kSwizzle = kSlots >= 16 ? 16 : kSlots;
  __device__ static __forceinline__ int swz(int row) { return (row / kRowsPer256) % kSwizzle; }
  __device__ static __forceinline__ int offset(int row, int c) {
    return row * (BK * 2) + ((c ^ swz(row)) << 4);
  }
};

// [BK][ROWS] bf16: a k-row is ROWS*2 bytes = ROWS/8 slots.  A transposing read takes 32 bytes of
// each of four consecutive k-rows: the swizzle puts those at four distinct 64-byte quarters of the
// 256 bytes that the banks span.  From 128 rows up, logical slot c of k-row kr sits at slot
// c ^ (4 * (kr & 3)); at 64 rows two k-rows share the 256 bytes and every second pair swaps its
// halves; at 32 rows four k-rows fill the 256 bytes by themselves.
template <int ROWS>
struct KMajor {
  static_assert(ROWS >= 32 && (ROWS & (ROWS - 1)) == 0, "K-major slab rows: a power of two");
  static constexpr int kPer256 = ROWS >= 128 ? 1 : 128 / ROWS;
  __device__ static __forceinline__ int swz(int kr) {
    return ((kr / kPer256) & (4 / kPer256 - 1)) << 2;
  }
  __device__ static __forceinline__ int offset(int kr, int c) {
    return kr * (ROWS * 2) + ((c ^ swz(kr)) << 4);
  }
};

// Raw buffer resource (stride 0, flags word of the gfx9 family) over `bytes` bytes at `base`.
// All four words are wave-uniform and live in SGPRs.
__device__ __forceinline__ i32x4_t make_rsrc(const uint16_t* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  i32x4_t r;
  r[0] = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(a)));
  r[1] = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(a >> 32) & 0xFFFFu));
  r[2] = __builtin_amdgcn_readfirstlane(static_cast<int>(bytes));
  r[3] = 0x00020000;
  return r;
}

// 32-bit LDS address of a pointer into dynamic shared memory (wave-uniform).
__device__ __forceinline__ uint32_t lds_addr(const char* ptr) {
  return __builtin_amdgcn_readfirstlane(
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void_ptr)(ptr))));
}

// One wave-instruction of DMA: lane L's 16 bytes at `voff` of the buffer land in LDS at
// lds + 16*L.  Issued as inline assembly so that the compiler neither reorders it nor inserts its
// own (conservative) waits on it; completion is tracked with wait_vmcnt below.
// Nor does the compiler put wait states inside: one is needed between the write of m0 and the copy,
// five between a vector instruction's write of a scalar register (the v_readfirstlane of a descriptor
// word) and a vector memory instruction that reads it.  s_nop 4 is five, whatever stands before the
// block.
__device__ __forceinline__ void dma16(i32x4_t rsrc, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}

// The same with a uniform byte offset `soff` on top of the lanes'; a lane at kOOB stays out of range.
__device__ __forceinline__ void dma16(i32x4_t rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory", "m0");
}

// MFMA operand of a 32-row fragment (rows R0..R0+31) at k-step ks (k = 16ks .. 16ks+15):
// lane l holds row R0 + l%32, k = 16ks + 8(l/32) + 0..7.
template <bool KMAJOR, int ROWS, int BK>
__device__ __forceinline__ bf16x8_t read_frag(const char* tile, int R0, int ks, int lane) {
  if constexpr (!KMAJOR) {
    const int row = R0 + (lane & 31);
    const int c = 2 * ks + (lane >> 5);
    return *reinterpret_cast<const bf16x8_t*>(tile + KContig<ROWS, BK>::offset(row, c));
  } else {
    const int grp = lane >> 4;
    const int r = lane & 15;
    const int i = R0 + 16 * (grp & 1) + 4 * (r & 3);
    const int kr = 16 * ks + 8 * (grp >> 1) + (r >> 2);
    const int c = i >> 3;
    const int half = ((i >> 2) & 1) * 8;
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s16x4_ptr)(tile + KMajor<ROWS>::offset(kr, c) + half));
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s16x4_ptr)(tile + KMajor<ROWS>::offset(kr + 4, c) + half));
    const s16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8_t, v);
  }
}

// Wait until at most N vector-memory operations of this wave are outstanding.
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// Wait for this wave's LDS operations (lgkmcnt(0)).
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }

// Workgroup id -> logical tile id such that each XCD gets a contiguous run of logical ids.
__device__ __forceinline__ int xcd_remap(int id, int total) {
  constexpr int kXcd = 8;
  const int q = total / kXcd;
  const int r = total % kXcd;
  const int x = id % kXcd;
  const int local = id / kXcd;
  return (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + local;
}

}  // namespace anvil
