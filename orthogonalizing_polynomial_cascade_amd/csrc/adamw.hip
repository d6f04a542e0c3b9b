// AdamW over a list of tensors in one launch.  Per element, in fp32 and every operation rounded on its own
// (the build takes no fused multiply-adds by itself), so that a step is the same numbers everywhere:
//   g = grad * grad_scale
//   m = m * beta1 + g * (1 - beta1),   v = v * beta2 + (g * g) * (1 - beta2)
//   p = p * (1 - lr * wd) - lr * ((m * fix1) / (sqrt(v) * fix2 + eps))
// with lr and wd times the tensor's own multipliers, fix1 = 1 / (1 - beta1^t), fix2 = 1 / sqrt(1 - beta2^t).
//
// 8-bit states hold m and sqrt(v) as e4m3 codes times an fp32 scale for each 256 elements (the largest
// magnitude of a block is 448 times its scale).  The root halves the range that v's codes have to span.
// Codes are rounded up or down at random with the probability that keeps the mean: to the nearest one,
// a second moment that moves by 1 - beta2 a step would never leave its code, whose neighbours are 2^-4 to 2^-3
// away.  The dither is a hash of (seed, tensor, element), so a step can be repeated bit for bit.  A root that is
// not zero keeps the least code, so that no denominator is lost.
//
// Bound by memory: 26 bytes an element with 32-bit states, a bf16 weight with its low half and a bf16
// gradient, 14.06 with 8-bit ones.  A workgroup takes 2048 elements of one tensor, eight consecutive ones a
// lane, so that 32 lanes hold a block and its maxima are five exchanges within half a wave; the tensors are
// found through a table of the pieces in device memory, which makes any number of them one launch.
// 77.3M weights as two halves with a bf16 gradient: 368 us with 32-bit states (5.5 TB/s), 210-217 with 8-bit
// ones (5.0-5.2 TB/s; about 90 vector operations an element, which bounds weights of 16 bits alone: 80M in 190
// us, 4.2 TB/s).  96 vectors of 256 to 2816 elements: 4.7 us.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "adamw.h"
#include "device_common.h"
#include "scalar_types.h"

namespace anvil {

namespace {

constexpr float kTop = 448.0f;              // the largest e4m3 value
constexpr float kLeast = 0x1p-100f;         // blocks below are taken as zero (their inverse scale is finite)
constexpr int kPer = 8;                     // elements of a lane

template <typename T>
using global_ptr = __attribute__((address_space(1))) T*;
template <typename T>
using eight = T __attribute__((ext_vector_type(8), aligned(sizeof(T))));

// The lane's eight elements from `at` on, n of them (FULL: all) in the tensor: in accesses of up to 16
// bytes at any element alignment.  The pointers come out of memory, so their address space has to be
// named for the loads not to be generic ones.
template <bool FULL, typename T>
__device__ __forceinline__ eight<T> load8(const void* base, int64_t at, int n) {
  const global_ptr<const T> p = (global_ptr<const T>)base + at;
  if (FULL || n >= kPer) return *(global_ptr<const eight<T>>)p;
  eight<T> v;
#pragma unroll
  for (int e = 0; e < kPer; ++e) v[e] = T(0);
  if (n > 0) {   // the tensor's last lane
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (e < n) v[e] = p[e];
  }
  return v;
}

template <bool FULL, typename T>
__device__ __forceinline__ void store8(void* base, int64_t at, int n, eight<T> v) {
  const global_ptr<T> p = (global_ptr<T>)base + at;
  if (FULL || n >= kPer) {
    *(global_ptr<eight<T>>)p = v;
  } else if (n > 0) {
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (e < n) p[e] = v[e];
  }
}

template <bool FULL, typename T>
__device__ __forceinline__ void load_as(const void* base, int64_t at, int n, float v[kPer]) {
  const eight<T> t = load8<FULL, T>(base, at, n);
#pragma unroll
  for (int e = 0; e < kPer; ++e) v[e] = to_f32(static_cast<T>(t[e]));
}

template <bool FULL, typename T>
__device__ __forceinline__ void store_as(void* base, int64_t at, int n, const float v[kPer]) {
  eight<T> t;
#pragma unroll
  for (int e = 0; e < kPer; ++e) t[e] = from_f32<T>(v[e]);
  store8<FULL, T>(base, at, n, t);
}

template <bool FULL>
__device__ __forceinline__ void load_type(int type, const void* p, int64_t at, int n, float v[kPer]) {
  switch (type) {
    case kF32: return load_as<FULL, float>(p, at, n, v);
    case kBf16: return load_as<FULL, bf16>(p, at, n, v);
    default: return load_as<FULL, f16>(p, at, n, v);
  }
}

// Weights: fp32, 16 bits rounded once, or the two halves of an fp32 master (bf16 bits, low 16 bits).
template <bool FULL>
__device__ __forceinline__ void load_weights(const AdamwTensor& t, int64_t at, int n, float v[kPer]) {
  if (!t.mantissa) return load_type<FULL>(t.param_type, t.param, at, n, v);
  const eight<uint16_t> hi = load8<FULL, uint16_t>(t.param, at, n);
  const eight<uint16_t> lo = load8<FULL, uint16_t>(t.mantissa, at, n);
#pragma unroll
  for (int e = 0; e < kPer; ++e) v[e] = __uint_as_float((uint32_t)hi[e] << 16 | lo[e]);
}

template <bool FULL>
__device__ __forceinline__ void store_weights(const AdamwTensor& t, int64_t at, int n,
                                              const float v[kPer]) {
  if (t.mantissa) {
    eight<uint16_t> hi, lo;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const uint32_t bits = __float_as_uint(v[e]);
      hi[e] = (uint16_t)(bits >> 16);
      lo[e] = (uint16_t)bits;
    }
    store8<FULL, uint16_t>(t.param, at, n, hi);
    store8<FULL, uint16_t>(t.mantissa, at, n, lo);
    return;
  }
  switch (t.param_type) {
    case kF32: return store_as<FULL, float>(t.param, at, n, v);
    case kBf16: return store_as<FULL, bf16>(t.param, at, n, v);
    default: return store_as<FULL, f16>(t.param, at, n, v);
  }
}

// Square roots, correctly rounded, of values that are not negative, by Tuckerman's test (Agarwal and others, IBM J.
// Res. Dev. 30, 1986): the hardware's root is within a step, and its neighbour is right if the product with it
// lies on the other side of the value.  Below 2^-96 those products lose
// bits: a wave that has such a value takes the compiler's root, which scales.
__device__ __forceinline__ void roots(const float v[kPer], float r[kPer]) {
  uint32_t least = ~0u;   // of bits - 1: zeros, infinities and NaN are far up
#pragma unroll
  for (int e = 0; e < kPer; ++e) least = min(least, __float_as_uint(v[e]) - 1u);
  if (__any(least < __float_as_uint(0x1p-96f))) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) r[e] = __builtin_sqrtf(v[e]);
    return;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const float s = __builtin_amdgcn_sqrtf(v[e]);
    const float down = __uint_as_float(__float_as_uint(s) - 1u);
    const float up = __uint_as_float(__float_as_uint(s) + 1u);
    const float below = fmaf(-down, s, v[e]), above = fmaf(-up, s, v[e]);
    const float t = below <= 0.0f ? down : s;
    r[e] = above > 0.0f ? up : t;
  }
}

// A hash of 32 bits.
__device__ __forceinline__ uint32_t mix(uint32_t h) {
  h = (h ^ (h >> 16)) * 0x7A3C5EB5u;
  h = (h ^ (h >> 15)) * 0x5D8E36CBu;
  return h ^ (h >> 16);
}

template <int CTRL>
__device__ __forceinline__ float moved(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF,
                                                               0xF, true));
}

// The largest magnitude of the block that the lane's half of the wave holds; NaN is left out.
__device__ __forceinline__ float block_top(const float v[kPer]) {
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) top = fmaxf(top, fabsf(v[e]));
  top = fmaxf(top, moved<0xB1>(top));    // within fours: 1 0 3 2,
  top = fmaxf(top, moved<0x4E>(top));    // 2 3 0 1;
  top = fmaxf(top, moved<0x141>(top));   // eights mirrored,
  top = fmaxf(top, moved<0x140>(top));   // sixteens mirrored
  return fmaxf(top, __shfl_xor(top, 16));
}

// e4m3 code of q >= 0 (at most 448 but for its rounding), before it is limited: at most 127, and more for
// NaN.  In fp32 an e4m3 number's kept bits end at bit 20 and its exponent begins at that of 2^-7; below 2^-6
// the codes are equally spaced, which adding 2^-6 makes of the fp32 numbers too.
__device__ __forceinline__ uint32_t raw_code(float q, uint32_t dither) {
  const bool small = q < 0x1p-6f;
  const uint32_t bits = __float_as_uint(small ? q + 0x1p-6f : q);
  return (bits + dither - __float_as_uint(small ? 0x1p-6f : 0x1p-7f)) >> 20;
}

// Codes and scale of the lane's eight values and their block.  SIGNED: m; else the root of v, of which a
// value that is not zero keeps the least code.
template <bool SIGNED>
__device__ __forceinline__ eight<uint8_t> encode(const float v[kPer], const uint32_t hash[kPer],
                                                 float* scale) {
  const float top = block_top(v);
  const float inverse = top >= kLeast ? kTop / top : 0.0f;
  *scale = top >= kLeast ? top / kTop : 0.0f;
  uint32_t code[kPer], most = 0;
  float q[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    q[e] = fabsf(v[e]) * inverse;
    code[e] = raw_code(q[e], SIGNED ? hash[e] & 0xFFFFFu : hash[e] >> 12);
    most = max(most, code[e]);
    code[e] = min(code[e], 126u);
    if (SIGNED) code[e] |= v[e] < 0.0f ? 128u : 0u;
    else code[e] = max(code[e], min(__float_as_uint(q[e]), 1u));
  }
  if (__any(most > 127u)) {
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (q[e] != q[e]) code[e] = 127u;
  }
  eight<uint8_t> t;
#pragma unroll
  for (int e = 0; e < kPer; ++e) t[e] = (uint8_t)code[e];
  return t;
}

template <bool FULL>
__device__ __forceinline__ void decode(const void* codes, int64_t at, int n, float scale,
                                       float v[kPer]) {
  const eight<uint8_t> t = load8<FULL, uint8_t>(codes, at, n);
  uint32_t w[2];
  __builtin_memcpy(w, &t, kPer);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    v[4 * h] = __builtin_amdgcn_cvt_f32_fp8((int)w[h], 0) * scale;
    v[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8((int)w[h], 1) * scale;
    v[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8((int)w[h], 2) * scale;
    v[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8((int)w[h], 3) * scale;
  }
}

template <bool BITS8, bool FULL>
__device__ __forceinline__ void adamw_piece(const AdamwTensor& t, const AdamwPiece& piece,
                                            const AdamwStep& step) {
  const int64_t at = (int64_t)piece.index * kAdamwPiece + threadIdx.x * kPer;
  const int64_t left = t.count - at;
  const int n = left >= kPer ? kPer : left > 0 ? (int)left : 0;
  const int64_t block = at / kAdamwBlock;
  const float lr = step.lr * t.lr_mul;
  const float keep = 1.0f - lr * (step.wd * t.wd_mul);

  float g[kPer], m[kPer], v[kPer], p[kPer], root[kPer];
  load_type<FULL>(t.grad_type, t.grad, at, n, g);
  if constexpr (BITS8) {
    const bool in = FULL || n;
    const float ms = in ? ((global_ptr<const float>)t.m_scale)[block] : 0.0f;
    const float vs = in ? ((global_ptr<const float>)t.v_scale)[block] : 0.0f;
    decode<FULL>(t.m, at, n, ms, m);
    decode<FULL>(t.v, at, n, vs, v);
#pragma unroll
    for (int e = 0; e < kPer; ++e) v[e] = v[e] * v[e];
  } else {
    load_as<FULL, float>(t.m, at, n, m);
    load_as<FULL, float>(t.v, at, n, v);
  }
  load_weights<FULL>(t, at, n, p);

  const float clip = step.grad_scale ? step.grad_scale[0] : 1.0f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const float x = g[e] * clip;
    m[e] = m[e] * step.beta1 + x * step.one_beta1;
    v[e] = v[e] * step.beta2 + (x * x) * step.one_beta2;
  }
  roots(v, root);
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    p[e] = p[e] * keep - lr * ((m[e] * step.fix1) / (root[e] * step.fix2 + step.eps));
  store_weights<FULL>(t, at, n, p);

  if constexpr (BITS8) {
    // lanes past the end hold zeros (or NaN, by an infinite clip), which do not count in a block's top
    const uint32_t key = mix(step.seed + ((uint32_t)piece.tensor + 1) * 0x9E3779B9u);
    uint32_t hash[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) hash[e] = mix((uint32_t)at + e + key);
    float ms, vs;
    store8<FULL, uint8_t>(t.m, at, n, encode<true>(m, hash, &ms));
    store8<FULL, uint8_t>(t.v, at, n, encode<false>(root, hash, &vs));
    if ((threadIdx.x & 31) == 0 && (FULL || n)) {
      ((global_ptr<float>)t.m_scale)[block] = ms;
      ((global_ptr<float>)t.v_scale)[block] = vs;
    }
  } else {
    store_as<FULL, float>(t.m, at, n, m);
    store_as<FULL, float>(t.v, at, n, v);
  }
}

__global__ __launch_bounds__(256) void adamw_kernel(const AdamwTensor* tensors,
                                                    const AdamwPiece* pieces, AdamwStep step) {
  const AdamwPiece piece = pieces[blockIdx.x];
  const AdamwTensor t = tensors[piece.tensor];
  if (step.device) {   // lr, weight decay, 1 - beta1^t, sqrt(1 - beta2^t), seed
    step.lr = step.device[0];
    step.wd = step.device[1];
    step.fix1 = 1.0f / step.device[2];
    step.fix2 = 1.0f / step.device[3];
    step.seed = (uint32_t)step.device[4];
  }
  const bool full = ((int64_t)piece.index + 1) * kAdamwPiece <= t.count;
  if (t.state_bits == 8) {
    if (full) adamw_piece<true, true>(t, piece, step);
    else adamw_piece<true, false>(t, piece, step);
  } else {
    if (full) adamw_piece<false, true>(t, piece, step);
    else adamw_piece<false, false>(t, piece, step);
  }
}

}  // namespace

hipError_t launch_adamw(const void* plan, int64_t tensors, int64_t pieces, const AdamwStep& step,
                        hipStream_t stream) {
  const AdamwTensor* t = static_cast<const AdamwTensor*>(plan);
  const AdamwPiece* p = reinterpret_cast<const AdamwPiece*>(t + tensors);
  constexpr int64_t kMost = 1 << 23;   // a launch counts its work-items in 32 bits
  for (int64_t at = 0; at < pieces; at += kMost) {
    adamw_kernel<<<dim3((unsigned)std::min(kMost, pieces - at)), 256, 0, stream>>>(t, p + at, step);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace anvil
