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

// A hash of 32 bits.
__device__ __forceinline__ uint32_t mix(uint32_t h) {
  h = (h ^ (h >> 16)) * 0x7A3C5EB5u;
  h = (h ^ (h >> 15)) * 0x5D8E36CBu;
  return h ^ (h >> 16);
}

// The largest magnitude of the block that the lane's half of the wave holds.
__device__ __forceinline__ float block_top(const float v[kPer]) {
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) top = fmaxf(top, fabsf(v[e]));   // NaN is left out
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  return top;
}

// e4m3 code of v, |v| * inverse <= 448 but for its rounding.  In fp32 an e4m3 number's kept bits end at bit 20; below
// 2^-6 the codes are equally spaced, which adding 2^-6 makes of the fp32 number too.  NaN gets the NaN code.
__device__ __forceinline__ uint32_t encode(float v, float inverse, uint32_t dither, uint32_t floor) {
  const float q = fabsf(v) * inverse;
  const bool small = q < 0x1p-6f;
  const uint32_t bits = __float_as_uint(small ? q + 0x1p-6f : q);
  uint32_t code = ((bits + dither) >> 20) - (small ? 968u : 960u);
  code = code > 126u ? 126u : code;
  if (q > 0.0f && code < floor) code = floor;
  if (q != q) code = 127u;
  return code | (v < 0.0f ? 128u : 0u);
}

// Eight codes at p (of n, unless n >= 8).
__device__ __forceinline__ void load_codes(const uint8_t* p, int n, float scale, float v[kPer]) {
  uint8_t t[kPer];
  if (n >= kPer) {
    __builtin_memcpy(t, p, kPer);
  } else {
#pragma unroll
    for (int e = 0; e < kPer; ++e) t[e] = e < n ? p[e] : (uint8_t)0;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) v[e] = __builtin_amdgcn_cvt_f32_fp8((int)t[e], 0) * scale;
}

__device__ __forceinline__ void store_codes(uint8_t* p, int n, const uint32_t c[kPer]) {
  uint8_t t[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) t[e] = (uint8_t)c[e];
  if (n >= kPer) {
    __builtin_memcpy(p, t, kPer);
  } else {
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (e < n) p[e] = t[e];
  }
}

template <typename T>
__device__ __forceinline__ void load_n(const void* base, int64_t at, int n, float v[kPer]) {
  const T* p = static_cast<const T*>(base) + at;
  if (n >= kPer) {
    load_vec<T, kPer>(p, v);
  } else {
#pragma unroll
    for (int e = 0; e < kPer; ++e) v[e] = e < n ? to_f32(p[e]) : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void store_n(void* base, int64_t at, int n, const float v[kPer]) {
  T* p = static_cast<T*>(base) + at;
  if (n >= kPer) {
    store_vec<T, kPer>(p, v);
  } else {
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (e < n) p[e] = from_f32<T>(v[e]);
  }
}

__device__ __forceinline__ void load_type(int type, const void* p, int64_t at, int n, float v[kPer]) {
  switch (type) {
    case kF32: return load_n<float>(p, at, n, v);
    case kBf16: return load_n<bf16>(p, at, n, v);
    default: return load_n<f16>(p, at, n, v);
  }
}

// Weights: fp32, 16 bits rounded once, or the two halves of an fp32 master (bf16 bits, low 16 bits).
__device__ __forceinline__ void load_halves(const AdamwTensor& t, int64_t at, int n, float v[kPer]) {
  uint16_t hi[kPer], lo[kPer];
  const uint16_t* p = static_cast<const uint16_t*>(t.param) + at;
  const uint16_t* q = t.mantissa + at;
  if (n >= kPer) {
    __builtin_memcpy(hi, p, 16);
    __builtin_memcpy(lo, q, 16);
  } else {
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      hi[e] = e < n ? p[e] : (uint16_t)0;
      lo[e] = e < n ? q[e] : (uint16_t)0;
    }
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) v[e] = __uint_as_float((uint32_t)hi[e] << 16 | lo[e]);
}

__device__ __forceinline__ void store_halves(const AdamwTensor& t, int64_t at, int n,
                                             const float v[kPer]) {
  uint16_t hi[kPer], lo[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const uint32_t bits = __float_as_uint(v[e]);
    hi[e] = (uint16_t)(bits >> 16);
    lo[e] = (uint16_t)bits;
  }
  uint16_t* p = static_cast<uint16_t*>(t.param) + at;
  uint16_t* q = t.mantissa + at;
  if (n >= kPer) {
    __builtin_memcpy(p, hi, 16);
    __builtin_memcpy(q, lo, 16);
  } else {
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (e < n) {
        p[e] = hi[e];
        q[e] = lo[e];
      }
  }
}

template <bool BITS8>
__device__ __forceinline__ void adamw_piece(const AdamwTensor& t, const AdamwPiece& piece,
                                            AdamwStep step) {
  const int64_t at = (int64_t)piece.index * kAdamwPiece + threadIdx.x * kPer;
  const int64_t left = t.count - at;
  const int n = left >= kPer ? kPer : left > 0 ? (int)left : 0;
  if (step.device) {   // lr, weight decay, 1 - beta1^t, sqrt(1 - beta2^t), seed
    step.lr = step.device[0];
    step.wd = step.device[1];
    step.fix1 = 1.0f / step.device[2];
    step.fix2 = 1.0f / step.device[3];
    step.seed = (uint32_t)step.device[4];
  }
  const float lr = step.lr * t.lr_mul;
  const float keep = 1.0f - lr * (step.wd * t.wd_mul);

  float g[kPer], m[kPer], v[kPer], p[kPer];
  const int64_t block = at / kAdamwBlock;
  load_type(t.grad_type, t.grad, at, n, g);
  if constexpr (BITS8) {
    const float ms = n ? t.m_scale[block] : 0.0f, vs = n ? t.v_scale[block] : 0.0f;
    load_codes(static_cast<const uint8_t*>(t.m) + at, n, ms, m);
    load_codes(static_cast<const uint8_t*>(t.v) + at, n, vs, v);
#pragma unroll
    for (int e = 0; e < kPer; ++e) v[e] = v[e] * v[e];
  } else {
    load_n<float>(t.m, at, n, m);
    load_n<float>(t.v, at, n, v);
  }
  if (t.mantissa) load_halves(t, at, n, p);
  else load_type(t.param_type, t.param, at, n, p);

  const float clip = step.grad_scale ? step.grad_scale[0] : 1.0f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const float x = g[e] * clip;
    m[e] = m[e] * step.beta1 + x * step.one_beta1;
    v[e] = v[e] * step.beta2 + (x * x) * step.one_beta2;
    const float root = __builtin_sqrtf(v[e]);
    p[e] = p[e] * keep - lr * ((m[e] * step.fix1) / (root * step.fix2 + step.eps));
    if constexpr (BITS8) v[e] = root;
  }

  if (t.mantissa) {
    store_halves(t, at, n, p);
  } else {
    switch (t.param_type) {
      case kF32: store_n<float>(t.param, at, n, p); break;
      case kBf16: store_n<bf16>(t.param, at, n, p); break;
      default: store_n<f16>(t.param, at, n, p); break;
    }
  }
  if constexpr (BITS8) {
    // lanes past the end hold zeros: loads, and so m and v, are zero there
    const float mt = block_top(m), vt = block_top(v);
    const float mi = mt >= kLeast ? kTop / mt : 0.0f, vi = vt >= kLeast ? kTop / vt : 0.0f;
    const uint32_t key = mix(step.seed + ((uint32_t)piece.tensor + 1) * 0x9E3779B9u);
    uint32_t mc[kPer], vc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const uint32_t h = mix((uint32_t)at + e + key);
      mc[e] = encode(m[e], mi, h & 0xFFFFFu, 0u);
      vc[e] = encode(v[e], vi, h >> 12, 1u);
    }
    store_codes(static_cast<uint8_t*>(t.m) + at, n, mc);
    store_codes(static_cast<uint8_t*>(t.v) + at, n, vc);
    if ((threadIdx.x & 31) == 0 && n) {
      t.m_scale[block] = mt >= kLeast ? mt / kTop : 0.0f;
      t.v_scale[block] = vt >= kLeast ? vt / kTop : 0.0f;
    }
  } else {
    store_n<float>(t.m, at, n, m);
    store_n<float>(t.v, at, n, v);
  }
}

__global__ __launch_bounds__(256) void adamw_kernel(const AdamwTensor* tensors,
                                                    const AdamwPiece* pieces, AdamwStep step) {
  const AdamwPiece piece = pieces[blockIdx.x];
  const AdamwTensor t = tensors[piece.tensor];
  if (t.state_bits == 8) adamw_piece<true>(t, piece, step);
  else adamw_piece<false>(t, piece, step);
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
