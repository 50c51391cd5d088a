// 8-bit floating-point codes (e4m3: four exponent bits, three of fraction, largest value 448, no
// infinity, NaN 0x7F / 0xFF) with a scale per block of 128, and the 16-bit types around them.
//
// scale = max|v| / 448 over a block, codes e4m3(v / scale), rounded to nearest even (by the
// reciprocals of both divisors: scale_of, encode8).  The codes use
// the block's largest value for the top of their range, so a value down to 1 / 28672 of it (448
// over 2^-6, the smallest normal code) keeps its four significant bits.  A block of zeros, or of
// values below 2^-100, is coded as if its largest value were 2^-100: the scale stays a normal
// number, and so does its product with a weight's scale above 2^-17.  A block with a NaN or an
// infinity has a scale that is not finite and a NaN code where the value was, so that no product
// hides it.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace qfp8 {

constexpr int kBlock = 128;         // columns that share a scale
constexpr float kTop = 448.f;       // largest e4m3 value
constexpr float kFloor = 7.88860905e-31f;  // 2^-100, see above

__host__ __device__ constexpr int blocks_of(int n) { return (n + kBlock - 1) / kBlock; }

// Sizes are compared as the bits of |v|, whose order is that of the numbers, infinity above them
// and NaN above that (fmaxf would drop a NaN).
__device__ __forceinline__ uint32_t size_of(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ float scale_of(uint32_t top) {
  return __uint_as_float(max(top, __float_as_uint(kFloor))) * (1.f / kTop);
}

// Without the steps that would keep subnormal arguments and results: off by 2^-22 and 2^-23.
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two codes, the first in the low byte.
__device__ __forceinline__ uint32_t encode2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// Eight codes of v / scale.  Scales are normal numbers below 2^120; their reciprocal is off by at
// most 2^-23 and the product rounded once: together less than 2^-22 of the value, which changes a
// code only that close to a border of two.
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float scale) {
  const float inv = rcp_fast(scale);
  uint2 r;
  r.x = encode2(v[0] * inv, v[1] * inv) | encode2(v[2] * inv, v[3] * inv) << 16;
  r.y = encode2(v[4] * inv, v[5] * inv) | encode2(v[6] * inv, v[7] * inv) << 16;
  return r;
}

// fp16 (BF16 false) or bf16 pairs.
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <bool BF16>
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<BF16>(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<BF16>(f[0], f[1]), pack2<BF16>(f[2], f[3]), pack2<BF16>(f[4], f[5]),
                    pack2<BF16>(f[6], f[7]));
}

__device__ __forceinline__ uint32_t top8(const float (&v)[8]) {
  uint32_t t = size_of(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) t = max(t, size_of(v[i]));
  return t;
}
// The same of eight 16-bit values, whose bits are ordered alike.
template <bool BF16>
__device__ __forceinline__ uint32_t top_of_words(uint4 v) {
  constexpr uint32_t kSign = 0x7FFF7FFFu;
  const uint32_t t =
      __vmaxu2(__vmaxu2(v.x & kSign, v.y & kSign), __vmaxu2(v.z & kSign, v.w & kSign));
  const float2 f = unpack2<BF16>(t);
  return max(__float_as_uint(f.x), __float_as_uint(f.y));
}
// Over the sixteen lanes whose eight columns each make up a block.
__device__ __forceinline__ uint32_t top_of_block(uint32_t t) {
#pragma unroll
  for (int o = 8; o; o >>= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, o));
  return t;
}

}  // namespace qfp8
