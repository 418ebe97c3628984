// Quantisation steps of the K/V cache, shared by the kernels that write it.
//
// Two formats.  FP8: one f32 scale = a / 448 per (token, head) row and e4m3
// codes of x * (448 / a), a the row's largest magnitude.  MXFP4: one
// power-of-two scale 2^s per 32 consecutive elements, kept as the byte s + 127
// (e8m0), and e2m1 codes of x * 2^-s, two per byte (the even element in the
// low nibble), with the least s such that a / 2^s <= 6, the largest e2m1
// value: no element saturates, where s = floor(log2 a) - 2 would clip a / 2^s
// in (6, 8).  Both round to nearest even.  a is taken as at least 2^-100 and
// at most the largest f32, so every scale and reciprocal is a normal f32 (a
// row of zeros has a positive scale and reads back as zeros; an infinite
// element takes the largest code).
#pragma once

#include <cuda_fp4.h>

#include "nr_internal.h"
#include "nr_pairs.cuh"

namespace nr {

constexpr float kScaleFloor = 0x1p-100f;
constexpr float kScaleCeil = 3.402823466e38f;

// Largest of the values' magnitudes (a NaN counts as nothing).
template <int N>
__device__ __forceinline__ float max_abs(const float (&x)[N]) {
  float a = 0.0f;
#pragma unroll
  for (int e = 0; e < N; e++) a = fmaxf(a, fabsf(x[e]));
  return a;
}

// Butterfly maximum over groups of `width` consecutive lanes.
template <int width>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int m = width / 2; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, m));
  return v;
}

__device__ __forceinline__ float clamp_scale(float a) {
  return fminf(fmaxf(a, kScaleFloor), kScaleCeil);
}

// a / 448 correctly rounded, without a division: q = a * RN(1/448) corrected by
// its remainder a - 448 q, which is exact (Markstein's method of dividing with a
// fused multiply-add).  The outcome depends on a's 2^23 significands alone while
// nothing underflows; a test compares every one of them with the division, at the
// least, the largest and other binades of a.
__device__ __forceinline__ float fp8_scale(float a) {
  constexpr float r = 1.0f / 448.0f;
  const float q = a * r;
  return fmaf(fmaf(-448.0f, q, a), r, q);
}
__device__ __forceinline__ float fp8_inverse(float a) { return __fdiv_rn(448.0f, a); }

// e4m3 codes of N values times `inv`, four to a word.
template <int N>
__device__ __forceinline__ void fp8_codes(const float (&x)[N], float inv, uint32_t (&c)[N / 4]) {
#pragma unroll
  for (int j = 0; j < N / 4; j++)
    c[j] = e4m3x2(x[4 * j] * inv, x[4 * j + 1] * inv) |
           e4m3x2(x[4 * j + 2] * inv, x[4 * j + 3] * inv) << 16;
}

// The same of values that have been multiplied already.
template <int N>
__device__ __forceinline__ void fp8_codes_scaled(const float (&x)[N], uint32_t (&c)[N / 4]) {
#pragma unroll
  for (int j = 0; j < N / 4; j++)
    c[j] = e4m3x2(x[4 * j], x[4 * j + 1]) | e4m3x2(x[4 * j + 2], x[4 * j + 3]) << 16;
}

// The e8m0 byte s + 127 of a normal a > 0: a = 1.m * 2^e gives s = e - 2 up to
// 1.m = 1.5 (a / 2^s = 6) and e - 1 above it.
__device__ __forceinline__ uint32_t mx_scale_byte(float a) {
  const uint32_t bits = __float_as_uint(a);
  return (bits >> 23) - 2u + ((bits & 0x7FFFFFu) > 0x400000u ? 1u : 0u);
}
// 2^-s and 2^s of a byte s + 127 in [1, 253].
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// e2m1 codes of N values times `inv`, N / 2 bytes in the low end of the word.
template <int N>
__device__ __forceinline__ uint32_t fp4_codes(const float (&x)[N], float inv) {
  static_assert(N == 4 || N == 8, "a word holds at most eight codes");
  uint32_t c = 0;
#pragma unroll
  for (int j = 0; j < N / 2; j++)
    c |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(
             make_float2(x[2 * j] * inv, x[2 * j + 1] * inv), __NV_E2M1, cudaRoundNearest))
         << (8 * j);
  return c;
}

// n / d for 0 <= n < 2^31 by a multiplication (d >= 1), the method of Granlund and
// Montgomery for divisions by an invariant integer: with s = ceil(log2 d)
// and m = floor(2^(31 + s) / d) + 1, floor(n m / 2^(31 + s)) is exact for such n.
struct FastDiv {
  uint32_t mul, shift, div;
  __host__ explicit FastDiv(uint32_t d) : mul(0), shift(0), div(d) {
    if (d <= 1) return;
    uint32_t s = 0;
    while ((uint64_t(1) << s) < d) s++;
    mul = static_cast<uint32_t>((uint64_t(1) << (31 + s)) / d + 1);
    shift = s - 1;
  }
  __device__ __forceinline__ uint32_t quot(uint32_t n) const {
    return mul == 0 ? n : __umulhi(n, mul) >> shift;
  }
};

// A cache as the kernels see it: codes and scales of K or of V.
struct CacheSide {
  unsigned char* codes;
  unsigned char* scales;
};

// Byte offsets of one slot (token place) of the paged cache.
struct CacheGeom {
  int64_t slots;               // blocks * block_size
  int64_t code_block_stride;   // bytes between blocks
  int64_t scale_block_stride;  // bytes between blocks
  int64_t code_row;            // bytes of one slot's codes (all heads)
  int64_t scale_row;           // bytes of one slot's scales
  int64_t block_size;
  int shift;  // log2(block_size), or -1

  __device__ __forceinline__ int64_t block_of(int64_t slot) const {
    return shift >= 0 ? slot >> shift : slot / block_size;
  }
};

inline CacheGeom cache_geometry(const KvCacheArgs& c) {
  CacheGeom g;
  g.slots = c.blocks * c.block_size;
  g.code_block_stride = c.code_block_stride;
  g.scale_block_stride = c.scale_block_stride;
  g.code_row = c.heads * (c.fp4 ? c.head_dim / 2 : c.head_dim);
  g.scale_row = c.heads * (c.fp4 ? c.head_dim / 32 : 4);
  g.block_size = c.block_size;
  g.shift = -1;
  for (int i = 0; i < 62; i++)
    if ((int64_t(1) << i) == c.block_size) g.shift = i;
  return g;
}

}  // namespace nr
