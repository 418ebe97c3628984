// Device helpers of the cache and group-norm kernels: 32-byte accesses and
// pairwise f32 arithmetic (sm_103a).
#pragma once

#include "nr_common.cuh"

namespace nr {

// ld_stream and st_stream of 32 bytes (32-byte aligned).
__device__ __forceinline__ void ld_stream32(const void* p, uint4& a, uint4& b) {
  asm volatile(
      "ld.global.L1::no_allocate.L2::256B.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
      : "l"(p));
}
__device__ __forceinline__ void st_stream32(void* p, uint4 a, uint4 b) {
  asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// Two f32 values side by side; one instruction works on both, each rounded as
// the f32 operation is.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(F2 a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 sub2(F2 a, F2 b) {
  F2 r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

template <int P>
__device__ __forceinline__ void from_pairs(const F2 (&p)[P], float (&v)[2 * P]) {
#pragma unroll
  for (int i = 0; i < P; i++) split(p[i], v[2 * i], v[2 * i + 1]);
}

// A 128-bit vector as pairs of values.
template <typename T>
struct Pairs {
  static constexpr int N = Vec<T>::N / 2;
  __device__ __forceinline__ static void unpack(const uint4& v, F2 (&p)[N]) {
    float f[Vec<T>::N];
    Vec<T>::unpack(v, f);
#pragma unroll
    for (int i = 0; i < N; i++) p[i] = f2(f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ static uint4 pack(const F2 (&p)[N]) {
    float f[Vec<T>::N];
#pragma unroll
    for (int i = 0; i < N; i++) split(p[i], f[2 * i], f[2 * i + 1]);
    return Vec<T>::pack(f);
  }
};

template <int P>
__device__ __forceinline__ void to_pairs(const float (&v)[2 * P], F2 (&p)[P]) {
#pragma unroll
  for (int i = 0; i < P; i++) p[i] = f2(v[2 * i], v[2 * i + 1]);
}

}  // namespace nr
