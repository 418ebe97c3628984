// RMSNorm with the optional residual add and an e4m3 output whose scales come from
// the data (sm_103a).
//
// With v = round(x + residual) (written back) and n = v / sqrt(mean v^2 + eps) * w
// in f32, not rounded, a the largest |n| of a scale's extent, clamped as the cache's
// (quant.cuh):
//   row, group   scale = a / 448, code = e4m3(n * (448 / a)); a row, or 128 elements
//   mx           the least s with a / 2^s <= 448, byte s + 127, code = e4m3(n / 2^s);
//                32 elements (OCP MXFP8)
//
// A row is held in registers: read once, its residual, codes and scales written
// once.  HBM bounds many rows, one row's chain of loads and reductions a few.  A row's
// scale needs no second reduction: 1 / sqrt(...) is common to all of it and
// cancels in n * (448 / a), so max |v w| is reduced together with the sum of squares.
// Measured: bf16 [8192, 5120] with the residual, a scale for 128: 47.0 us (0.93 of the copy rate);
// f32 [2049, 4096], mx: 8.4 us (0.74, one wave of blocks and its ramp); bf16 [8, 5120]: 2.1 us, latency.
// (With f32 arithmetic one value at a time instead of pairs: 47.3, 8.8 and 2.2 us.)
#include <type_traits>

#include "nr_pairs.cuh"
#include "quant.cuh"

namespace nr {
namespace {

enum ScaleMode { kRow, kGroup, kMx };

constexpr int kManyThreads = 256;   // threads a row with many rows
constexpr int kFewThreads = 1024;   // and with few

struct QuantArgs {
  uint8_t* codes;
  void* scales;
  const void* x;
  const void* w;
  void* res;
  int nvec;
  float hidden, inv_hidden, eps, w_add;
  int64_t rows;
  int64_t prefetch_rows;
};

// One Newton step on the hardware's reciprocal square root: the error of n decides
// how many codes fall on the other side of a rounding border.
__device__ __forceinline__ float rstd_refined(float mean_square, float eps) {
  const float v = mean_square + eps, r = rsqrtf(v);
  const float h = fmaf(-0.5f * v * r, r, 0.5f);
  return v > 0.0f && v < kScaleCeil ? fmaf(r, h, r) : r;
}

// Sum and maximum over the block, in warp order, with one barrier.
__device__ __forceinline__ void block_sum_max(float& sum, float& top, float2* scratch) {
  sum = group_sum<kWarp>(sum);
  top = group_max<kWarp>(top);
  const int warp = threadIdx.x / kWarp;
  if (threadIdx.x % kWarp == 0) scratch[warp] = make_float2(sum, top);
  __syncthreads();
  sum = 0.0f, top = 0.0f;
  const int warps = (blockDim.x + kWarp - 1) / kWarp;
  for (int i = 0; i < warps; i++) {
    const float2 v = scratch[i];
    sum += v.x;
    top = fmaxf(top, v.y);
  }
}

template <typename T>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&f)[Vec<T>::N]) {
  uint32_t c[Vec<T>::N / 4];
  fp8_codes_scaled(f, c);
  if constexpr (Vec<T>::N == 8)
    st_stream8(p, make_uint2(c[0], c[1]));
  else
    st_stream4(p, c[0]);
}

// One block a row; thread t owns vectors t, t + blockDim, ...  FEW: the launch has few
// rows, w is loaded with the row (one round trip less), and blocks may be large.
template <typename T, int VPT, bool RES, ScaleMode MODE, bool FEW>
__global__ void __launch_bounds__(FEW ? kFewThreads : kManyThreads)
    rmsnorm_quant_kernel(const QuantArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ float2 scratch[kFewThreads / kWarp];
  __shared__ float2 scratch2[kFewThreads / kWarp];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * a.nvec;  // in vectors
  const uint4* x = static_cast<const uint4*>(a.x) + row;
  uint4* r = RES ? static_cast<uint4*>(a.res) + row : nullptr;
  const uint4* w = static_cast<const uint4*>(a.w);
  uint4 xv[VPT], rv[RES ? VPT : 1], wv[FEW ? VPT : 1];
  pdl_enter();  // before any global read: the previous kernel may still run
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const int i = threadIdx.x + k * blockDim.x;
    if (i < a.nvec) {
      xv[k] = ld_stream(x + i);
      if (RES) rv[RES ? k : 0] = ld_stream(r + i);
      if (FEW) wv[FEW ? k : 0] = ld_param(w + i);
    }
  }
  if (!FEW && threadIdx.x == 0 && blockIdx.x + a.prefetch_rows < a.rows) {
    bulk_prefetch_l2(x + a.prefetch_rows * a.nvec, static_cast<unsigned>(a.nvec) * 16u);
    if (RES) bulk_prefetch_l2(r + a.prefetch_rows * a.nvec, static_cast<unsigned>(a.nvec) * 16u);
  }
  F2 squares = f2(0.0f, 0.0f);
  float top = 0.0f;
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const int i = threadIdx.x + k * blockDim.x;
    if (i < a.nvec) {
      float v[N];
      Vec<T>::unpack(xv[k], v);
      if (RES) {
        float q[N];
        Vec<T>::unpack(rv[RES ? k : 0], q);
#pragma unroll
        for (int e = 0; e < N; e += 2) split(add2(f2(v[e], v[e + 1]), f2(q[e], q[e + 1])), v[e], v[e + 1]);
        xv[k] = Vec<T>::pack(v);  // rounded: what is written back is what is normed
        st_stream(r + i, xv[k]);
        Vec<T>::unpack(xv[k], v);
      }
#pragma unroll
      for (int e = 0; e < N; e += 2) squares = fma2(f2(v[e], v[e + 1]), f2(v[e], v[e + 1]), squares);
      if (MODE == kRow) {
        float u[N];
        Vec<T>::unpack(FEW ? wv[FEW ? k : 0] : ld_param(w + i), u);
#pragma unroll
        for (int e = 0; e < N; e++) top = fmaxf(top, fabsf(v[e] * (u[e] + a.w_add)));
      }
    }
  }
  float sum, odd;
  split(squares, sum, odd);
  sum += odd;
  block_sum_max(sum, top, scratch);
  float inv;
  {
    const float ms = row_mean_of(sum, a.hidden, a.inv_hidden);
    if (ms + a.eps >= 0x1p-80f && ms <= 0x1p120f) {
      inv = rstd_refined(ms, a.eps);
    } else {  // squares near the ends of f32's range: of scaled values (the same for the block)
      const float f = ms < 1.0f ? 0x1p60f : 0x1p-80f;
      float none = 0.0f;
      sum = 0.0f;
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        const int i = threadIdx.x + k * blockDim.x;
        if (i < a.nvec) {
          float v[N];
          Vec<T>::unpack(xv[k], v);
#pragma unroll
          for (int e = 0; e < N; e++) sum = fmaf(v[e] * f, v[e] * f, sum);
        }
      }
      block_sum_max(sum, none, scratch2);
      inv = rstd_refined(row_mean_of(sum, a.hidden, a.inv_hidden), a.eps * f * f) * f;
      __syncthreads();  // scratch2 may be used again
    }
  }
  // n = (v inv) w, or (row scales) v w with inv in the factor.  The latter loses
  // nothing while v w stays far from the ends of f32's range; a row that does not
  // (a NaN among them) takes its maximum from n.
  float factor = 1.0f, n_inv = inv;
  if (MODE == kRow) {
    float am = top * inv;
    const bool plain = am >= kScaleFloor && am <= kScaleCeil && top > 0x1p-60f && top < 0x1p100f;
    if (plain) {
      factor = __fdiv_rn(448.0f, top);
      n_inv = 1.0f;
    } else {  // the same for the whole block
      am = 0.0f;
      float none = 0.0f;
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        const int i = threadIdx.x + k * blockDim.x;
        if (i < a.nvec) {
          float v[N], u[N];
          Vec<T>::unpack(xv[k], v);
          Vec<T>::unpack(FEW ? wv[FEW ? k : 0] : ld_param(w + i), u);
#pragma unroll
          for (int e = 0; e < N; e++) am = fmaxf(am, fabsf(v[e] * inv * (u[e] + a.w_add)));
        }
      }
      block_sum_max(none, am, scratch2);
      am = clamp_scale(am);
      factor = fp8_inverse(am);
    }
    if (threadIdx.x == 0) static_cast<float*>(a.scales)[blockIdx.x] = fp8_scale(am);
  }
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const int i = threadIdx.x + k * blockDim.x;
    float v[N], u[N];
    const bool in = i < a.nvec;
    if (in) {
      Vec<T>::unpack(xv[k], v);
      Vec<T>::unpack(FEW ? wv[FEW ? k : 0] : ld_param(w + i), u);
#pragma unroll
      for (int e = 0; e < N; e += 2)
        split(mul2(mul2(f2(v[e], v[e + 1]), f2(n_inv, n_inv)),
                   add2(f2(u[e], u[e + 1]), f2(a.w_add, a.w_add))), v[e], v[e + 1]);
    } else {
#pragma unroll
      for (int e = 0; e < N; e++) v[e] = 0.0f;
    }
    if (MODE != kRow) {
      // a scale's extent is `lanes` neighbouring vectors, in neighbouring lanes; it ends
      // with the row, whose last lanes join the butterfly with zeros
      constexpr int lanes = (MODE == kGroup ? 128 : 32) / N;
      const float am = clamp_scale(group_max<lanes>(max_abs(v)));
      if (!in) continue;
      const int64_t at = row / lanes + i / lanes;
      const bool first = i % lanes == 0;
      if (MODE == kGroup) {
        factor = fp8_inverse(am);
        if (first) static_cast<float*>(a.scales)[at] = fp8_scale(am);
      } else {
        // a = 1.m 2^e: s = e - 8 up to 1.m = 1.75 (a / 2^s = 448), e - 7 above it
        const uint32_t bits = __float_as_uint(am);
        const uint32_t byte = (bits >> 23) - 8u + ((bits & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
        factor = mx_inverse(byte);
        if (first) static_cast<uint8_t*>(a.scales)[at] = static_cast<uint8_t>(byte);
      }
    }
    if (!in) continue;
#pragma unroll
    for (int e = 0; e < N; e += 2)
      split(mul2(f2(v[e], v[e + 1]), f2(factor, factor)), v[e], v[e + 1]);
    store_codes<T>(a.codes + (row + i) * N, v);
  }
}

template <typename T, int VPT, bool RES, ScaleMode MODE, bool FEW>
cudaError_t go(QuantArgs a, int threads, cudaStream_t s) {
  auto kernel = rmsnorm_quant_kernel<T, VPT, RES, MODE, FEW>;
  a.prefetch_rows = a.rows;
  if (!FEW) {
    static std::atomic<int> cache[64];
    int resident = 0;
    const cudaError_t e = resident_blocks(kernel, threads, cache, &resident);
    if (e != cudaSuccess) return e;
    a.prefetch_rows = resident;
  }
  return launch_pdl(kernel, dim3(static_cast<unsigned>(a.rows)), dim3(threads), 0, s, a);
}

template <typename T, bool RES, ScaleMode MODE>
cudaError_t go_rows(const QuantArgs& a, cudaStream_t s) {
  const int n = a.nvec;
  auto threads = [n](int vpt) { return ((n + vpt - 1) / vpt + 31) / 32 * 32; };
  // Few rows: short chains, one or two vectors a thread.  The borders are nr_rmsnorm's
  // (measured there for the same loads and reduction).
  if (a.rows <= 256) {
    if (n <= 256 || (n <= 512 && a.rows <= 32)) return go<T, 1, RES, MODE, true>(a, threads(1), s);
    if (n <= 2 * kFewThreads) return go<T, 2, RES, MODE, true>(a, threads(2), s);
  }
  if (n <= 128) return go<T, 1, RES, MODE, false>(a, threads(1), s);
  if (n <= 512) return go<T, 2, RES, MODE, false>(a, threads(2), s);
  if (n <= 1024) return go<T, 4, RES, MODE, false>(a, threads(4), s);
  if (n <= 2048) return go<T, 8, RES, MODE, false>(a, threads(8), s);
  return go<T, 16, RES, MODE, false>(a, threads(16), s);
}

template <typename T>
cudaError_t go_mode(const QuantArgs& a, int mode, cudaStream_t s) {
  const bool res = a.res != nullptr;
  if (mode == kRow) return res ? go_rows<T, true, kRow>(a, s) : go_rows<T, false, kRow>(a, s);
  if (mode == kGroup) return res ? go_rows<T, true, kGroup>(a, s) : go_rows<T, false, kGroup>(a, s);
  return res ? go_rows<T, true, kMx>(a, s) : go_rows<T, false, kMx>(a, s);
}

}  // namespace

cudaError_t launch_rmsnorm_quant(void* codes, void* scales, const void* x, const void* w,
                                 void* residual, int64_t rows, int64_t hidden, int is_bf16,
                                 float eps, int gemma, int mode, cudaStream_t stream) {
  QuantArgs a = {};
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.x = x;
  a.w = w;
  a.res = residual;
  a.nvec = static_cast<int>(hidden / (is_bf16 ? 8 : 4));
  a.hidden = static_cast<float>(hidden);
  a.inv_hidden = 1.0f / a.hidden;
  a.eps = eps;
  a.w_add = gemma ? 1.0f : 0.0f;
  a.rows = rows;
  return is_bf16 ? go_mode<__nv_bfloat16>(a, mode, stream) : go_mode<float>(a, mode, stream);
}

}  // namespace nr
