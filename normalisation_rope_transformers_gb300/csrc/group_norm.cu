// Group norm with an optional SiLU over channels-last tensors, and its
// gradient, for sm_103a.
//
// x is [samples, space, channels] (channels contiguous).  Per sample and group
// of cpg = channels / groups channels, over the space * cpg values of the group:
//     xhat = (x - mean) * rstd,  z = xhat * w_c + b_c,  y = z or silu(z)
// and backwards, with dz = dy * act'(z), S1_c = sum dz, S2_c = sum dz * xhat:
//     db_c = sum_n S1,  dw_c = sum_n S2,
//     dx = rstd * (w_c dz - mean_g(w dz) - xhat * mean_g(w dz xhat))
//
// A group's values are strided by `channels`, so its statistics need the whole
// sample: the tensor is read twice (statistics, then the output) and written
// once, and HBM bounds every pass.  A block owns a range of rows (a chunk) and
// a tile of vector columns; each thread keeps one 128-bit column of N channels
// and walks down the rows, so all reads are whole rows, each value belongs to
// a fixed channel register, and any channels / groups works (a vector may span
// several groups).  Blocks write partial results, a small kernel joins them in
// a fixed order (no atomics: the same inputs give the same bits), and the
// output pass walks each chunk from its end, so that what the statistics pass
// read last is still in L2.
#include "nr_common.cuh"
#include "nr_internal.h"

namespace nr {
namespace {

constexpr int kGnThreads = 256;
// Blocks that the geometry aims at: as many as the kernels' registers let
// reside on 152 SMs, so that a pass is one wave.
constexpr int kGnPerSm = 3, kGnGradPerSm = 2;
// Rows that a thread loads before it works on them (backward: of each tensor).
constexpr int kGnRows = 8, kGnGradRows = 4;

// Columns and rows of one launch; the same for every pass of a call.
struct GnGeom {
  int64_t space;
  int64_t rows;  // rows of a chunk (the last one may be shorter)
  int channels, groups, cpg;
  int cols;       // 128-bit vectors of a row
  int tile_cols;  // vector columns of a block
  int tiles;
  int lanes;  // rows that a block reads at once
  int chunks;
};

GnGeom gn_geometry(int64_t samples, int64_t space, int64_t channels, int64_t groups, int vec,
                   int per_sm) {
  GnGeom g;
  g.space = space;
  g.channels = static_cast<int>(channels);
  g.groups = static_cast<int>(groups);
  g.cpg = static_cast<int>(channels / groups);
  g.cols = static_cast<int>(channels / vec);
  g.tiles = (g.cols + kGnThreads - 1) / kGnThreads;
  g.tile_cols = (g.cols + g.tiles - 1) / g.tiles;
  g.lanes = kGnThreads / g.tile_cols;
  // at least four rows a thread, so that its loads overlap
  const int64_t most = (space + 4 * g.lanes - 1) / (4 * g.lanes);
  int64_t want = 152 * per_sm / (samples * g.tiles);
  want = want < 1 ? 1 : want > most ? most : want;
  g.rows = (space + want - 1) / want;
  g.chunks = static_cast<int>((space + g.rows - 1) / g.rows);
  return g;
}

// Where a block stands: sample, chunk, and this thread's column and row lane.
struct GnPlace {
  int64_t sample, row0, row1;  // rows of the chunk
  int chunk, tile, col, lane, channel;
  bool active;
  __device__ __forceinline__ GnPlace(const GnGeom& g, unsigned block, int vec) {
    tile = static_cast<int>(block % g.tiles);
    const unsigned rest = block / g.tiles;
    chunk = static_cast<int>(rest % g.chunks);
    sample = rest / g.chunks;
    row0 = chunk * g.rows;
    row1 = min(row0 + g.rows, g.space);
    lane = threadIdx.x / g.tile_cols;
    col = tile * g.tile_cols + static_cast<int>(threadIdx.x) % g.tile_cols;
    active = col < g.cols;
    channel = col * vec;
  }
};

// A parameter vector's N values of this thread's channels (`none` without one).
template <int N>
__device__ __forceinline__ void gn_params(const void* p, int is_bf16, int channel, float none,
                                          float (&v)[N]) {
#pragma unroll
  for (int e = 0; e < N; e++) {
    if (p == nullptr)
      v[e] = none;
    else if (is_bf16)
      v[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(p)[channel + e]);
    else
      v[e] = static_cast<const float*>(p)[channel + e];
  }
}

// sigmoid(z).  Where the result is rounded to bf16: the hardware exponential
// and reciprocal (each about 2^-22), two instructions of the special unit a
// value; below z = -88 the exponential is infinite and the sigmoid zero, off by
// less than 2^-126.  For f32 from t = e^-|z|, which never overflows.
template <typename T>
__device__ __forceinline__ float gn_sigmoid(float z);
template <>
__device__ __forceinline__ float gn_sigmoid<__nv_bfloat16>(float z) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
  return s;
}
template <>
__device__ __forceinline__ float gn_sigmoid<float>(float z) {
  const float t = expf(-fabsf(z));
  return z >= 0.0f ? 1.0f / (1.0f + t) : t / (1.0f + t);
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
// Mean and sum of squared deviations (M2) of each group's part in this block.
// A thread sums each channel's values minus the first of them that it sees, so
// a channel far from zero cancels nothing and one outlier spoils no other
// thread's sums; parts are joined by their means and counts (the update of
// Chan, Golub and LeVeque).  A group that lies in two tiles has a part in each:
// part (group, tile) is at place group + tile, which no other part has, as the
// groups of a tile are never below those of the tile before.
template <typename T>
__global__ void __launch_bounds__(kGnThreads, kGnPerSm) gn_stats_kernel(float2* __restrict__ parts,
                                                              const T* __restrict__ x,
                                                              const GnGeom g) {
  constexpr int N = Vec<T>::N;
  __shared__ float2 sm[kGnThreads * N];  // [lane][channel of the tile]: mean, M2
  pdl_enter();
  const GnPlace at(g, blockIdx.x, N);
  const int width = g.tile_cols * N;
  if (at.active && at.lane < g.lanes) {
    float first[N], s1[N], s2[N];
#pragma unroll
    for (int e = 0; e < N; e++) first[e] = s1[e] = s2[e] = 0.0f;
    const int64_t step = static_cast<int64_t>(g.lanes) * g.cols;
    const uint4* p = reinterpret_cast<const uint4*>(x) +
                     (at.sample * g.space + at.row0 + at.lane) * g.cols + at.col;
    const int rows = static_cast<int>(at.row1 - at.row0);
    int count = 0;
    for (int r = at.lane; r < rows; r += kGnRows * g.lanes) {
      uint4 v[kGnRows];
#pragma unroll
      for (int u = 0; u < kGnRows; u++, p += step)
        if (r + u * g.lanes < rows) v[u] = ld_stream(p);
      if (count == 0) Vec<T>::unpack(v[0], first);
#pragma unroll
      for (int u = 0; u < kGnRows; u++)
        if (r + u * g.lanes < rows) {
          float f[N];
          Vec<T>::unpack(v[u], f);
#pragma unroll
          for (int e = 0; e < N; e++) {
            const float d = f[e] - first[e];
            s1[e] += d;
            s2[e] = fmaf(d, d, s2[e]);
          }
          count++;
        }
    }
    const float inv = count > 0 ? 1.0f / static_cast<float>(count) : 0.0f;
    float2* o = sm + at.lane * width + (at.channel - at.tile * width);
#pragma unroll
    for (int e = 0; e < N; e++)
      o[e] = make_float2(fmaf(s1[e], inv, first[e]), fmaf(-s1[e] * inv, s1[e], s2[e]));
  }
  __syncthreads();
  // one warp a group: the lanes' parts of its channels that are in this tile
  const int c0 = at.tile * width, c1 = min(c0 + width, g.channels);
  const int g0 = c0 / g.cpg, g1 = (c1 - 1) / g.cpg;
  const int warp = threadIdx.x / kWarp, lane32 = threadIdx.x % kWarp;
  const int warps = (blockDim.x + kWarp - 1) / kWarp;
  const int span = static_cast<int>(at.row1 - at.row0);
  for (int grp = g0 + warp; grp <= g1; grp += warps) {
    const int a = max(c0, grp * g.cpg), b = min(c1, (grp + 1) * g.cpg);
    const int n = (b - a) * g.lanes;
    // rows of lane i: those i, i + lanes, ... of the chunk
    auto rows_of = [&](int i) { return i < span ? (span - 1 - i) / g.lanes + 1 : 0; };
    float s = 0.0f;
    for (int i = lane32; i < n; i += kWarp) {
      const int l = i / (b - a);
      s = fmaf(static_cast<float>(rows_of(l)), sm[l * width + a - c0 + i - l * (b - a)].x, s);
    }
    const float total = static_cast<float>(span) * static_cast<float>(b - a);
    const float mean = __fdiv_rn(group_sum<kWarp>(s), total);
    float m2 = 0.0f;
    for (int i = lane32; i < n; i += kWarp) {
      const int l = i / (b - a);
      const float2 v = sm[l * width + a - c0 + i - l * (b - a)];
      const float d = v.x - mean, k = static_cast<float>(rows_of(l));
      if (k > 0.0f) m2 += fmaf(k * d, d, v.y);
    }
    m2 = group_sum<kWarp>(m2);
    if (lane32 == 0)
      parts[(at.sample * g.chunks + at.chunk) * (g.groups + g.tiles) + grp + at.tile] =
          make_float2(mean, m2);
  }
}

constexpr int kGnJoinThreads = 128;

// One block a (sample, group): joins its parts into mean and rstd.
__global__ void __launch_bounds__(kGnJoinThreads) gn_join_kernel(float* __restrict__ mean_out,
                                                                 float* __restrict__ rstd_out,
                                                                 const float2* __restrict__ parts,
                                                                 const GnGeom g, int width,
                                                                 float eps) {
  __shared__ float scratch[2][kGnJoinThreads / kWarp];
  pdl_enter();
  const int64_t sample = blockIdx.x / g.groups;
  const int grp = static_cast<int>(blockIdx.x % g.groups);
  const int ca = grp * g.cpg, cb = ca + g.cpg;  // the group's channels
  const int t0 = ca / width, t1 = (cb - 1) / width;
  const int per = t1 - t0 + 1;
  const int n = g.chunks * per;
  const float2* p = parts + sample * g.chunks * (g.groups + g.tiles) + grp;
  auto part = [&](int i, float& count) {
    const int chunk = i / per, tile = t0 + i % per;
    const int64_t rows = min(g.rows, g.space - chunk * g.rows);
    count = static_cast<float>(rows) *
            static_cast<float>(min(cb, (tile + 1) * width) - max(ca, tile * width));
    return p[static_cast<int64_t>(chunk) * (g.groups + g.tiles) + tile];
  };
  float s = 0.0f, count;
  for (int i = threadIdx.x; i < n; i += kGnJoinThreads) {
    const float2 v = part(i, count);
    s = fmaf(count, v.x, s);
  }
  const float total = static_cast<float>(g.space) * static_cast<float>(g.cpg);
  const float mean = __fdiv_rn(block_sum(s, scratch[0]), total);
  float m2 = 0.0f;
  for (int i = threadIdx.x; i < n; i += kGnJoinThreads) {
    const float2 v = part(i, count);
    const float d = v.x - mean;
    m2 += fmaf(count * d, d, v.y);
  }
  m2 = block_sum(m2, scratch[1]);
  m2 = m2 < 0.0f ? 0.0f : m2;  // a part's rounding may leave a constant group just below zero
  if (threadIdx.x == 0) {
    mean_out[blockIdx.x] = mean;
    rstd_out[blockIdx.x] = 1.0f / sqrtf(__fdiv_rn(m2, total) + eps);
  }
}

struct GnParams {
  const void* w;
  const void* b;
  int is_bf16;
};

template <typename T, bool SILU>
__global__ void __launch_bounds__(kGnThreads, kGnPerSm) gn_apply_kernel(T* __restrict__ out,
                                                              const T* __restrict__ x,
                                                              const float* __restrict__ mean,
                                                              const float* __restrict__ rstd,
                                                              const GnParams prm, const GnGeom g) {
  constexpr int N = Vec<T>::N;
  pdl_enter();
  const GnPlace at(g, gridDim.x - 1 - blockIdx.x, N);
  if (!at.active || at.lane >= g.lanes) return;
  float mu[N], a[N], b[N];
  gn_params<N>(prm.w, prm.is_bf16, at.channel, 1.0f, a);
  gn_params<N>(prm.b, prm.is_bf16, at.channel, 0.0f, b);
#pragma unroll
  for (int e = 0; e < N; e++) {
    const int64_t i = at.sample * g.groups + (at.channel + e) / g.cpg;
    mu[e] = mean[i];
    a[e] *= rstd[i];
  }
  const int64_t step = static_cast<int64_t>(g.lanes) * g.cols;
  const int rows = static_cast<int>(at.row1 - at.row0);
  const int64_t base = (at.sample * g.space + at.row1 - 1 - at.lane) * g.cols + at.col;
  const uint4* p = reinterpret_cast<const uint4*>(x) + base;
  uint4* o = reinterpret_cast<uint4*>(out) + base;
  for (int r = at.lane; r < rows; r += kGnRows * g.lanes) {
    uint4 v[kGnRows];
#pragma unroll
    for (int u = 0; u < kGnRows; u++, p -= step)
      if (r + u * g.lanes < rows) v[u] = ld_stream(p);
#pragma unroll
    for (int u = 0; u < kGnRows; u++, o -= step)
      if (r + u * g.lanes < rows) {
        float f[N];
        Vec<T>::unpack(v[u], f);
#pragma unroll
        for (int e = 0; e < N; e++) {
          const float z = fmaf(f[e] - mu[e], a[e], b[e]);
          f[e] = SILU ? z * gn_sigmoid<T>(z) : z;
        }
        st_stream(o, Vec<T>::pack(f));
      }
  }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
// dz = dy * act'(z); silu'(z) = s (1 + z (1 - s)) with s = sigmoid(z).
template <typename T, bool SILU>
__device__ __forceinline__ float gn_dz(float dy, float z) {
  if (!SILU) return dy;
  const float s = gn_sigmoid<T>(z);
  return dy * (s * fmaf(z, 1.0f - s, 1.0f));
}

struct GnGradIn {
  const void* dy;
  const void* x;
  const float* mean;
  const float* rstd;
  GnParams prm;
};

// Per channel and chunk: sum dz and sum dz * (x - mean).
template <typename T, bool SILU>
__global__ void __launch_bounds__(kGnThreads, kGnGradPerSm) gn_grad_stats_kernel(float2* __restrict__ parts,
                                                                   const GnGradIn in,
                                                                   const GnGeom g) {
  constexpr int N = Vec<T>::N;
  __shared__ float2 sm[kGnThreads * N];
  pdl_enter();
  const GnPlace at(g, blockIdx.x, N);
  const int width = g.tile_cols * N;
  if (at.active && at.lane < g.lanes) {
    float mu[N], a[N], b[N], s1[N], s2[N];
    gn_params<N>(in.prm.w, in.prm.is_bf16, at.channel, 1.0f, a);
    gn_params<N>(in.prm.b, in.prm.is_bf16, at.channel, 0.0f, b);
#pragma unroll
    for (int e = 0; e < N; e++) {
      const int64_t i = at.sample * g.groups + (at.channel + e) / g.cpg;
      mu[e] = in.mean[i];
      a[e] *= in.rstd[i];
      s1[e] = s2[e] = 0.0f;
    }
    const int64_t step = static_cast<int64_t>(g.lanes) * g.cols;
    const int rows = static_cast<int>(at.row1 - at.row0);
    const int64_t base = (at.sample * g.space + at.row0 + at.lane) * g.cols + at.col;
    const uint4* px = static_cast<const uint4*>(in.x) + base;
    const uint4* pd = static_cast<const uint4*>(in.dy) + base;
    for (int r = at.lane; r < rows; r += kGnGradRows * g.lanes) {
      uint4 vx[kGnGradRows], vd[kGnGradRows];
#pragma unroll
      for (int u = 0; u < kGnGradRows; u++, px += step, pd += step)
        if (r + u * g.lanes < rows) {
          vx[u] = ld_stream(px);
          vd[u] = ld_stream(pd);
        }
#pragma unroll
      for (int u = 0; u < kGnGradRows; u++)
        if (r + u * g.lanes < rows) {
          float f[N], d[N];
          Vec<T>::unpack(vx[u], f);
          Vec<T>::unpack(vd[u], d);
#pragma unroll
          for (int e = 0; e < N; e++) {
            const float c = f[e] - mu[e];
            const float dz = gn_dz<T, SILU>(d[e], fmaf(c, a[e], b[e]));
            s1[e] += dz;
            s2[e] = fmaf(dz, c, s2[e]);
          }
        }
    }
    float2* o = sm + at.lane * width + (at.channel - at.tile * width);
#pragma unroll
    for (int e = 0; e < N; e++) o[e] = make_float2(s1[e], s2[e]);
  }
  __syncthreads();
  const int c0 = at.tile * width, c1 = min(c0 + width, g.channels);
  for (int c = threadIdx.x; c < c1 - c0; c += blockDim.x) {
    float2 s = make_float2(0.0f, 0.0f);
    for (int l = 0; l < g.lanes; l++) {
      const float2 v = sm[l * width + c];
      s.x += v.x;
      s.y += v.y;
    }
    parts[(at.sample * g.chunks + at.chunk) * g.channels + c0 + c] = s;
  }
}

constexpr int kGnSumLanes = 32;  // chunk lanes of the joining block (x 32 channels)

// Sums the chunks of 32 channels of one sample: S1 and S2 (with xhat) per channel.
__global__ void __launch_bounds__(32 * kGnSumLanes) gn_grad_join_kernel(
    float2* __restrict__ sums, const float2* __restrict__ parts, const float* __restrict__ rstd,
    const GnGeom g) {
  __shared__ float2 sm[kGnSumLanes][32 + 1];
  pdl_enter();
  const int blocks = (g.channels + 31) / 32;
  const int64_t sample = blockIdx.x / blocks;
  const int c = static_cast<int>(blockIdx.x % blocks) * 32 + threadIdx.x % 32;
  const int lane = threadIdx.x / 32;
  float2 s = make_float2(0.0f, 0.0f);
  if (c < g.channels)
    for (int k = lane; k < g.chunks; k += kGnSumLanes) {
      const float2 v = parts[(sample * g.chunks + k) * g.channels + c];
      s.x += v.x;
      s.y += v.y;
    }
  sm[lane][threadIdx.x % 32] = s;
  __syncthreads();
  // warp `lane` joins channel `lane` of the block
  float2 v = sm[threadIdx.x % 32][lane];
  v.x = group_sum<32>(v.x);
  v.y = group_sum<32>(v.y);
  const int mine = static_cast<int>(blockIdx.x % blocks) * 32 + lane;
  if (threadIdx.x % 32 == 0 && mine < g.channels)
    sums[sample * g.channels + mine] =
        make_float2(v.x, v.y * rstd[sample * g.groups + mine / g.cpg]);
}

template <typename T, bool SILU>
__global__ void __launch_bounds__(kGnThreads, kGnGradPerSm) gn_grad_apply_kernel(
    T* __restrict__ dx, void* __restrict__ dw, void* __restrict__ db,
    const float2* __restrict__ sums, const GnGradIn in, const GnGeom g, int samples) {
  constexpr int N = Vec<T>::N;
  // mean_g(w dz) and mean_g(w dz xhat) of the groups that this tile touches
  extern __shared__ float2 grp_mean[];
  pdl_enter();
  const GnPlace at(g, gridDim.x - 1 - blockIdx.x, N);
  const int width = g.tile_cols * N;
  const int c0 = at.tile * width, c1 = min(c0 + width, g.channels);
  const int g0 = c0 / g.cpg, g1 = (c1 - 1) / g.cpg;
  const int warp = threadIdx.x / kWarp, lane32 = threadIdx.x % kWarp;
  const int warps = (blockDim.x + kWarp - 1) / kWarp;
  const float inv = 1.0f / (static_cast<float>(g.space) * static_cast<float>(g.cpg));
  auto weight = [&](int c) {
    float v[1];
    gn_params<1>(in.prm.w, in.prm.is_bf16, c, 1.0f, v);
    return v[0];
  };
  for (int grp = g0 + warp; grp <= g1; grp += warps) {
    float m1 = 0.0f, m2 = 0.0f;
    for (int i = lane32; i < g.cpg; i += kWarp) {
      const int c = grp * g.cpg + i;
      const float2 v = sums[at.sample * g.channels + c];
      const float w = weight(c);
      m1 = fmaf(w, v.x, m1);
      m2 = fmaf(w, v.y, m2);
    }
    m1 = group_sum<kWarp>(m1);
    m2 = group_sum<kWarp>(m2);
    if (lane32 == 0) grp_mean[grp - g0] = make_float2(m1 * inv, m2 * inv);
  }
  // the first chunk's blocks of sample 0 also write their channels' dw and db
  if (at.sample == 0 && at.chunk == 0 && dw != nullptr)
    for (int c = c0 + threadIdx.x; c < c1; c += blockDim.x) {
      float2 s = make_float2(0.0f, 0.0f);
      for (int n = 0; n < samples; n++) {
        const float2 v = sums[static_cast<int64_t>(n) * g.channels + c];
        s.x += v.x;
        s.y += v.y;
      }
      if (in.prm.is_bf16) {
        static_cast<__nv_bfloat16*>(db)[c] = __float2bfloat16_rn(s.x);
        static_cast<__nv_bfloat16*>(dw)[c] = __float2bfloat16_rn(s.y);
      } else {
        static_cast<float*>(db)[c] = s.x;
        static_cast<float*>(dw)[c] = s.y;
      }
    }
  __syncthreads();
  if (!at.active || at.lane >= g.lanes) return;
  // dx = a dz - k1 - (x - mean) k2 with a = rstd w, k1 = rstd m1, k2 = rstd^2 m2
  float mu[N], a[N], b[N], k1[N], k2[N];
  gn_params<N>(in.prm.w, in.prm.is_bf16, at.channel, 1.0f, a);
  gn_params<N>(in.prm.b, in.prm.is_bf16, at.channel, 0.0f, b);
#pragma unroll
  for (int e = 0; e < N; e++) {
    const int grp = (at.channel + e) / g.cpg;
    const float rs = in.rstd[at.sample * g.groups + grp];
    mu[e] = in.mean[at.sample * g.groups + grp];
    a[e] *= rs;
    k1[e] = rs * grp_mean[grp - g0].x;
    k2[e] = rs * rs * grp_mean[grp - g0].y;
  }
  const int64_t step = static_cast<int64_t>(g.lanes) * g.cols;
  const int rows = static_cast<int>(at.row1 - at.row0);
  const int64_t base = (at.sample * g.space + at.row1 - 1 - at.lane) * g.cols + at.col;
  const uint4* px = static_cast<const uint4*>(in.x) + base;
  const uint4* pd = static_cast<const uint4*>(in.dy) + base;
  uint4* o = reinterpret_cast<uint4*>(dx) + base;
  for (int r = at.lane; r < rows; r += kGnGradRows * g.lanes) {
    uint4 vx[kGnGradRows], vd[kGnGradRows];
#pragma unroll
    for (int u = 0; u < kGnGradRows; u++, px -= step, pd -= step)
      if (r + u * g.lanes < rows) {
        vx[u] = ld_stream(px);
        vd[u] = ld_stream(pd);
      }
#pragma unroll
    for (int u = 0; u < kGnGradRows; u++, o -= step)
      if (r + u * g.lanes < rows) {
        float f[N], d[N];
        Vec<T>::unpack(vx[u], f);
        Vec<T>::unpack(vd[u], d);
#pragma unroll
        for (int e = 0; e < N; e++) {
          const float c = f[e] - mu[e];
          const float dz = gn_dz<T, SILU>(d[e], fmaf(c, a[e], b[e]));
          f[e] = fmaf(a[e], dz, -fmaf(c, k2[e], k1[e]));
        }
        st_stream(o, Vec<T>::pack(f));
      }
  }
}

// Threads of a block: its columns and lanes, in whole warps (the warps of the
// reductions shuffle with every lane).
unsigned gn_threads(const GnGeom& g) {
  return static_cast<unsigned>((g.tile_cols * g.lanes + kWarp - 1) / kWarp * kWarp);
}

unsigned gn_grid(const GnGeom& g, int64_t samples) {
  return static_cast<unsigned>(samples * g.chunks * g.tiles);
}

template <typename T>
cudaError_t gn_forward(const GroupNormArgs& a, cudaStream_t s) {
  const GnGeom g = gn_geometry(a.samples, a.space, a.channels, a.groups, Vec<T>::N, kGnPerSm);
  const GnParams prm{a.w, a.b, a.w_is_bf16};
  float2* parts = static_cast<float2*>(a.workspace);
  const T* x = static_cast<const T*>(a.x);
  const unsigned grid = gn_grid(g, a.samples);
  const unsigned threads = gn_threads(g);
  cudaError_t e = launch_pdl(gn_stats_kernel<T>, dim3(grid), dim3(threads), 0, s, parts, x, g);
  if (e != cudaSuccess) return e;
  e = launch_pdl(gn_join_kernel, dim3(static_cast<unsigned>(a.samples * a.groups)),
                 dim3(kGnJoinThreads), 0, s, a.mean, a.rstd,
                 static_cast<const float2*>(parts), g, g.tile_cols * Vec<T>::N, a.eps);
  if (e != cudaSuccess) return e;
  auto kernel = a.silu ? gn_apply_kernel<T, true> : gn_apply_kernel<T, false>;
  return launch_pdl(kernel, dim3(grid), dim3(threads), 0, s, static_cast<T*>(a.out), x,
                    static_cast<const float*>(a.mean), static_cast<const float*>(a.rstd), prm, g);
}

template <typename T>
cudaError_t gn_backward(const GroupNormArgs& a, cudaStream_t s) {
  const GnGeom g = gn_geometry(a.samples, a.space, a.channels, a.groups, Vec<T>::N, kGnGradPerSm);
  const GnGradIn in{a.dy, a.x, a.mean, a.rstd, GnParams{a.w, a.b, a.w_is_bf16}};
  float2* parts = static_cast<float2*>(a.workspace);
  float2* sums = parts + a.samples * g.chunks * a.channels;
  const unsigned grid = gn_grid(g, a.samples);
  const unsigned threads = gn_threads(g);
  auto stats = a.silu ? gn_grad_stats_kernel<T, true> : gn_grad_stats_kernel<T, false>;
  cudaError_t e = launch_pdl(stats, dim3(grid), dim3(threads), 0, s, parts, in, g);
  if (e != cudaSuccess) return e;
  e = launch_pdl(gn_grad_join_kernel,
                 dim3(static_cast<unsigned>(a.samples * ((a.channels + 31) / 32))),
                 dim3(32 * kGnSumLanes), 0, s, sums, static_cast<const float2*>(parts), a.rstd, g);
  if (e != cudaSuccess) return e;
  auto apply = a.silu ? gn_grad_apply_kernel<T, true> : gn_grad_apply_kernel<T, false>;
  // groups that one tile can touch
  const int width = g.tile_cols * Vec<T>::N;
  const size_t smem = sizeof(float2) * static_cast<size_t>((width - 1) / g.cpg + 2);
  return launch_pdl(apply, dim3(grid), dim3(threads), smem, s, static_cast<T*>(a.out), a.dw, a.db,
                    static_cast<const float2*>(sums), in, g, static_cast<int>(a.samples));
}

}  // namespace

int64_t group_norm_workspace(int64_t samples, int64_t space, int64_t channels, int64_t groups,
                             int is_bf16) {
  const int vec = is_bf16 ? 8 : 4;
  const GnGeom f = gn_geometry(samples, space, channels, groups, vec, kGnPerSm);
  const GnGeom b = gn_geometry(samples, space, channels, groups, vec, kGnGradPerSm);
  const int64_t forward = samples * f.chunks * (groups + f.tiles);
  const int64_t backward = samples * (b.chunks + 1) * channels;
  return static_cast<int64_t>(sizeof(float2)) * (forward > backward ? forward : backward);
}

int64_t group_norm_blocks(int64_t samples, int64_t space, int64_t channels, int64_t groups,
                          int is_bf16) {
  const GnGeom g = gn_geometry(samples, space, channels, groups, is_bf16 ? 8 : 4, kGnPerSm);
  const int64_t blocks = g.chunks * static_cast<int64_t>(g.tiles);
  const int64_t joins = groups > (channels + 31) / 32 ? groups : (channels + 31) / 32;
  return samples * (blocks > joins ? blocks : joins);
}

cudaError_t launch_group_norm(const GroupNormArgs& a, int is_bf16, cudaStream_t stream) {
  return is_bf16 ? gn_forward<__nv_bfloat16>(a, stream) : gn_forward<float>(a, stream);
}

cudaError_t launch_group_norm_backward(const GroupNormArgs& a, int is_bf16, cudaStream_t stream) {
  return is_bf16 ? gn_backward<__nv_bfloat16>(a, stream) : gn_backward<float>(a, stream);
}

}  // namespace nr
