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
// A group's values are strided by `channels` and its statistics need the whole
// sample, so every value is used twice, far apart: a statistics kernel and an
// output kernel, both bound by HBM.  The output kernel takes the rows in the
// opposite order, so that what was read last still comes from L2.  One block
// fills an SM; each thread copies its vectors many rows ahead into a ring of
// its own in shared memory (cp.async), which keeps 64 to 98 KB an SM in flight
// without registers or barriers.  Samples so small that a cluster of up to eight
// blocks holds all rows of a few groups take one launch and are read once.
//
// Any channels / groups works: a thread keeps one 128-bit column of N channels
// and walks down the rows, sums stay per channel until the block's end, and a
// vector may span several groups.  Every sum has a fixed order (no atomics):
// the same inputs give the same bits.
//
// [1, 1048576, 128] bf16 with SiLU takes 135 us: the statistics 45 us (268 MB at
// 6.0 TB/s), the output pass the rest (486 MB, some 50 MB of x coming from L2; 132 us
// in all without the activation, so the traffic bounds it).  The gradient at
// [2, 262144, 256] takes 205 us, 1285 MB at 6.3 TB/s.  Slower: one cooperative
// kernel with a barrier between the passes and 170 KB an SM of rows kept on chip
// (178 us), loads into registers and a joining kernel between the passes (144
// us), two blocks an SM (150 us: 64 registers are too few).
#include <atomic>

#include "nr_internal.h"
#include "nr_pairs.cuh"

namespace nr {
namespace {

constexpr int kGnSms = 152;

// A direction's block: threads, rows of a lane in a step, steps in the ring.
template <typename T, bool BACK>
struct GnBlock {
  static constexpr int N = Vec<T>::N;
  static constexpr int kThreads = 512;
  static constexpr int kTensors = BACK ? 2 : 1;  // read side by side
  static constexpr int kRows = BACK ? 2 : 4;
  static constexpr int kRing = BACK ? 2 : 3;
  static constexpr int kStepBytes = kThreads * kRows * kTensors * static_cast<int>(sizeof(uint4));
  static constexpr int kScratch = kThreads * N * static_cast<int>(sizeof(float2));
  static constexpr int kMostSmem = kRing * kStepBytes > kScratch ? kRing * kStepBytes : kScratch;
};

// What a block of the one-launch kernels holds at most: rows of a thread, groups.
template <typename T, bool BACK>
struct GnSmall {
  using B = GnBlock<T, BACK>;
  static constexpr int kRows = BACK ? 12 : 20;
  static constexpr int kGroups = 64;
  // Costs besides a block's rows: of a block, of two launches, of summing samples.
  static constexpr int kBlockCost = BACK ? 12 : 13;
  static constexpr int kTwoCost = BACK ? 24 : 20;
  static constexpr int kSumCost = 5;
  static constexpr int kSlot = B::kThreads * static_cast<int>(sizeof(uint4));
  static constexpr int smem(int rows) { return B::kScratch + rows * B::kTensors * kSlot; }
};

// How a call is laid out.  Block (sample, chunk, tile) has the tile's columns of
// every chunks-th step of step_rows rows of its sample, so that at any time the
// blocks read one window of the tensor.
struct GnGeom {
  int64_t samples, space;
  int64_t steps;  // steps of a sample (the last one may be short)
  int channels, groups, cpg;
  int cols;       // 128-bit vectors of a row
  int tile_cols;  // vector columns of a block
  int tiles;
  int lanes;      // rows that a block reads side by side
  int step_rows;  // lanes * rows of a lane in a step
  int unroll;     // rows of a lane in a step
  int chunks;
  // Closed forms of what a chunk has: steps / chunks steps and one more below
  // steps % chunks; the chunk with the last step misses `missing` rows of it.
  int chunk_steps, more_steps, last_chunk, missing;

  __device__ __forceinline__ int steps_of(int chunk) const {
    return chunk_steps + (chunk < more_steps ? 1 : 0);
  }
  __device__ __forceinline__ int64_t rows_of(int chunk) const {
    return static_cast<int64_t>(steps_of(chunk)) * step_rows - (chunk == last_chunk ? missing : 0);
  }
};

// What a block costs besides its rows (launch, joining its lanes, parameters),
// as rows of a thread: about 2 us.
constexpr int64_t kGnBlockCost = 16;

template <typename T, bool BACK>
GnGeom gn_geometry(int64_t samples, int64_t space, int64_t channels, int64_t groups) {
  using B = GnBlock<T, BACK>;
  GnGeom g;
  g.samples = samples;
  g.space = space;
  g.channels = static_cast<int>(channels);
  g.groups = static_cast<int>(groups);
  g.cpg = static_cast<int>(channels / groups);
  g.cols = static_cast<int>(channels / B::N);
  g.tiles = (g.cols + B::kThreads - 1) / B::kThreads;
  g.tile_cols = (g.cols + g.tiles - 1) / g.tiles;
  g.lanes = B::kThreads / g.tile_cols;
  // Chunks a sample: as many as one to four waves of blocks hold, whichever
  // takes the least time.
  const int64_t sets = (space + g.lanes - 1) / g.lanes;  // of `lanes` rows
  const int64_t columns = samples * g.tiles;
  int64_t best = 1, best_cost = INT64_MAX;
  for (int64_t w = 1; w <= 4; w++) {
    int64_t c = kGnSms * w / columns;
    c = c < 1 ? 1 : c > sets ? sets : c;
    const int64_t waves = (columns * c + kGnSms - 1) / kGnSms;
    const int64_t cost = waves * ((sets + c - 1) / c + kGnBlockCost);
    if (cost < best_cost) best = c, best_cost = cost;
  }
  // even steps: as many rows of a lane as share a chunk's rows out best
  const int64_t per = (sets + best - 1) / best;
  const int64_t turns = (per + B::kRows - 1) / B::kRows;
  g.unroll = static_cast<int>((per + turns - 1) / turns);
  g.step_rows = g.lanes * g.unroll;
  g.steps = (space + g.step_rows - 1) / g.step_rows;
  g.chunks = static_cast<int>(best < g.steps ? best : g.steps);
  g.chunk_steps = static_cast<int>(g.steps / g.chunks);
  g.more_steps = static_cast<int>(g.steps % g.chunks);
  g.last_chunk = static_cast<int>((g.steps - 1) % g.chunks);
  g.missing = static_cast<int>(g.steps * g.step_rows - space);
  return g;
}

// The layout of the one-launch kernels: tiles of whole groups, and chunks of one
// step, the blocks of a cluster.  False where eight blocks do not hold a tile's rows
// of a sample, or where two launches are faster.  Costs are in rows of a thread
// (0.4 us forward, 0.55 us backward), fitted to: forward [2, 256, 1280] 6.2 / 11 us
// (one / two launches), [8, 159, 464] f32 6.7 / 8.6 us (clusters of 4 / single
// blocks), [3, 7161, 320] f32 24.4 / 15.8 us, [1, 26229, 48] 16.5 / 8.4 us; backward
// [4, 1024, 640] 12.8 / 16.0 us.
constexpr int kGnCluster = 8;

template <typename T, bool BACK>
bool gn_small_geometry(int64_t samples, int64_t space, int64_t channels, int64_t groups,
                       GnGeom* out) {
  using B = GnBlock<T, BACK>;
  using S = GnSmall<T, BACK>;
  // the fewest groups that make whole vectors, and sectors of 32 bytes if they can
  const int64_t cpg = channels / groups;
  int64_t tile_groups = 1;
  while (tile_groups * cpg % B::N != 0) tile_groups *= 2;
  const int64_t sector = 32 / static_cast<int64_t>(sizeof(T));
  while (tile_groups * cpg < sector && groups % (2 * tile_groups) == 0) tile_groups *= 2;
  const int64_t cols = tile_groups * cpg / B::N;
  if (cols > B::kThreads || tile_groups > S::kGroups) return false;
  const int64_t lanes = B::kThreads / cols, sets = (space + lanes - 1) / lanes;
  const int64_t tiles = groups / tile_groups;
  // Blocks a cluster: waves of blocks, each with a fixed cost and its rows.
  int64_t chunks = 0, best = INT64_MAX;
  for (int64_t c = 1; c <= kGnCluster; c *= 2) {
    const int64_t rows = (sets + c - 1) / c, waves = (samples * tiles * c + kGnSms - 1) / kGnSms;
    const int64_t cost = waves * (S::kBlockCost + rows) + (c > 1 ? 2 : 0);
    if (rows <= S::kRows && cost < best) chunks = c, best = cost;
  }
  const int64_t all = samples * space * (channels / B::N);
  const int64_t two = S::kTwoCost + all / (kGnSms * B::kThreads);
  if (BACK && samples > 1) best += S::kSumCost;  // its third kernel
  if (chunks == 0 || best > two || samples * tiles * chunks > INT32_MAX) return false;
  const int64_t rows = (sets + chunks - 1) / chunks;
  GnGeom& g = *out;
  g.samples = samples;
  g.space = space;
  g.channels = static_cast<int>(channels);
  g.groups = static_cast<int>(groups);
  g.cpg = static_cast<int>(cpg);
  g.cols = static_cast<int>(channels / B::N);
  g.tile_cols = static_cast<int>(cols);
  g.tiles = static_cast<int>(tiles);
  g.lanes = static_cast<int>(lanes);
  g.unroll = static_cast<int>(rows);
  g.step_rows = g.lanes * g.unroll;
  g.chunks = static_cast<int>(chunks);
  g.steps = (space + g.step_rows - 1) / g.step_rows;
  g.chunk_steps = static_cast<int>(g.steps / chunks);  // 0 where some blocks have no rows
  g.more_steps = static_cast<int>(g.steps % chunks);
  g.last_chunk = static_cast<int>(g.steps - 1);
  g.missing = static_cast<int>(g.steps * g.step_rows - space);
  return true;
}

// Global scratch: partial results of the blocks.  A group that lies in two tiles
// has a part in each; part (group, tile) is in row group + tile, which no other
// part has, as the groups of a tile are never below those of the tile before.
// The chunks of a part are side by side, so that joining them (every block of
// the output kernel does) reads whole sectors.
struct GnScratch {
  float2* parts;  // [samples][groups + tiles][chunks]
  float2* sums;   // backward: [samples][chunks][channels]
};

template <typename T, bool BACK>
int64_t gn_scratch_bytes(const GnGeom& g) {
  const int64_t row = g.groups + g.tiles + (BACK ? g.channels : 0);
  return g.samples * g.chunks * row * static_cast<int64_t>(sizeof(float2));
}

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

// sigmoid(z).  For bf16 tensors the hardware exponential and reciprocal, two
// instructions of the special unit a value: within (1.3 |z| + 7) 2^-24 of itself
// for z < 0 (a rounding of z log2(e), 2^-22 of the exponential, 2^-23 of the
// reciprocal) and less above; below 2^-126 it is zero.  y and dx are rounded to
// bf16 after it.  dw and db of f32 parameters are not: there the choice rests on x
// and dy, whose own bf16 roundings (2^-9) moved every term of those sums by far
// more.  For f32 tensors from t = e^-|z|, which never overflows.
template <typename T>
__device__ __forceinline__ F2 gn_sigmoid2(F2 z);
template <>
__device__ __forceinline__ F2 gn_sigmoid2<float>(F2 z) {
  float x[2];
  split(z, x[0], x[1]);
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const float t = expf(-fabsf(x[i]));
    x[i] = x[i] >= 0.0f ? 1.0f / (1.0f + t) : t / (1.0f + t);
  }
  return f2(x[0], x[1]);
}
template <>
__device__ __forceinline__ F2 gn_sigmoid2<__nv_bfloat16>(F2 z) {
  float lo, hi;
  split(mul2(z, f2(-1.4426950408889634f, -1.4426950408889634f)), lo, hi);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(lo));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(hi));
  split(add2(f2(lo, hi), f2(1.0f, 1.0f)), lo, hi);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(lo));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(hi));
  return f2(lo, hi);
}

// Where a block and a thread stand.
struct GnPlace {
  int64_t sample;
  int chunk, tile;
  int lane, col, channel;  // of this thread
  int c0, c1;              // the tile's channels
  int g0, g1;              // the groups that they belong to
  bool active;
  // Blocks of a chunk (its tiles) follow one another, or (CLUSTER) those of a tile.
  template <typename B, bool CLUSTER = false>
  __device__ __forceinline__ static GnPlace of(const GnGeom& g, unsigned block) {
    GnPlace p;
    const unsigned inner = CLUSTER ? g.chunks : g.tiles, outer = CLUSTER ? g.tiles : g.chunks;
    const unsigned rest = block / inner;
    const int i = static_cast<int>(block % inner), o = static_cast<int>(rest % outer);
    p.tile = CLUSTER ? o : i;
    p.chunk = CLUSTER ? i : o;
    p.sample = rest / outer;
    p.lane = static_cast<int>(threadIdx.x) / g.tile_cols;
    p.col = p.tile * g.tile_cols + static_cast<int>(threadIdx.x) % g.tile_cols;
    p.active = p.col < g.cols && p.lane < g.lanes;
    p.channel = p.col * B::N;
    p.c0 = p.tile * g.tile_cols * B::N;
    p.c1 = min(p.c0 + g.tile_cols * B::N, g.channels);
    p.g0 = p.c0 / g.cpg;
    p.g1 = (p.c1 - 1) / g.cpg;
    return p;
  }
};

// Rows of the lanes of a block: `base` each, and one more below `more`.
struct GnLaneRows {
  int base, more;
  __device__ __forceinline__ GnLaneRows(const GnGeom& g, int chunk) {
    base = g.steps_of(chunk) * g.unroll;
    more = 0;
    if (chunk == g.last_chunk && g.missing > 0) {
      const int rest = g.step_rows - g.missing;  // rows of the short step
      base += rest / g.lanes - g.unroll;
      more = rest % g.lanes;
    }
  }
  // Rows of lanes [l0, l1).
  __device__ __forceinline__ int of(int l0, int l1) const {
    return (l1 - l0) * base + max(0, min(more, l1) - l0);
  }
};

// (The kernels' dynamic shared memory is aligned to 128 bytes: behind 192 bytes of
// static arrays every 512-byte access of a warp would straddle a fifth line, 2 us
// of the 134 at [1, 1048576, 128].)

// Walks this thread's rows of a chunk, from the first step to the last or
// (REVERSE) back, copying kRing steps ahead: visit(offset, n, v) gets the n rows
// of a step, one vector of each tensor, `offset` in vectors from the tensors'
// start to the first of them.
template <typename B, bool REVERSE, typename Visit>
__device__ __forceinline__ void gn_walk(const GnGeom& g, const GnPlace& at,
                                        const void* const (&src)[B::kTensors], unsigned char* smem,
                                        Visit visit) {
  constexpr int R = B::kRows, K = B::kTensors, RING = B::kRing;
  const int64_t row_step = static_cast<int64_t>(g.lanes) * g.cols;
  const int64_t base = (at.sample * g.space + at.lane) * g.cols + at.col;
  const int steps = g.steps_of(at.chunk);
  const int whole = steps - (at.chunk == g.last_chunk && g.missing > 0 ? 1 : 0);
  const int short_rows = GnLaneRows(g, at.chunk).of(at.lane, at.lane + 1) - whole * g.unroll;
  const unsigned ring = smem_addr(smem) + threadIdx.x * sizeof(uint4);
  // Vectors from the tensors' start to step i of this walk, and its rows here.
  const int64_t step_vecs = static_cast<int64_t>(g.step_rows) * g.cols;
  auto offset = [&](int i) {
    const int64_t j = REVERSE ? steps - 1 - i : i;
    return base + (at.chunk + j * g.chunks) * step_vecs;
  };
  auto rows_in = [&](int i) {
    return (REVERSE ? steps - 1 - i : i) < whole ? g.unroll : short_rows;
  };
  auto issue = [&](int i, int place) {
    if (i < steps) {
      const int64_t off = offset(i);
      const int n = rows_in(i);
#pragma unroll
      for (int k = 0; k < K; k++) {
        const uint4* p = static_cast<const uint4*>(src[k]) + off;
        unsigned dst = ring + (place * R * K + k) * B::kThreads * 16;
#pragma unroll
        for (int u = 0; u < R; u++, p += row_step, dst += K * B::kThreads * 16)
          if (u < n) cp_async16(dst, p);
      }
    }
    cp_async_commit();  // possibly empty: one group a step
  };
  for (int i = 0; i < RING; i++) issue(i, i);
  int place = 0;
  for (int i = 0; i < steps; i++) {
    cp_async_wait<RING - 1>();
    const int n = rows_in(i);
    uint4 v[R][K];
    const unsigned char* slot = smem + threadIdx.x * sizeof(uint4) +
                                static_cast<size_t>(place) * R * K * B::kThreads * 16;
#pragma unroll
    for (int u = 0; u < R; u++)
      if (u < n)
#pragma unroll
        for (int k = 0; k < K; k++) v[u][k] = lds128(slot + (u * K + k) * B::kThreads * 16);
    visit(offset(i), n, v);
    issue(i + RING, place);  // the slot's values have been used
    place = place + 1 == RING ? 0 : place + 1;
  }
  cp_async_wait<0>();
}

// The group of each of N consecutive channels, by one division.
template <int N>
__device__ __forceinline__ void gn_groups_of(int channel, int cpg, int (&grp)[N]) {
  int at = channel / cpg, place = channel - at * cpg;
#pragma unroll
  for (int e = 0; e < N; e++) {
    grp[e] = at;
    if (++place == cpg) place = 0, at++;
  }
}

struct GnParams {
  const void* w;
  const void* b;
  int is_bf16;
};

struct GnArgs {
  void* out;
  const void* x;
  const void* dy;
  float* mean;
  float* rstd;
  GnParams prm;
  void* dw;
  void* db;
  float eps;
  GnScratch scratch;
};

// The blocks of a cluster: everyone arrives (its shared-memory writes are then
// visible to the others) and waits; and one float2 of another block's memory.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float2 cluster_read(const float2* p, int rank) {
  unsigned at;
  float2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at)
               : "memory");
  return v;
}

// How the lanes of a channel are joined: `subs` threads a channel, `per` lanes each.
struct GnSubs {
  int per, subs;
  __device__ __forceinline__ GnSubs(const GnGeom& g, int width, int threads) {
    const int most = width < threads ? threads / width : 1;
    per = (g.lanes + most - 1) / most;
    subs = (g.lanes + per - 1) / per;
  }
};

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
// Statistics are means and sums of squared deviations (M2).  A thread sums each
// channel's values minus the first of them that it sees, so a channel far from
// zero cancels nothing and one outlier spoils no other thread's sums; parts are
// joined by their means and counts (the update of Chan, Golub and LeVeque).

// Sums of one thread's rows.
template <typename T>
struct GnSums {
  static constexpr int P = Vec<T>::N / 2;
  F2 minus[P], s1[P], s2[P];  // minus the first value of each channel; sums of d and d^2
  bool begun;
  __device__ __forceinline__ GnSums() : begun(false) {
#pragma unroll
    for (int i = 0; i < P; i++) minus[i] = s1[i] = s2[i] = f2(0.0f, 0.0f);
  }
  __device__ __forceinline__ void begin(const uint4& v) {
    Pairs<T>::unpack(v, minus);
#pragma unroll
    for (int i = 0; i < P; i++) minus[i] = mul2(minus[i], f2(-1.0f, -1.0f));
    begun = true;
  }
  __device__ __forceinline__ void add(const uint4& v) {
    F2 f[P];
    Pairs<T>::unpack(v, f);
#pragma unroll
    for (int i = 0; i < P; i++) {
      const F2 d = add2(f[i], minus[i]);
      s1[i] = add2(s1[i], d);
      s2[i] = fma2(d, d, s2[i]);
    }
  }
};

// Warps that share one group of `elements` values in a join: one, but where few
// and wide groups would leave most warps idle.  [1, 436, 1824] f32 in one group:
// 10.1 us, 13.5 us with one warp; groups of 58 to 139 values lose 0.7 us by it.
__device__ __forceinline__ int gn_group_warps(int groups, int elements, int warps) {
  return groups < warps && elements >= 512 ? warps / groups : 1;
}

// Joins a block's threads: use(group, mean, M2) is called by one lane for each of
// the tile's groups, over its channels in the tile.  `rows` are the lanes' rows,
// `total_rows` their sum; sm holds threads * N values.
template <typename T, typename Use>
__device__ __forceinline__ void gn_join_lanes(const GnGeom& g, const GnPlace& at,
                                              const GnSums<T>& sums, const GnLaneRows& rows,
                                              float total_rows, float2* sm, Use use) {
  using B = GnBlock<T, false>;
  const int width = g.tile_cols * B::N;
  if (at.active) {
    const float count = static_cast<float>(rows.of(at.lane, at.lane + 1));
    const float inv = count > 0.0f ? 1.0f / count : 0.0f;
    float2* o = sm + at.lane * width + (at.channel - at.c0);
#pragma unroll
    for (int i = 0; i < GnSums<T>::P; i++) {
      float m0, m1, a0, a1, b0, b1;
      split(sums.minus[i], m0, m1);
      split(sums.s1[i], a0, a1);
      split(sums.s2[i], b0, b1);
      o[2 * i] = make_float2(fmaf(a0, inv, -m0), fmaf(-a0 * inv, a0, b0));
      o[2 * i + 1] = make_float2(fmaf(a1, inv, -m1), fmaf(-a1 * inv, a1, b1));
    }
  }
  __syncthreads();
  // Lanes of a channel: sub s joins lanes s * per ... and leaves the result in
  // the first of them.
  const GnSubs sub(g, width, B::kThreads);
  const int tile_channels = at.c1 - at.c0;
  for (int i = threadIdx.x; i < sub.subs * tile_channels; i += B::kThreads) {
    const int s = i / tile_channels, c = i - s * tile_channels;
    const int l0 = s * sub.per, l1 = min(l0 + sub.per, g.lanes);
    float2* col = sm + c;
    float sum = 0.0f;
    for (int l = l0; l < l1; l++)
      sum = fmaf(static_cast<float>(rows.of(l, l + 1)), col[l * width].x, sum);
    const int count = rows.of(l0, l1);
    const float mean = count > 0 ? __fdiv_rn(sum, static_cast<float>(count)) : 0.0f;
    float m2 = 0.0f;
    for (int l = l0; l < l1; l++) {
      const float2 v = col[l * width];
      const float d = v.x - mean, k = static_cast<float>(rows.of(l, l + 1));
      if (k > 0.0f) m2 += fmaf(k * d, d, v.y);
    }
    col[l0 * width] = make_float2(mean, m2);
  }
  __syncthreads();
  // A group's channels in this tile: one warp a group, or several that take a
  // share each of the (sub, channel) elements.
  const int warp = threadIdx.x / kWarp, lane32 = threadIdx.x % kWarp;
  constexpr int kWarps = B::kThreads / kWarp;
  // Elements [from, end) of a group: sub i / cn, channel i % cn; a lane's are 32 apart.
  auto each = [&](int ca, int cn, int from, int end, auto take) {
    int i = from + lane32, s = i / cn, c = i - s * cn;
    const int ds = kWarp / cn, dc = kWarp % cn;
    for (; i < end; i += kWarp) {
      const int l0 = s * sub.per;
      const float k = static_cast<float>(rows.of(l0, min(l0 + sub.per, g.lanes)));
      take(k, sm[l0 * width + ca - at.c0 + c]);
      s += ds;
      c += dc;
      if (c >= cn) c -= cn, s++;
    }
  };
  const int groups = at.g1 - at.g0 + 1;
  const int split_by = gn_group_warps(groups, sub.subs * min(g.cpg, tile_channels), kWarps);
  if (split_by == 1) {
    for (int grp = at.g0 + warp; grp <= at.g1; grp += kWarps) {
      const int ca = max(at.c0, grp * g.cpg), cn = min(at.c1, (grp + 1) * g.cpg) - ca;
      const int n = sub.subs * cn;
      float sum = 0.0f, m2 = 0.0f;
      each(ca, cn, 0, n, [&](float k, const float2& v) { sum = fmaf(k, v.x, sum); });
      const float mean = __fdiv_rn(group_sum<kWarp>(sum), total_rows * static_cast<float>(cn));
      each(ca, cn, 0, n, [&](float k, const float2& v) {
        const float d = v.x - mean;
        if (k > 0.0f) m2 += fmaf(k * d, d, v.y);
      });
      m2 = group_sum<kWarp>(m2);
      if (lane32 == 0) use(grp, mean, m2);
    }
    return;
  }
  __shared__ float3 shares[kWarps];  // rows, mean, M2
  if (warp < groups * split_by) {
    const int grp = at.g0 + warp / split_by, part = warp % split_by;
    const int ca = max(at.c0, grp * g.cpg), cn = min(at.c1, (grp + 1) * g.cpg) - ca;
    const int share = (sub.subs * cn + split_by - 1) / split_by;
    const int from = part * share, end = min(sub.subs * cn, from + share);
    float sum = 0.0f, count = 0.0f, m2 = 0.0f;
    each(ca, cn, from, end, [&](float k, const float2& v) {
      sum = fmaf(k, v.x, sum);
      count += k;
    });
    sum = group_sum<kWarp>(sum);
    count = group_sum<kWarp>(count);
    const float mean = count > 0.0f ? __fdiv_rn(sum, count) : 0.0f;
    each(ca, cn, from, end, [&](float k, const float2& v) {
      const float d = v.x - mean;
      if (k > 0.0f) m2 += fmaf(k * d, d, v.y);
    });
    m2 = group_sum<kWarp>(m2);
    if (lane32 == 0) shares[warp] = make_float3(count, mean, m2);
  }
  __syncthreads();
  if (warp < groups) {
    const float3 v = lane32 < split_by ? shares[warp * split_by + lane32]
                                       : make_float3(0.0f, 0.0f, 0.0f);
    const float count = group_sum<kWarp>(v.x);
    const float mean = __fdiv_rn(group_sum<kWarp>(v.x * v.y), count);
    const float d = v.y - mean;
    const float m2 = group_sum<kWarp>(v.x > 0.0f ? fmaf(v.x * d, d, v.z) : 0.0f);
    if (lane32 == 0) use(at.g0 + warp, mean, m2);
  }
}

template <typename T>
__global__ void __launch_bounds__(GnBlock<T, false>::kThreads, 1)
    gn_stats_kernel(const GnArgs a, const GnGeom g) {
  using B = GnBlock<T, false>;
  constexpr int R = B::kRows;
  extern __shared__ __align__(128) unsigned char smem[];
  const GnPlace at = GnPlace::of<B>(g, blockIdx.x);
  pdl_enter();  // before any global read: the previous kernel may still run
  GnSums<T> sums;
  if (at.active) {
    const void* const src[1] = {a.x};
    gn_walk<B, false>(g, at, src, smem, [&](int64_t, int n, const uint4 (&v)[R][1]) {
      if (!sums.begun && n > 0) sums.begin(v[0][0]);
#pragma unroll
      for (int u = 0; u < R; u++)
        if (u < n) sums.add(v[u][0]);
    });
  }
  __syncthreads();  // the rings are done with
  gn_join_lanes<T>(g, at, sums, GnLaneRows(g, at.chunk), static_cast<float>(g.rows_of(at.chunk)),
                   reinterpret_cast<float2*>(smem), [&](int grp, float mean, float m2) {
    a.scratch.parts[(at.sample * (g.groups + g.tiles) + grp + at.tile) * g.chunks + at.chunk] =
        make_float2(mean, m2);
  });
}

__device__ __forceinline__ float gn_rstd(float m2, float total, float eps) {
  m2 = m2 < 0.0f ? 0.0f : m2;  // rounding may leave a constant group just below zero
  return 1.0f / sqrtf(__fdiv_rn(m2, total) + eps);
}

// Joins the parts of one group of the sample into mean and rstd (a warp's work).
__device__ __forceinline__ float2 gn_join(const GnArgs& a, const GnGeom& g, int64_t sample, int grp,
                                          int width) {
  const int lane32 = threadIdx.x % kWarp;
  const int ca = grp * g.cpg, cb = ca + g.cpg;
  const int t0 = ca / width, tn = (cb - 1) / width - t0 + 1;
  const int n = g.chunks * tn;
  // the rows of a group's tiles follow one another
  const float2* parts = a.scratch.parts +
                        (sample * (g.groups + g.tiles) + grp + t0) * static_cast<int64_t>(g.chunks);
  auto part = [&](int i, float& count) {
    const int t = tn == 1 ? 0 : i / g.chunks, chunk = i - t * g.chunks, tile = t0 + t;
    count = static_cast<float>(g.rows_of(chunk)) *
            static_cast<float>(min(cb, (tile + 1) * width) - max(ca, tile * width));
    return parts[i];
  };
  // a lane's first parts stay in registers for the second sum
  constexpr int kHeld = 5;
  float2 held[kHeld];
  float counts[kHeld], sum = 0.0f, count;
#pragma unroll
  for (int j = 0; j < kHeld; j++) {
    counts[j] = 0.0f;
    held[j] = make_float2(0.0f, 0.0f);
    if (lane32 + j * kWarp < n) held[j] = part(lane32 + j * kWarp, counts[j]);
  }
#pragma unroll
  for (int j = 0; j < kHeld; j++) sum = fmaf(counts[j], held[j].x, sum);
  for (int i = lane32 + kHeld * kWarp; i < n; i += kWarp) {
    const float2 v = part(i, count);
    sum = fmaf(count, v.x, sum);
  }
  const float total = static_cast<float>(g.space) * static_cast<float>(g.cpg);
  const float mean = __fdiv_rn(group_sum<kWarp>(sum), total);
  float m2 = 0.0f;
#pragma unroll
  for (int j = 0; j < kHeld; j++) {
    const float d = held[j].x - mean;
    if (counts[j] > 0.0f) m2 += fmaf(counts[j] * d, d, held[j].y);
  }
  for (int i = lane32 + kHeld * kWarp; i < n; i += kWarp) {
    const float2 v = part(i, count);
    const float d = v.x - mean;
    m2 += fmaf(count * d, d, v.y);
  }
  return make_float2(mean, gn_rstd(group_sum<kWarp>(m2), total, a.eps));
}

// This thread's channels of the output: y = act((x - mean) * sc + sh).  Made from
// w and b, whose reads then overlap what comes before the statistics.
template <typename T, bool SILU>
struct GnOut {
  static constexpr int N = Vec<T>::N, P = N / 2;
  F2 mu[P], sc[P], sh[P];  // minus the mean, rstd * w, b
  __device__ __forceinline__ GnOut(const GnArgs& a, int channel) {
    float fa[N], fb[N];
    gn_params<N>(a.prm.w, a.prm.is_bf16, channel, 1.0f, fa);
    gn_params<N>(a.prm.b, a.prm.is_bf16, channel, 0.0f, fb);
    to_pairs<P>(fa, sc);
    to_pairs<P>(fb, sh);
  }
  // `stats`: mean and rstd of the tile's groups.
  __device__ __forceinline__ void take(const GnGeom& g, const GnPlace& at, int channel,
                                       const float2* stats) {
    int grp[N];
    gn_groups_of<N>(channel, g.cpg, grp);
#pragma unroll
    for (int i = 0; i < P; i++) {
      const float2 u = stats[grp[2 * i] - at.g0], v = stats[grp[2 * i + 1] - at.g0];
      mu[i] = f2(-u.x, -v.x);
      sc[i] = mul2(sc[i], f2(u.y, v.y));
    }
  }
  __device__ __forceinline__ uint4 operator()(const uint4& v) const {
    F2 f[P];
    Pairs<T>::unpack(v, f);
#pragma unroll
    for (int i = 0; i < P; i++) {
      f[i] = fma2(add2(f[i], mu[i]), sc[i], sh[i]);
      if (SILU) f[i] = mul2(f[i], gn_sigmoid2<T>(f[i]));
    }
    return Pairs<T>::pack(f);
  }
};

template <typename T, bool SILU>
__global__ void __launch_bounds__(GnBlock<T, false>::kThreads, 1)
    gn_apply_kernel(const GnArgs a, const GnGeom g) {
  using B = GnBlock<T, false>;
  constexpr int R = B::kRows;
  extern __shared__ __align__(128) unsigned char smem[];
  float2* sm = reinterpret_cast<float2*>(smem);  // before the walk: mean, rstd of the groups
  const GnPlace at = GnPlace::of<B>(g, gridDim.x - 1 - blockIdx.x);
  pdl_enter();  // before any global read: the previous kernel may still run
  const int warp = threadIdx.x / kWarp, lane32 = threadIdx.x % kWarp;
  // (an inactive thread's column may lie past the tile: it takes the first one)
  const int channel = at.active ? at.channel : at.c0;
  GnOut<T, SILU> value(a, channel);
  for (int grp = at.g0 + warp; grp <= at.g1; grp += B::kThreads / kWarp) {
    const float2 v = gn_join(a, g, at.sample, grp, g.tile_cols * B::N);
    if (lane32 == 0) {
      sm[grp - at.g0] = v;
      if (at.chunk == 0 && grp * g.cpg >= at.c0) {  // one block of the sample writes a group's
        a.mean[at.sample * g.groups + grp] = v.x;
        a.rstd[at.sample * g.groups + grp] = v.y;
      }
    }
  }
  __syncthreads();
  value.take(g, at, channel, sm);
  __syncthreads();  // the rings take the place of sm
  if (!at.active) return;
  const int64_t row_step = static_cast<int64_t>(g.lanes) * g.cols;
  const void* const src[1] = {a.x};
  gn_walk<B, true>(g, at, src, smem, [&](int64_t off, int n, const uint4 (&v)[R][1]) {
    uint4* o = static_cast<uint4*>(a.out) + off;
#pragma unroll
    for (int u = 0; u < R; u++, o += row_step)
      if (u < n) st_stream(o, value(v[u][0]));
  });
}

// Both passes in one launch, for samples so small that a cluster of blocks holds
// all rows of a few groups in shared memory: x is read once.  Block (sample, tile,
// chunk), a tile being whole groups; the blocks of a cluster join their means and M2
// through distributed shared memory, in the order of their ranks.
template <typename T, bool SILU>
__global__ void __launch_bounds__(GnBlock<T, false>::kThreads, 1)
    gn_small_kernel(const GnArgs a, const GnGeom g) {
  using B = GnBlock<T, false>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float2 parts[GnSmall<T, false>::kGroups], stats[GnSmall<T, false>::kGroups];
  unsigned char* held = smem + B::kScratch + threadIdx.x * sizeof(uint4);
  constexpr int kSlot = GnSmall<T, false>::kSlot;
  const GnPlace at = GnPlace::of<B, true>(g, blockIdx.x);
  pdl_enter();  // before any global read: the previous kernel may still run
  const GnLaneRows rows(g, at.chunk);
  const int64_t row0 = static_cast<int64_t>(at.chunk) * g.step_rows;
  const int64_t base = (at.sample * g.space + row0 + at.lane) * g.cols + at.col;
  const int64_t row_step = static_cast<int64_t>(g.lanes) * g.cols;
  const int n = at.active ? rows.of(at.lane, at.lane + 1) : 0;
  const uint4* p = static_cast<const uint4*>(a.x) + base;
  for (int i = 0; i < n; i++) cp_async16(smem_addr(held + i * kSlot), p + i * row_step);
  cp_async_commit();
  const int channel = at.active ? at.channel : at.c0;
  GnOut<T, SILU> value(a, channel);
  cp_async_wait<0>();  // a thread reads back only what it copied
  GnSums<T> sums;
  if (n > 0) sums.begin(lds128(held));
  for (int i = 0; i < n; i++) sums.add(lds128(held + i * kSlot));
  const float total = static_cast<float>(g.space) * static_cast<float>(g.cpg);
  auto finish = [&](int grp, float mean, float m2) {
    const float rstd = gn_rstd(m2, total, a.eps);
    stats[grp - at.g0] = make_float2(mean, rstd);
    if (at.chunk == 0) {
      a.mean[at.sample * g.groups + grp] = mean;
      a.rstd[at.sample * g.groups + grp] = rstd;
    }
  };
  const float part_rows = static_cast<float>(g.rows_of(at.chunk));
  gn_join_lanes<T>(g, at, sums, rows, part_rows, reinterpret_cast<float2*>(smem),
                   [&](int grp, float mean, float m2) {
    if (g.chunks == 1)
      finish(grp, mean, m2);
    else
      parts[grp - at.g0] = make_float2(mean, m2);
  });
  if (g.chunks > 1) {
    cluster_arrive();
    cluster_wait();
    const int warp = threadIdx.x / kWarp, lane32 = threadIdx.x % kWarp;
    for (int grp = at.g0 + warp; grp <= at.g1; grp += B::kThreads / kWarp) {
      float2 v = make_float2(0.0f, 0.0f);
      float count = 0.0f;
      if (lane32 < g.chunks && g.steps_of(lane32) > 0) {  // a block without rows has no part
        v = cluster_read(parts + grp - at.g0, lane32);
        count = static_cast<float>(g.rows_of(lane32)) * static_cast<float>(g.cpg);
      }
      const float mean = __fdiv_rn(group_sum<kWarp>(count * v.x), total);
      const float d = v.x - mean;
      const float m2 = group_sum<kWarp>(count > 0.0f ? fmaf(count * d, d, v.y) : 0.0f);
      if (lane32 == 0) finish(grp, mean, m2);
    }
    cluster_arrive();  // this block has read the others' parts
  }
  __syncthreads();
  if (at.active) {
    value.take(g, at, channel, stats);
    uint4* o = static_cast<uint4*>(a.out) + base;
    for (int i = 0; i < n; i++) st_stream(o + i * row_step, value(lds128(held + i * kSlot)));
  }
  if (g.chunks > 1) cluster_wait();  // nobody reads this block's memory any more
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
// dz = dy * act'(z); silu'(z) = s (1 + z (1 - s)) with s = sigmoid(z).
template <typename T, bool SILU>
__device__ __forceinline__ F2 gn_dz(F2 dy, F2 z) {
  if (!SILU) return dy;
  const F2 one = f2(1.0f, 1.0f);
  const F2 s = gn_sigmoid2<T>(z);
  const F2 rest = fma2(s, f2(-1.0f, -1.0f), one);
  return mul2(dy, mul2(s, fma2(z, rest, one)));
}

// This thread's channels: minus the mean, rstd * w, b.
template <int N, int P>
__device__ __forceinline__ void gn_grad_params(const GnArgs& a, const GnGeom& g, int64_t sample,
                                               int channel, F2 (&mu)[P], F2 (&sc)[P],
                                               F2 (&sh)[P]) {
  float fm[N], fa[N], fb[N];
  gn_params<N>(a.prm.w, a.prm.is_bf16, channel, 1.0f, fa);
  gn_params<N>(a.prm.b, a.prm.is_bf16, channel, 0.0f, fb);
  int grp[N];
  gn_groups_of<N>(channel, g.cpg, grp);
#pragma unroll
  for (int e = 0; e < N; e++) {
    const int64_t i = sample * g.groups + grp[e];
    fm[e] = -a.mean[i];
    fa[e] *= a.rstd[i];
  }
  to_pairs<P>(fm, mu);
  to_pairs<P>(fa, sc);
  to_pairs<P>(fb, sh);
}

// Sums of one thread's rows, of dz and of dz (x - mean).
template <typename T, bool SILU>
struct GnGradSums {
  static constexpr int N = Vec<T>::N, P = N / 2;
  F2 mu[P], sc[P], sh[P], s1[P], s2[P];
  __device__ __forceinline__ GnGradSums() {
#pragma unroll
    for (int i = 0; i < P; i++) mu[i] = sc[i] = sh[i] = s1[i] = s2[i] = f2(0.0f, 0.0f);
  }
  __device__ __forceinline__ void add(const uint4& x, const uint4& dy) {
    F2 f[P], d[P];
    Pairs<T>::unpack(x, f);
    Pairs<T>::unpack(dy, d);
#pragma unroll
    for (int i = 0; i < P; i++) {
      const F2 c = add2(f[i], mu[i]);
      const F2 dz = gn_dz<T, SILU>(d[i], fma2(c, sc[i], sh[i]));
      s1[i] = add2(s1[i], dz);
      s2[i] = fma2(dz, c, s2[i]);
    }
  }
};

// Joins a block's threads: of(channel, S1, S2) is called for each of the tile's
// channels (and sm is left with them, from the tile's first), then use(group, sum
// of w S1, sum of w S2) for each of its groups, over its channels in the tile,
// each once.
template <typename T, bool SILU, typename Of, typename Use>
__device__ __forceinline__ void gn_grad_join(const GnArgs& a, const GnGeom& g, const GnPlace& at,
                                             const GnGradSums<T, SILU>& sums, float2* sm, Of of,
                                             Use use) {
  using B = GnBlock<T, true>;
  const int width = g.tile_cols * B::N;
  if (at.active) {
    float2* o = sm + at.lane * width + (at.channel - at.c0);
#pragma unroll
    for (int i = 0; i < B::N / 2; i++) {
      float a0, a1, b0, b1;
      split(sums.s1[i], a0, a1);
      split(sums.s2[i], b0, b1);
      o[2 * i] = make_float2(a0, b0);
      o[2 * i + 1] = make_float2(a1, b1);
    }
  }
  __syncthreads();
  // The lanes of a channel, in two steps.
  const GnSubs sub(g, width, B::kThreads);
  const int tile_channels = at.c1 - at.c0;
  for (int i = threadIdx.x; i < sub.subs * tile_channels; i += B::kThreads) {
    const int s = i / tile_channels, c = i - s * tile_channels;
    const int l0 = s * sub.per, l1 = min(l0 + sub.per, g.lanes);
    float2 v = sm[l0 * width + c];
    for (int l = l0 + 1; l < l1; l++) {
      v.x += sm[l * width + c].x;
      v.y += sm[l * width + c].y;
    }
    sm[l0 * width + c] = v;
  }
  __syncthreads();
  for (int c = threadIdx.x; c < tile_channels; c += B::kThreads) {
    float2 v = sm[c];
    for (int s = 1; s < sub.subs; s++) {
      v.x += sm[s * sub.per * width + c].x;
      v.y += sm[s * sub.per * width + c].y;
    }
    v.y *= a.rstd[at.sample * g.groups + (at.c0 + c) / g.cpg];
    of(at.c0 + c, v.x, v.y);
    sm[c] = v;
  }
  __syncthreads();
  const int warp = threadIdx.x / kWarp, lane32 = threadIdx.x % kWarp;
  constexpr int kWarps = B::kThreads / kWarp;
  const int groups = at.g1 - at.g0 + 1;
  const int split_by = gn_group_warps(groups, min(g.cpg, tile_channels), kWarps);
  auto sum = [&](int from, int end) {  // of channels [from, end), by w
    float m1 = 0.0f, m2 = 0.0f;
    for (int c = from + lane32; c < end; c += kWarp) {
      float w[1];
      gn_params<1>(a.prm.w, a.prm.is_bf16, c, 1.0f, w);
      m1 = fmaf(w[0], sm[c - at.c0].x, m1);
      m2 = fmaf(w[0], sm[c - at.c0].y, m2);
    }
    return make_float2(group_sum<kWarp>(m1), group_sum<kWarp>(m2));
  };
  if (split_by == 1) {
    for (int grp = at.g0 + warp; grp <= at.g1; grp += kWarps) {
      const float2 v = sum(max(at.c0, grp * g.cpg), min(at.c1, (grp + 1) * g.cpg));
      if (lane32 == 0) use(grp, v.x, v.y);
    }
    return;
  }
  __shared__ float2 shares[kWarps];
  if (warp < groups * split_by) {
    const int grp = at.g0 + warp / split_by, part = warp % split_by;
    const int ca = max(at.c0, grp * g.cpg), cb = min(at.c1, (grp + 1) * g.cpg);
    const int share = (cb - ca + split_by - 1) / split_by;
    const float2 v = sum(ca + part * share, min(cb, ca + (part + 1) * share));
    if (lane32 == 0) shares[warp] = v;
  }
  __syncthreads();
  if (warp < groups) {
    const float2 v = lane32 < split_by ? shares[warp * split_by + lane32]
                                       : make_float2(0.0f, 0.0f);
    const float m1 = group_sum<kWarp>(v.x), m2 = group_sum<kWarp>(v.y);
    if (lane32 == 0) use(at.g0 + warp, m1, m2);
  }
}

template <typename T, bool SILU>
__global__ void __launch_bounds__(GnBlock<T, true>::kThreads, 1)
    gn_grad_stats_kernel(const GnArgs a, const GnGeom g) {
  using B = GnBlock<T, true>;
  constexpr int R = B::kRows;
  extern __shared__ __align__(128) unsigned char smem[];
  const GnPlace at = GnPlace::of<B>(g, blockIdx.x);
  pdl_enter();  // before any global read: the previous kernel may still run
  GnGradSums<T, SILU> sums;
  if (at.active) {
    gn_grad_params<B::N, B::N / 2>(a, g, at.sample, at.channel, sums.mu, sums.sc, sums.sh);
    const void* const src[2] = {a.x, a.dy};
    gn_walk<B, false>(g, at, src, smem, [&](int64_t, int n, const uint4 (&v)[R][2]) {
#pragma unroll
      for (int u = 0; u < R; u++)
        if (u < n) sums.add(v[u][0], v[u][1]);
    });
  }
  __syncthreads();  // the rings are done with
  const int64_t block = at.sample * g.chunks + at.chunk;
  gn_grad_join<T, SILU>(
      a, g, at, sums, reinterpret_cast<float2*>(smem),
      [&](int c, float s1, float s2) {
        if (a.dw != nullptr) a.scratch.sums[block * g.channels + c] = make_float2(s1, s2);
      },
      [&](int grp, float m1, float m2) {
        a.scratch.parts[(at.sample * (g.groups + g.tiles) + grp + at.tile) * g.chunks + at.chunk] =
            make_float2(m1, m2);
      });
}

// dw and db of one channel.
__device__ __forceinline__ void gn_put_grads(const GnArgs& a, int64_t c, float s1, float s2) {
  if (a.prm.is_bf16) {
    static_cast<__nv_bfloat16*>(a.db)[c] = __float2bfloat16_rn(s1);
    static_cast<__nv_bfloat16*>(a.dw)[c] = __float2bfloat16_rn(s2);
  } else {
    static_cast<float*>(a.db)[c] = s1;
    static_cast<float*>(a.dw)[c] = s2;
  }
}

// dw and db of channels first, first + step, ... from `rows` rows of channel sums: a
// warp's work.
__device__ __forceinline__ void gn_sum_grads(const GnArgs& a, const GnGeom& g, int64_t rows,
                                             int64_t first, int64_t step) {
  const int lane32 = threadIdx.x % kWarp;
  for (int64_t c = first; c < g.channels; c += step) {
    float t1 = 0.0f, t2 = 0.0f;
    for (int64_t i = lane32; i < rows; i += kWarp) {
      const float2 v = a.scratch.sums[i * g.channels + c];
      t1 += v.x;
      t2 += v.y;
    }
    t1 = group_sum<kWarp>(t1);
    t2 = group_sum<kWarp>(t2);
    if (lane32 == 0) gn_put_grads(a, c, t1, t2);
  }
}

// This thread's channels of the input's gradient:
// dx = a dz - k1 - (x - mean) k2 with a = rstd w, k1 = rstd m1, k2 = rstd^2 m2.
template <typename T, bool SILU>
struct GnGradOut {
  static constexpr int N = Vec<T>::N, P = N / 2;
  F2 mu[P], sc[P], sh[P], k1[P], k2[P];  // k1 and k2 negated
  // `means`: m1 and m2 of the tile's groups.
  __device__ __forceinline__ void take(const GnArgs& a, const GnGeom& g, const GnPlace& at,
                                       int channel, const float2* means) {
    int grp[N];
    gn_groups_of<N>(channel, g.cpg, grp);
    const float* rstd = a.rstd + at.sample * g.groups;
#pragma unroll
    for (int i = 0; i < P; i++) {
      const float2 u = means[grp[2 * i] - at.g0], v = means[grp[2 * i + 1] - at.g0];
      const float ru = rstd[grp[2 * i]], rv = rstd[grp[2 * i + 1]];
      k1[i] = f2(-ru * u.x, -rv * v.x);
      k2[i] = f2(-ru * ru * u.y, -rv * rv * v.y);
    }
  }
  __device__ __forceinline__ uint4 operator()(const uint4& x, const uint4& dy) const {
    F2 f[P], d[P];
    Pairs<T>::unpack(x, f);
    Pairs<T>::unpack(dy, d);
#pragma unroll
    for (int i = 0; i < P; i++) {
      const F2 c = add2(f[i], mu[i]);
      const F2 dz = gn_dz<T, SILU>(d[i], fma2(c, sc[i], sh[i]));
      f[i] = fma2(sc[i], dz, fma2(c, k2[i], k1[i]));
    }
    return Pairs<T>::pack(f);
  }
};

template <typename T, bool SILU>
__global__ void __launch_bounds__(GnBlock<T, true>::kThreads, 1)
    gn_grad_apply_kernel(const GnArgs a, const GnGeom g) {
  using B = GnBlock<T, true>;
  constexpr int N = B::N, R = B::kRows;
  constexpr int kWarps = B::kThreads / kWarp;
  extern __shared__ __align__(128) unsigned char smem[];
  float2* sm = reinterpret_cast<float2*>(smem);  // before the walk: the groups' means
  const GnPlace at = GnPlace::of<B>(g, gridDim.x - 1 - blockIdx.x);
  pdl_enter();  // before any global read: the previous kernel may still run
  const int width = g.tile_cols * N;
  const int warp = threadIdx.x / kWarp, lane32 = threadIdx.x % kWarp;
  const float inv = 1.0f / (static_cast<float>(g.space) * static_cast<float>(g.cpg));
  // (an inactive thread's column may lie past the tile: it takes the first one)
  const int channel = at.active ? at.channel : at.c0;
  GnGradOut<T, SILU> value;
  gn_grad_params<N, N / 2>(a, g, at.sample, channel, value.mu, value.sc, value.sh);
  for (int grp = at.g0 + warp; grp <= at.g1; grp += kWarps) {
    const int t0 = grp * g.cpg / width, tn = ((grp + 1) * g.cpg - 1) / width - t0 + 1;
    float m1 = 0.0f, m2 = 0.0f;
    const float2* parts = a.scratch.parts + (at.sample * (g.groups + g.tiles) + grp + t0) *
                                                static_cast<int64_t>(g.chunks);
    for (int i = lane32; i < g.chunks * tn; i += kWarp) {
      const float2 v = parts[i];
      m1 += v.x;
      m2 += v.y;
    }
    m1 = group_sum<kWarp>(m1);
    m2 = group_sum<kWarp>(m2);
    if (lane32 == 0) sm[grp - at.g0] = make_float2(m1 * inv, m2 * inv);
  }
  // dw and db: the blocks share the channels, one warp each.
  if (a.dw != nullptr)
    gn_sum_grads(a, g, g.samples * g.chunks, blockIdx.x + static_cast<int64_t>(gridDim.x) * warp,
                 static_cast<int64_t>(gridDim.x) * kWarps);
  __syncthreads();
  value.take(a, g, at, channel, sm);
  __syncthreads();  // the rings take the place of sm
  if (!at.active) return;
  const int64_t row_step = static_cast<int64_t>(g.lanes) * g.cols;
  const void* const src[2] = {a.x, a.dy};
  gn_walk<B, true>(g, at, src, smem, [&](int64_t off, int n, const uint4 (&v)[R][2]) {
    uint4* o = static_cast<uint4*>(a.out) + off;
#pragma unroll
    for (int u = 0; u < R; u++, o += row_step)
      if (u < n) st_stream(o, value(v[u][0], v[u][1]));
  });
}

// Both passes in one launch, as gn_small_kernel.  The channel sums of one sample
// are dw and db; those of several are added by gn_grad_sum_kernel.
template <typename T, bool SILU>
__global__ void __launch_bounds__(GnBlock<T, true>::kThreads, 1)
    gn_grad_small_kernel(const GnArgs a, const GnGeom g) {
  using B = GnBlock<T, true>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float2 parts[GnSmall<T, true>::kGroups], means[GnSmall<T, true>::kGroups];
  float2* sm = reinterpret_cast<float2*>(smem);
  unsigned char* held = smem + B::kScratch + threadIdx.x * sizeof(uint4);
  constexpr int kSlot = GnSmall<T, true>::kSlot;
  const GnPlace at = GnPlace::of<B, true>(g, blockIdx.x);
  pdl_enter();  // before any global read: the previous kernel may still run
  const int64_t row0 = static_cast<int64_t>(at.chunk) * g.step_rows;
  const int64_t base = (at.sample * g.space + row0 + at.lane) * g.cols + at.col;
  const int64_t row_step = static_cast<int64_t>(g.lanes) * g.cols;
  const int n = at.active ? GnLaneRows(g, at.chunk).of(at.lane, at.lane + 1) : 0;
  const uint4* px = static_cast<const uint4*>(a.x) + base;
  const uint4* pd = static_cast<const uint4*>(a.dy) + base;
  for (int i = 0; i < n; i++) {
    cp_async16(smem_addr(held + 2 * i * kSlot), px + i * row_step);
    cp_async16(smem_addr(held + (2 * i + 1) * kSlot), pd + i * row_step);
  }
  cp_async_commit();
  GnGradSums<T, SILU> sums;
  if (n > 0)
    gn_grad_params<B::N, B::N / 2>(a, g, at.sample, at.channel, sums.mu, sums.sc, sums.sh);
  cp_async_wait<0>();  // a thread reads back only what it copied
  for (int i = 0; i < n; i++)
    sums.add(lds128(held + 2 * i * kSlot), lds128(held + (2 * i + 1) * kSlot));
  const float inv = 1.0f / (static_cast<float>(g.space) * static_cast<float>(g.cpg));
  auto channel_sums = [&](int c, float s1, float s2) {
    if (a.dw == nullptr) return;
    if (g.samples == 1)
      gn_put_grads(a, c, s1, s2);
    else
      a.scratch.sums[at.sample * g.channels + c] = make_float2(s1, s2);
  };
  gn_grad_join<T, SILU>(
      a, g, at, sums, sm,
      [&](int c, float s1, float s2) {
        if (g.chunks == 1) channel_sums(c, s1, s2);
      },
      [&](int grp, float m1, float m2) {
        (g.chunks == 1 ? means : parts)[grp - at.g0] =
            g.chunks == 1 ? make_float2(m1 * inv, m2 * inv) : make_float2(m1, m2);
      });
  if (g.chunks > 1) {
    cluster_arrive();
    cluster_wait();
    const int tile_channels = at.c1 - at.c0;
    // the blocks share the channels, and each adds up every group's parts
    for (int i = threadIdx.x; i < tile_channels + at.g1 - at.g0 + 1; i += B::kThreads) {
      const bool is_channel = i < tile_channels;
      if (is_channel && i % g.chunks != at.chunk) continue;
      float s1 = 0.0f, s2 = 0.0f;
      for (int r = 0; r < g.chunks; r++) {
        const float2 v = cluster_read(is_channel ? sm + i : parts + i - tile_channels, r);
        s1 += v.x;
        s2 += v.y;
      }
      if (is_channel)
        channel_sums(at.c0 + i, s1, s2);
      else
        means[i - tile_channels] = make_float2(s1 * inv, s2 * inv);
    }
    cluster_arrive();  // this block has read the others' parts
  }
  __syncthreads();
  if (at.active) {
    GnGradOut<T, SILU> value;
#pragma unroll
    for (int i = 0; i < B::N / 2; i++) {
      value.mu[i] = sums.mu[i];
      value.sc[i] = sums.sc[i];
      value.sh[i] = sums.sh[i];
    }
    value.take(a, g, at, at.channel, means);
    uint4* o = static_cast<uint4*>(a.out) + base;
    for (int i = 0; i < n; i++)
      st_stream(o + i * row_step,
                value(lds128(held + 2 * i * kSlot), lds128(held + (2 * i + 1) * kSlot)));
  }
  if (g.chunks > 1) cluster_wait();  // nobody reads this block's memory any more
}

constexpr int kGnSumThreads = 256;

__global__ void __launch_bounds__(kGnSumThreads)
    gn_grad_sum_kernel(const GnArgs a, const GnGeom g) {
  pdl_enter();
  constexpr int kWarps = kGnSumThreads / kWarp;
  gn_sum_grads(a, g, g.samples, static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / kWarp,
               static_cast<int64_t>(gridDim.x) * kWarps);
}

// Raises the shared-memory limit of kernels, once a device.
template <typename... Kernels>
cudaError_t gn_raise(std::atomic<int>* done, int bytes, Kernels... kernels) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  if (done[device].load(std::memory_order_acquire)) return cudaSuccess;
  for (auto kernel : {kernels...}) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
  }
  done[device].store(1, std::memory_order_release);
  return cudaSuccess;
}

template <typename T, bool BACK, bool SILU>
cudaError_t gn_launch(const GroupNormArgs& in, cudaStream_t s) {
  using B = GnBlock<T, BACK>;
  static std::atomic<int> done[64];
  void (*stats)(const GnArgs, const GnGeom);
  void (*apply)(const GnArgs, const GnGeom);
  void (*small)(const GnArgs, const GnGeom);
  if constexpr (BACK) {
    stats = gn_grad_stats_kernel<T, SILU>;
    apply = gn_grad_apply_kernel<T, SILU>;
    small = gn_grad_small_kernel<T, SILU>;
  } else {
    stats = gn_stats_kernel<T>;
    apply = gn_apply_kernel<T, SILU>;
    small = gn_small_kernel<T, SILU>;
  }
  using S = GnSmall<T, BACK>;
  constexpr int most = S::smem(S::kRows);
  static_assert(most <= 232448 - 2048, "a block's shared memory, less its static arrays");
  cudaError_t e =
      gn_raise(done, B::kMostSmem > most ? B::kMostSmem : most, stats, apply, small);
  if (e != cudaSuccess) return e;
  GnArgs a;
  a.out = in.out;
  a.x = in.x;
  a.dy = in.dy;
  a.mean = in.mean;
  a.rstd = in.rstd;
  a.prm = GnParams{in.w, in.b, in.w_is_bf16};
  a.dw = in.dw;
  a.db = in.db;
  a.eps = in.eps;
  GnGeom g;
  if (gn_small_geometry<T, BACK>(in.samples, in.space, in.channels, in.groups, &g)) {
    a.scratch.sums = static_cast<float2*>(in.workspace);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(in.samples * g.tiles * g.chunks));
    cfg.blockDim = dim3(B::kThreads);
    cfg.dynamicSmemBytes = S::smem(g.unroll);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(g.chunks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = NR_PDL ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, small, a, g);
    if (e != cudaSuccess || in.dw == nullptr || in.samples == 1) return e;
    // a warp a channel, up to the SMs' worth of blocks
    const int64_t blocks = (in.channels * kWarp + kGnSumThreads - 1) / kGnSumThreads;
    return launch_pdl(gn_grad_sum_kernel,
                      dim3(static_cast<unsigned>(blocks < 4 * kGnSms ? blocks : 4 * kGnSms)),
                      dim3(kGnSumThreads), 0, s, a, g);
  }
  g = gn_geometry<T, BACK>(in.samples, in.space, in.channels, in.groups);
  a.scratch.parts = static_cast<float2*>(in.workspace);
  a.scratch.sums = a.scratch.parts + g.samples * g.chunks * (g.groups + g.tiles);
  // the ring's used part, or what joining needs
  const int64_t turns = (g.steps + g.chunks - 1) / g.chunks;
  const int ring = B::kStepBytes * static_cast<int>(turns < B::kRing ? turns : B::kRing);
  const size_t smem = ring > B::kScratch ? ring : B::kScratch;
  const dim3 grid(static_cast<unsigned>(g.samples * g.chunks * g.tiles));
  e = launch_pdl(stats, grid, dim3(B::kThreads), smem, s, a, g);
  if (e != cudaSuccess) return e;
  return launch_pdl(apply, grid, dim3(B::kThreads), smem, s, a, g);
}

template <typename T, bool BACK>
cudaError_t gn_launch_act(const GroupNormArgs& in, cudaStream_t s) {
  return in.silu ? gn_launch<T, BACK, true>(in, s) : gn_launch<T, BACK, false>(in, s);
}

// Bytes of scratch, and blocks of a launch.
template <typename T>
int64_t gn_workspace(int64_t samples, int64_t space, int64_t channels, int64_t groups, int backward,
                     int64_t* blocks) {
  GnGeom g;
  if (backward ? gn_small_geometry<T, true>(samples, space, channels, groups, &g)
               : gn_small_geometry<T, false>(samples, space, channels, groups, &g)) {
    *blocks = samples * g.tiles * g.chunks;
    return backward && samples > 1 ? samples * channels * static_cast<int64_t>(sizeof(float2)) : 0;
  }
  g = backward ? gn_geometry<T, true>(samples, space, channels, groups)
               : gn_geometry<T, false>(samples, space, channels, groups);
  *blocks = samples * g.chunks * g.tiles;
  return backward ? gn_scratch_bytes<T, true>(g) : gn_scratch_bytes<T, false>(g);
}

}  // namespace

int64_t group_norm_workspace(int64_t samples, int64_t space, int64_t channels, int64_t groups,
                             int backward, int is_bf16, int64_t* blocks) {
  return is_bf16
             ? gn_workspace<__nv_bfloat16>(samples, space, channels, groups, backward, blocks)
             : gn_workspace<float>(samples, space, channels, groups, backward, blocks);
}

cudaError_t launch_group_norm(const GroupNormArgs& a, int is_bf16, cudaStream_t stream) {
  return is_bf16 ? gn_launch_act<__nv_bfloat16, false>(a, stream)
                 : gn_launch_act<float, false>(a, stream);
}

cudaError_t launch_group_norm_backward(const GroupNormArgs& a, int is_bf16, cudaStream_t stream) {
  return is_bf16 ? gn_launch_act<__nv_bfloat16, true>(a, stream)
                 : gn_launch_act<float, true>(a, stream);
}

}  // namespace nr
