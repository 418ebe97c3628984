// How cache attention's work is shared out, and the pieces its kernels have in common
// (sm_103a).
//
// An item is a block of up to R query rows of one sequence and K/V head (row t * group + i
// is query token t, the i-th of the head's query heads); its work is counted in tiles of
// TILE positions, behind COST units for what an item costs besides them (its queries, the start
// of its loads, its result).  All items' units, in order of (sequence, head, row block, tile),
// are cut into equal shares, one a block: lengths are known on the device alone, and long
// sequences are split while short ones share a block.  A tile belongs to the share that its unit is in.  A block meets at most one item that
// began before its share and one that ends behind it; their partial results go to the
// workspace and a second kernel joins them, in the order of the shares.
#pragma once

#include "quant.cuh"

namespace nr {

constexpr int kAttnMostPositions = 1 << 30;
constexpr float kAttnLog2e = 1.4426950408889634f;
constexpr float kAttnLn2 = 0.6931471805599453f;

struct AttnArgs {
  const void* q;
  void* out;
  float* lse;  // or null
  CacheSide side[2];
  CacheGeom geo;
  const int32_t* table;  // [seqs, width]
  const int32_t* lens;   // [seqs]
  const int32_t* cu;     // [seqs + 1], or null: one query token a sequence
  const uint32_t* tree;  // [tokens, words], or null
  int64_t width;
  int64_t blocks;
  int64_t q_stride;  // elements between tokens
  int64_t tokens;
  int seqs;
  int heads;
  FastDiv group;  // query heads a K/V head
  FastDiv page;
  int words;
  float scale_log2;  // the scores' scale, times log2(e)
  bool wide_scales;  // MXFP4: a head's scale bytes are aligned to their number
  float* partial;    // [2 shares, R, DIM + 2]
  int4* joins;       // [shares]: sequence, head, row block, shares of the item that begins there
};

// One sequence's queries and lengths, clamped to what is there: the tables are data that the
// host does not see.
template <int TILE>
struct AttnSeq {
  int first;     // its first query token
  int queries;   // T
  int length;    // L
  int context;   // L - T, may be negative: position of its first own token
  int tiles;     // of positions that the table reaches; at least one
  __device__ __forceinline__ AttnSeq(const AttnArgs& a, int s) {
    first = s, queries = 1;
    if (a.cu != nullptr) {
      const int64_t lo = a.cu[s], hi = a.cu[s + 1];
      first = static_cast<int>(lo < 0 ? 0 : lo > a.tokens ? a.tokens : lo);
      const int64_t end = hi > a.tokens ? a.tokens : hi;
      queries = end > first ? static_cast<int>(end - first) : 0;
    }
    length = min(max(a.lens[s], 0), kAttnMostPositions);
    context = length - queries;
    const int64_t reach = a.width * a.geo.block_size;
    const int n = reach < length ? static_cast<int>(reach) : length;
    tiles = max(1, (n + TILE - 1) / TILE);  // an item without positions writes zeros
  }
};

// R rows an item: row blocks of a sequence.
template <int R>
__device__ __forceinline__ int64_t row_blocks(const AttnArgs& a, int queries) {
  return (static_cast<int64_t>(queries) * a.group.div + R - 1) / R;
}

// Where in the order of all tiles each thread's sequences begin; shared by the block.
template <int THREADS>
struct AttnPlan {
  int64_t at[THREADS + 1];
  int64_t warp[THREADS / kWarp];
};

template <int R, int TILE, int COST, int THREADS>
__device__ __forceinline__ void make_plan(const AttnArgs& a, AttnPlan<THREADS>& plan) {
  const int t = threadIdx.x, lane = t % kWarp;
  const int per = (a.seqs + THREADS - 1) / THREADS;
  int64_t n = 0;
  for (int i = 0; i < per; i++) {
    const int64_t s = static_cast<int64_t>(t) * per + i;
    if (s >= a.seqs) break;
    const AttnSeq<TILE> q(a, static_cast<int>(s));
    n += row_blocks<R>(a, q.queries) * a.heads * (q.tiles + COST);
  }
#pragma unroll
  for (int d = 1; d < kWarp; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xFFFFFFFFu, n, d);
    if (lane >= d) n += o;
  }
  if (lane == kWarp - 1) plan.warp[t / kWarp] = n;
  __syncthreads();
  for (int w = 0; w < t / kWarp; w++) n += plan.warp[w];
  plan.at[t + 1] = n;
  if (t == 0) plan.at[0] = 0;
  __syncthreads();
}

// The tiles of one share; the last shares may be empty.
__device__ __forceinline__ int64_t share_size(int64_t total, int64_t shares) {
  return (total + shares - 1) / shares;
}

// A place in the order: an item and a tile of it.
struct AttnItem {
  int seq, head, rb, tile;
};

// The first tile at or behind `unit` (moved on to that tile's).
template <int R, int TILE, int COST, int THREADS>
__device__ __forceinline__ AttnItem locate(const AttnArgs& a, const AttnPlan<THREADS>& plan,
                                           int64_t& unit) {
  int lo = 0, hi = THREADS;  // at[lo] <= unit < at[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (plan.at[mid] <= unit) lo = mid;
    else hi = mid;
  }
  const int per = (a.seqs + THREADS - 1) / THREADS;
  int s = lo * per;
  int64_t left = unit - plan.at[lo];
  for (;; s++) {
    const AttnSeq<TILE> q(a, s);
    const int64_t rbs = row_blocks<R>(a, q.queries), each = q.tiles + COST, n = rbs * a.heads * each;
    if (left < n) {
      const int64_t item = left / each;
      const int h = static_cast<int>(item / rbs);
      const int off = static_cast<int>(left - item * each) - COST;
      if (off < 0) unit -= off;
      return AttnItem{s, h, static_cast<int>(item - h * rbs), off < 0 ? 0 : off};
    }
    left -= n;
  }
}

// The first tile of the item behind `it` in the order (there is one).
template <int R, int TILE>
__device__ __forceinline__ void next_item(const AttnArgs& a, AttnItem& it, int queries) {
  it.tile = 0;
  if (++it.rb < row_blocks<R>(a, queries)) return;
  it.rb = 0;
  if (++it.head < a.heads) return;
  it.head = 0;
  do it.seq++;
  while (AttnSeq<TILE>(a, it.seq).queries == 0);
}

__device__ __forceinline__ float attn_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Whether query token t (row `token` of q) of a sequence sees position p < length.
template <int TILE>
__device__ __forceinline__ bool attn_sees(const AttnArgs& a, const AttnSeq<TILE>& s, int t, int p) {
  const int j = p - s.context;
  if (j < 0) return true;
  if (a.tree == nullptr) return j <= t;
  if ((j >> 5) >= a.words) return false;
  return a.tree[static_cast<int64_t>(s.first + t) * a.words + (j >> 5)] >> (j & 31) & 1u;
}

// Widening two codes to f16 (exact).
__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
// Four bytes, two e2m1 codes each.
__device__ __forceinline__ void half2_of_e2m1(uint32_t x, uint32_t (&r)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(x));
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 floats_of_half2(uint32_t h) {
  float2 v;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.f32.f16 %0, lo;\n cvt.f32.f16 %1, hi;\n}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(h));
  return v;
}

constexpr int kScaleUp = 13;  // MXFP4 values are held times 2^13

// The scale bytes of one token and head: f16 multipliers relative to the largest (a NaN scale
// stays a NaN), times 2^kScaleUp; the largest as f32 without that factor.
template <int G>
__device__ __forceinline__ float mx_multipliers(uint64_t bytes, uint16_t (&m)[G]) {
  auto byte = [&](int i) { return static_cast<int>(bytes >> (8 * i)) & 255; };
  int top = 0;
#pragma unroll
  for (int i = 0; i < G; i++) top = max(top, byte(i));
  const bool nan = top == 255;
  if (nan) {  // seldom
    top = 0;
#pragma unroll
    for (int i = 0; i < G; i++)
      if (byte(i) != 255) top = max(top, byte(i));
  }
  // 2^(byte - top + kScaleUp) as f32, then as f16: below its smallest, 2^-24, it becomes 0 (2^-25 is
  // halfway and 0 the even neighbour)
  const int base = 127 + kScaleUp - top;
#pragma unroll
  for (int i = 0; i < G; i += 2) {
    const uint32_t two =
        half2_of(__uint_as_float(static_cast<uint32_t>(max(byte(i) + base, 0)) << 23),
                 __uint_as_float(static_cast<uint32_t>(max(byte(i + 1) + base, 0)) << 23));
    m[i] = static_cast<uint16_t>(two);
    m[i + 1] = static_cast<uint16_t>(two >> 16);
  }
  if (nan) {
#pragma unroll
    for (int i = 0; i < G; i++)
      if (byte(i) == 255) m[i] = 0x7E00;
  }
  // 2^(top - 127 - kScaleUp); below 2^-126: nothing that f32 scores would see
  const int e = top - kScaleUp;
  return e > 0 ? __uint_as_float(static_cast<uint32_t>(e) << 23) : 0.0f;
}

// Weights times V's scales, for the second product's f16.  A row holds e^(score - m) |scale| as that times
// a power of two, so that the largest it has met (t, the maximum of score + k in units of log2, with
// |scale| < 2^k) is held in [2^(HOLD - 3/2), 2^(HOLD + 1/2)): a token that nobody attends to does not
// count, whatever its scale.
__device__ __forceinline__ float scale_exponent(float s) {  // k; none for a scale that is not finite
  const uint32_t e = __float_as_uint(s) >> 23 & 255u;
  return e == 255u ? -__builtin_huge_valf() : static_cast<float>(static_cast<int>(e) - 126);
}
// That power of two, 2^(HOLD - round(t - m)).  (Below -104 the products with it would leave f32's range;
// above 128 there is no scale.)  Behind the addition the low bits are the exponent's.
template <int HOLD>
__device__ __forceinline__ float hold_factor(float t, float m) {
  const float r = fminf(fmaxf(t - m, -104.0f), 128.0f);
  return __uint_as_float(__float_as_uint((12582912.0f + (127 + HOLD)) - r) << 23);
}
// The reciprocal of a power of two between 2^-126 and 2^126.
__device__ __forceinline__ float power_reciprocal(float p) {
  return __uint_as_float((254u << 23) - __float_as_uint(p));
}

template <typename T>
__device__ __forceinline__ T narrow(float x) {
  return static_cast<T>(x);
}

namespace {

// Joins the parts of the items that more than one share worked on: block (i, y) rows
// kJoinRows y + threadIdx.y of the item that begins in share i, four dimensions a thread.  (FP4 says
// whose parts: each kernel's own joining asks for the shared memory that the kernel asks for.)
constexpr int kJoinRows = 4;
template <typename T, int R, int DIM, bool FP4>
__global__ void __launch_bounds__(DIM / 4 * kJoinRows) cache_attention_join_kernel(const AttnArgs a) {
  pdl_enter();
  const int4 join = a.joins[blockIdx.x];
  if (join.w == 0) return;
  const AttnSeq<1> seq(a, join.x);
  const int r = blockIdx.y * kJoinRows + threadIdx.y;
  const int row = join.z * R + r;
  if (row >= seq.queries * static_cast<int>(a.group.div)) return;
  constexpr int64_t kPart = R * (DIM + 2);
  const float* first = a.partial + (2 * static_cast<int64_t>(blockIdx.x) + 1) * kPart;
  const float* rest = first + kPart;  // share i + 1's first part, and every second one behind it
  auto part = [&](int i) { return i == 0 ? first : rest + (i - 1) * 2 * kPart; };
  // Some parts' sums and values at a time, on their way together.
  constexpr int kAtOnce = 8;
  float top = -__builtin_huge_valf(), sum = 0.0f;
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int base = 0; base < join.w; base += kAtOnce) {
    float2 ml[kAtOnce];
    float4 y[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; i++) {
      const bool in = base + i < join.w;
      const float* p = part(in ? base + i : 0);
      ml[i] = in ? *reinterpret_cast<const float2*>(p + R * DIM + 2 * r)
                 : make_float2(-__builtin_huge_valf(), 0.0f);
      y[i] = in ? *reinterpret_cast<const float4*>(p + r * DIM + 4 * threadIdx.x)
                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    float to = top;
#pragma unroll
    for (int i = 0; i < kAtOnce; i++) to = fmaxf(to, ml[i].x);
    if (top != -__builtin_huge_valf()) {
      const float f = attn_exp2(top - to);
      sum *= f;
      x.x *= f, x.y *= f, x.z *= f, x.w *= f;
    }
    top = to;
#pragma unroll
    for (int i = 0; i < kAtOnce; i++) {
      if (ml[i].y == 0.0f) continue;
      const float f = attn_exp2(ml[i].x - top);
      sum = fmaf(ml[i].y, f, sum);
      x.x = fmaf(y[i].x, f, x.x), x.y = fmaf(y[i].y, f, x.y);
      x.z = fmaf(y[i].z, f, x.z), x.w = fmaf(y[i].w, f, x.w);
    }
  }
  const int tok = a.group.quot(row), i_head = row - tok * a.group.div;
  const int64_t head = static_cast<int64_t>(seq.first + tok) * a.heads * a.group.div +
                       join.y * a.group.div + i_head;
  const float inv = sum != 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
  T* out = static_cast<T*>(a.out) + head * DIM + 4 * threadIdx.x;
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(out) =
        make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
  else
    *reinterpret_cast<float4*>(out) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
  if (threadIdx.x == 0 && a.lse != nullptr)
    a.lse[head] = sum != 0.0f ? (top + log2f(sum)) * kAttnLn2 : -__builtin_huge_valf();
}

// Shared memory of a kernel, once a device: the opt-in to more than 48 KB, and how much of the SM's
// memory is to be shared memory, in percent.  Both kernels of a call ask for the same: an SM that
// the join ran on with a small share has no room for all blocks of the next call, which then runs in
// two waves (400009 tokens, calls back to back: 428 us, calls apart 272 us).
template <typename Kernel>
cudaError_t allow_shared(Kernel kernel, size_t bytes, std::atomic<int>* done, int percent = 100) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  if (done[device].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             percent);
  if (e == cudaSuccess) done[device].store(1, std::memory_order_relaxed);
  return e;
}

// Room for the joins of `shares` shares of R rows: 16 bytes a share, then two parts each.
constexpr int64_t attn_joins_bytes(int64_t shares) { return (shares * 16 + 127) / 128 * 128; }
constexpr int64_t attn_bytes(int64_t shares, int64_t rows, int64_t dim) {
  return attn_joins_bytes(shares) + 2 * shares * rows * (dim + 2) * 4;
}

}  // namespace

// Many rows an item, bf16 tensors, heads of 64 or 128 (cache_attention_rows.cu).
int64_t attn_rows_bytes(int64_t head_dim);
cudaError_t launch_attn_rows(const AttnArgs& a, bool fp4, int64_t head_dim, void* workspace,
                             cudaStream_t stream);

}  // namespace nr
