// How cache attention's work is shared out, and the pieces its kernels have in common
// (sm_103a).
//
// An item is a block of up to R query rows of one sequence and K/V head (row t * group + i
// is query token t, the i-th of the head's query heads); its work is counted in tiles of
// kAttnTile positions.  All items' tiles, in order of (sequence, head, row block, tile),
// are cut into equal shares, one a block: lengths are known on the device alone, and long
// sequences are split while short ones share a block.  A block meets at most one item that
// began before its share and one that ends behind it; their partial results go to the
// workspace and a second kernel joins them, in the order of the shares.
#pragma once

#include "quant.cuh"

namespace nr {

constexpr int kAttnTile = 64;  // positions
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
    tiles = max(1, (n + kAttnTile - 1) / kAttnTile);  // an item without positions writes zeros
  }
};

// R rows an item: row blocks of a sequence.
template <int R>
__device__ __forceinline__ int64_t row_blocks(const AttnArgs& a, const AttnSeq& s) {
  return (static_cast<int64_t>(s.queries) * a.group.div + R - 1) / R;
}

// Where in the order of all tiles each thread's sequences begin; shared by the block.
template <int THREADS>
struct AttnPlan {
  int64_t at[THREADS + 1];
  int64_t warp[THREADS / kWarp];
};

template <int R, int THREADS>
__device__ __forceinline__ void make_plan(const AttnArgs& a, AttnPlan<THREADS>& plan) {
  const int t = threadIdx.x, lane = t % kWarp;
  const int per = (a.seqs + THREADS - 1) / THREADS;
  int64_t n = 0;
  for (int i = 0; i < per; i++) {
    const int64_t s = static_cast<int64_t>(t) * per + i;
    if (s >= a.seqs) break;
    const AttnSeq q(a, static_cast<int>(s));
    n += row_blocks<R>(a, q) * a.heads * q.tiles;
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

template <int R, int THREADS>
__device__ __forceinline__ AttnItem locate(const AttnArgs& a, const AttnPlan<THREADS>& plan,
                                           int64_t unit) {
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
    const AttnSeq q(a, s);
    const int64_t rbs = row_blocks<R>(a, q), n = rbs * a.heads * q.tiles;
    if (left < n) {
      const int64_t item = left / q.tiles;
      const int h = static_cast<int>(item / rbs);
      return AttnItem{s, h, static_cast<int>(item - h * rbs),
                      static_cast<int>(left - item * q.tiles)};
    }
    left -= n;
  }
}

__device__ __forceinline__ float attn_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Whether query token t (row `token` of q) of a sequence sees position p < length.
__device__ __forceinline__ bool attn_sees(const AttnArgs& a, const AttnSeq& s, int t, int p) {
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

}  // namespace nr
