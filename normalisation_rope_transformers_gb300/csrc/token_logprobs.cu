// Log probabilities of given tokens, entropy and the largest alternatives of rows of
// logits, and the gradient with respect to the logits (sm_103a).
//
// With z = logits / temperature, m = max z and d = z - m <= 0:
//   l = sum e^d,  e = sum d e^d,  lse = m + ln l,  logprob = z_token - lse,
//   entropy = ln l - e / l
// One pass: each thread keeps its own (m, l, e) and rescales them when its maximum
// grows, the block joins them at the end.  HBM bounds many rows (one read of the
// logits), a block's latency few of them; those are split over a cluster of blocks
// that join through distributed shared memory, in rank order.
//
// Alternatives: every element has a key of its own, value first, then the lowest
// index.  The k-th largest of the threads' maxima of the first chunk is a lower bound
// of the k-th largest element; the vectors whose maxima reach it are noted in a list in
// shared memory.  At the end one warp raises the bound to the k-th largest of the noted
// maxima, reads the vectors that reach that again and orders their elements.  (Noting the
// elements themselves costs 30 us at [4093, 151551] with k = 5, 110 us with k = 20.)  Where
// the list does not hold them (rising rows, many equal values) the whole row is read again,
// with a list that is cut to its k largest when it fills up, which raises the bound: any order
// of values ends.
//
// Gradient: dz = p (-g - h (ln p + H)) + g [j = token], p = e^(z - lse), g and h the
// gradients of logprob and entropy H: one read and one write of the logits.
//
// Measured, bf16: [4093, 151551] with five alternatives 237 us (0.77 of the copy rate; 197 us without:
// bound by issue, 70% of the slots), [5, 131072] with twenty 14 us (latency: one read, the bound, the
// list); the gradient at [4096, 131072] 303 us (1.05 of the copy rate), f32 [96, 32003] 4.7 us.
#include <cooperative_groups.h>

#include "nr_internal.h"
#include "nr_pairs.cuh"

namespace nr {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                       // vectors a thread and chunk
constexpr int kChunk = kThreads * kUnroll;       // vectors
constexpr int kList = 1000;                      // noted vectors, or candidates (below 1024)
constexpr int kFew = 64;                         // vectors read again
constexpr int kCandidates = 256;                 // elements of theirs
constexpr float kInf = __builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Running statistics in units of the logits: l = sum e^((x - m) / T), e = sum (x - m)
// e^((x - m) / T).
struct Stats {
  float m, l, e;
};

// a + b; c = log2(e) / T.  A side without elements above -inf has l = e = 0.
__device__ __forceinline__ Stats join(const Stats& a, const Stats& b, float c) {
  const float m = fmaxf(a.m, b.m);
  if (m == -kInf) return Stats{m, a.l + b.l, a.e + b.e};
  const float da = fmaxf(a.m - m, -1e30f), db = fmaxf(b.m - m, -1e30f);
  const float fa = exp2_fast(da * c), fb = exp2_fast(db * c);
  return Stats{m, fmaf(a.l, fa, b.l * fb),
               fmaf(fmaf(a.l, da, a.e), fa, fmaf(b.l, db, b.e) * fb)};
}

// Order-preserving whole numbers of f32 values (no NaN; -0 as 0).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
  return static_cast<uint64_t>(ordered(x)) << 32 | (0xFFFFFFFFu - index);
}

struct LogprobArgs {
  const void* logits;
  const int64_t* tokens;
  float* logprob;
  float* entropy;
  float* lse;
  float* top_logprob;  // [rows, top]
  int64_t* top_ids;
  int64_t stride;  // elements between rows
  uint32_t vocab;
  int top;
  int ranks;  // blocks a row (a cluster)
  float inv_t;
};

// A row's elements in front of its first 16-byte boundary, its whole vectors, and the
// elements behind them.
struct RowParts {
  uint32_t head, vecs, tail;
};
template <typename T>
__device__ __forceinline__ RowParts parts_of(const T* row, uint32_t vocab) {
  constexpr uint32_t N = Vec<T>::N;
  const uint32_t off = (reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T);
  RowParts p;
  p.head = off == 0 ? 0 : N - off;
  if (p.head > vocab) p.head = vocab;
  p.vecs = (vocab - p.head) / N;
  p.tail = vocab - p.head - p.vecs * N;
  return p;
}
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ uint4 all_low() {  // a vector of -inf
  const uint32_t w = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
  return make_uint4(w, w, w, w);
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Largest element of a vector (a NaN counts as nothing).
template <typename T>
__device__ __forceinline__ float top_of(const uint4& v);
template <>
__device__ __forceinline__ float top_of<__nv_bfloat16>(const uint4& v) {
  const uint32_t m = max_bf16x2(max_bf16x2(v.x, v.y), max_bf16x2(v.z, v.w));
  return fmaxf(fmaxf(bf16_lo(m), bf16_hi(m)), -kInf);
}
template <>
__device__ __forceinline__ float top_of<float>(const uint4& v) {
  return fmaxf(fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                     fmaxf(__uint_as_float(v.z), __uint_as_float(v.w))),
               -kInf);
}

// The largest T, zero below bit LOW, that at least k of a warp's values reach (0 if there are
// fewer): two bits at a time, three counts of at most 1023 in one word.  each(f) calls f with
// each value of the lane.
template <int LOW, typename Each>
__device__ __forceinline__ uint32_t kth_bound(const Each& each, int k, uint32_t from = 0,
                                              int high = 30) {
  uint32_t bound = from;
#pragma unroll 1
  for (int bit = high; bit >= LOW; bit -= 2) {
    uint32_t n = 0;
    each([&](uint32_t v) {
      n += (v >= (bound | 1u << bit) ? 1u : 0u) + (v >= (bound | 2u << bit) ? 1u << 10 : 0u) +
           (v >= (bound | 3u << bit) ? 1u << 20 : 0u);
    });
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    const uint32_t need = static_cast<uint32_t>(k);
    bound |= (n >> 20 >= need ? 3u : (n >> 10 & 1023u) >= need ? 2u : (n & 1023u) >= need ? 1u : 0u)
             << bit;
  }
  return bound;
}

// The k largest of `n` keys in shared memory, by one warp, in order, into `best`
// (zeros where there are fewer), one after the other.  The keys are lost.
__device__ __noinline__ void take_one_by_one(uint64_t* keys, int n, int k, uint64_t* best) {
  const int lane = threadIdx.x % kWarp;
  uint64_t mine = 0;
  int at = -1;
  auto scan = [&]() {
    mine = 0;
    for (int i = lane; i < n; i += kWarp)
      if (keys[i] > mine) mine = keys[i], at = i;
  };
  scan();
  for (int r = 0; r < k; r++) {
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(mine >> 32));
    const uint32_t lo = __reduce_max_sync(
        0xFFFFFFFFu, static_cast<uint32_t>(mine >> 32) == hi ? static_cast<uint32_t>(mine) : 0u);
    const uint64_t top = static_cast<uint64_t>(hi) << 32 | lo;
    if (lane == 0) best[r] = top;
    if (top != 0 && mine == top) {
      keys[at] = 0;
      scan();
    }
    __syncwarp();
  }
}

// The same where at most 32 keys reach the k-th largest value (its neighbours in the order
// included): a bound by bits of the value, and places by counting.  No key is there twice.
__device__ __forceinline__ void take_largest(uint64_t* keys, int n, int k, uint64_t* best) {
  const int lane = threadIdx.x % kWarp;
  auto each = [&](auto&& f) {
    for (int i = lane; i < n; i += kWarp) f(static_cast<uint32_t>(keys[i] >> 32));
  };
  auto reach = [&](uint32_t bound) {
    uint32_t c = 0;
    each([&](uint32_t v) { c += v >= bound; });
    return __reduce_add_sync(0xFFFFFFFFu, c);
  };
  uint32_t bound = 0;
  if (n > kWarp) {
    bound = kth_bound<16>(each, k);
    if (reach(bound) > kWarp) {
      bound = kth_bound<0>(each, k, bound, 14);
      if (reach(bound) > kWarp) {  // equal values
        take_one_by_one(keys, n, k, best);
        return;
      }
    }
  }
  int have = 0;
  for (int base = 0; base < n; base += kWarp) {
    const uint64_t key = base + lane < n ? keys[base + lane] : 0;
    const unsigned in = __ballot_sync(0xFFFFFFFFu, key != 0 && static_cast<uint32_t>(key >> 32) >= bound);
    const int at = have + __popc(in & ((1u << lane) - 1u));
    if (in >> lane & 1u) best[at] = key;
    have += __popc(in);
  }
  __syncwarp();
  const uint64_t mine = lane < have ? best[lane] : 0;
  int rank = 0;
#pragma unroll 8
  for (int i = 0; i < kWarp; i++) rank += __shfl_sync(0xFFFFFFFFu, mine, i) > mine;
  __syncwarp();
  best[lane] = 0;
  __syncwarp();
  if (mine != 0 && rank < k) best[rank] = mine;
  __syncwarp();
}

// What a block shares; the other blocks of its cluster are read by the first.
struct Shared {
  uint64_t list[kList];
  uint64_t candidates[kCandidates];
  uint32_t few[kFew];
  uint64_t best[kLogprobMostTop];
  uint64_t bound;
  uint32_t maxima[kThreads];
  Stats stats[kThreads / kWarp];
  Stats total;
  int count;
  int lost;  // something had no room
};

// A thread's element outside the vectors.
struct Extra {
  float x;
  uint32_t at;
};

// The largest elements from the noted vectors and the extra elements, by one warp.  Sets
// sh.lost where they have no room.
template <typename T>
__device__ __forceinline__ void read_noted(Shared& sh, const uint4* body, uint32_t head,
                                           const Extra& extra, int top) {
  constexpr int N = Vec<T>::N;
  const int lane = threadIdx.x % kWarp;
  const int n = sh.count;
  const uint32_t bound = kth_bound<16>(
      [&](auto&& f) {
        for (int i = lane; i < n; i += kWarp) f(static_cast<uint32_t>(sh.list[i] >> 32));
      },
      top);
  const unsigned before = (1u << lane) - 1u;
  int few = 0;
  for (int base = 0; base < n; base += kWarp) {
    const uint64_t note = base + lane < n ? sh.list[base + lane] : 0;
    const bool in = note != 0 && static_cast<uint32_t>(note >> 32) >= bound;
    const unsigned all = __ballot_sync(0xFFFFFFFFu, in);
    const int at = few + __popc(all & before);
    if (in && at < kFew) sh.few[at] = static_cast<uint32_t>(note);
    few += __popc(all);
  }
  __syncwarp();
  int have = 0;
  auto offer = [&](uint64_t key) {  // by the whole warp; 0: nothing
    const bool in = key != 0 && static_cast<uint32_t>(key >> 32) >= bound;
    const unsigned all = __ballot_sync(0xFFFFFFFFu, in);
    const int at = have + __popc(all & before);
    if (in && at < kCandidates) sh.candidates[at] = key;
    have += __popc(all);
  };
  for (int base = 0; base < min(few, kFew); base += kWarp) {
    const bool in = base + lane < min(few, kFew);
    const uint32_t v = in ? sh.few[base + lane] : 0;
    float u[N];
    Vec<T>::unpack(in ? ld_param(body + v) : make_uint4(0u, 0u, 0u, 0u), u);
#pragma unroll
    for (int i = 0; i < N; i++) offer(in && u[i] == u[i] ? key_of(u[i], head + v * N + i) : 0);
  }
  offer(extra.at != 0xFFFFFFFFu && extra.x == extra.x ? key_of(extra.x, extra.at) : 0);
  __syncwarp();
  if (few > kFew || have > kCandidates) {
    if (lane == 0) sh.lost = 1;
  } else {
    take_largest(sh.candidates, have, top, sh.best);
  }
}

// The candidates of the vectors [v0, v1) and of the extra elements once more, into a list that
// is cut to its `top` largest whenever it is full.  All threads of the block.
template <typename T>
__device__ __noinline__ void collect_again(Shared& sh, const uint4* body, uint32_t head, uint32_t v0,
                                           uint32_t v1, Extra extra, uint64_t bound, int top) {
  constexpr int N = Vec<T>::N;
  const int t = threadIdx.x;
  __syncthreads();
  if (t == 0) sh.count = 0;
  __syncthreads();
  for (uint32_t base = v0; base < v1 + kThreads; base += kThreads) {
    // one vector a thread; past the last ones, the extra elements
    uint64_t key[N];
    const uint32_t v = base + t;
    float u[N];
    if (v < v1) Vec<T>::unpack(ld_param(body + v), u);
#pragma unroll
    for (int i = 0; i < N; i++)
      key[i] = v < v1 && u[i] == u[i] ? key_of(u[i], head + v * N + i) : 0;
    if (base >= v1) key[0] = extra.at != 0xFFFFFFFFu && extra.x == extra.x ? key_of(extra.x, extra.at) : 0;
    bool left = true;
    for (;;) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < N; i++) n += left && key[i] > bound;
      bool kept = true;
      if (n > 0) {
        int at = atomicAdd(&sh.count, n);
        kept = at + n <= kList;
        if (kept) {
#pragma unroll
          for (int i = 0; i < N; i++)
            if (key[i] > bound) sh.list[at++] = key[i];
        } else {
          for (int i = at; i < kList && i < at + n; i++) sh.list[i] = 0;
        }
      }
      if (kept) left = false;
      if (!__syncthreads_or(!kept)) break;
      if (t < kWarp) {
        take_largest(sh.list, kList, top, sh.best);
        for (int i = t; i < top; i += kWarp) sh.list[i] = sh.best[i];
        if (t == 0) sh.count = top, sh.bound = sh.best[top - 1];
      }
      __syncthreads();
      bound = sh.bound;
    }
  }
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, 4) token_logprobs_kernel(const LogprobArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ Shared sh;
  const int t = threadIdx.x;
  const uint32_t ranks = static_cast<uint32_t>(a.ranks);
  const uint32_t row = blockIdx.x / ranks, rank = blockIdx.x - row * ranks;
  const T* x = static_cast<const T*>(a.logits) + static_cast<int64_t>(row) * a.stride;
  const RowParts part = parts_of(x, a.vocab);
  const uint4* body = reinterpret_cast<const uint4*>(x + part.head);
  const uint32_t per = (part.vecs + ranks - 1) / ranks;
  const uint32_t v0 = min(rank * per, part.vecs), v1 = min(v0 + per, part.vecs);
  const float c = kLog2e * a.inv_t;
  if (TOP) {
    if (t == 0) sh.count = 0, sh.lost = 0;
    __syncthreads();
  }
  pdl_enter();  // before any global read: the previous kernel may still run

  uint4 next[kUnroll];
  auto load = [&](uint32_t base) {
#pragma unroll
    for (int j = 0; j < kUnroll; j++) {
      const uint32_t v = base + t + j * kThreads;
      next[j] = v < v1 ? ld_stream(body + v) : all_low<T>();
    }
  };
  load(v0);
  // An element outside the vectors: thread t < head has element t, thread 8 + i the
  // i-th behind them (the first block alone).
  float extra = -kInf;
  uint32_t extra_at = 0xFFFFFFFFu;
  if (rank == 0) {
    if (static_cast<uint32_t>(t) < part.head) extra_at = t;
    if (t >= 8 && static_cast<uint32_t>(t - 8) < part.tail)
      extra_at = a.vocab - part.tail + (t - 8);
    if (extra_at < a.vocab) extra = widen(x[extra_at]);
  }
  int64_t token = -1;
  float at_token = 0.0f;
  if (rank == 0 && t == 0) {
    token = a.tokens[row];
    if (token >= 0 && token < a.vocab) at_token = widen(x[token]);
  }

  Stats s{-kInf, 0.0f, 0.0f};
  uint64_t bound = 0;      // keys above it are candidates
  float bound_v = -kInf;   // its value
  bool first = true;
  for (uint32_t base = v0; base < v1; base += kChunk) {
    uint4 raw[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; j++) raw[j] = next[j];
    if (base + kChunk < v1) load(base + kChunk);
    float tops[kUnroll], top = -kInf;
#pragma unroll
    for (int j = 0; j < kUnroll; j++) tops[j] = top_of<T>(raw[j]), top = fmaxf(top, tops[j]);
    if (top > s.m) {
      const float d = fmaxf(s.m - top, -1e30f), f = exp2_fast(d * c);
      s.e = fmaf(s.l, d, s.e) * f;
      s.l *= f;
      s.m = top;
    }
    const float m = s.m == -kInf ? 0.0f : s.m;
    const F2 m2 = f2(m, m), c2 = f2(c, c);
    F2 l2 = f2(0.0f, 0.0f), e2 = f2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < kUnroll; j++) {
      F2 v[N / 2];
      Pairs<T>::unpack(raw[j], v);
#pragma unroll
      for (int i = 0; i < N / 2; i++) {
        const F2 d = sub2(v[i], m2);
        float u[2], p[2], q[2];
        split(d, u[0], u[1]);
        split(mul2(d, c2), p[0], p[1]);
#pragma unroll
        for (int h = 0; h < 2; h++) {
          p[h] = exp2_fast(p[h]);
          q[h] = fmaxf(u[h], -1e30f);  // 0 * -inf of a masked logit would be a NaN
        }
        const F2 pp = f2(p[0], p[1]);
        l2 = add2(l2, pp);
        e2 = fma2(pp, f2(q[0], q[1]), e2);
      }
    }
    float lo, hi;
    split(l2, lo, hi);
    s.l += lo + hi;
    split(e2, lo, hi);
    s.e += lo + hi;
    if (TOP) {
      if (first) {
        // the k-th largest of the threads' maxima, its leading bits
        first = false;
        sh.maxima[t] = ordered(top);
        __syncthreads();
        uint32_t have[kThreads / kWarp];
#pragma unroll
        for (int i = 0; i < kThreads / kWarp; i++) have[i] = sh.maxima[i * kWarp + t % kWarp];
        const uint32_t kth = kth_bound<16>(
            [&](auto&& f) {
#pragma unroll
              for (int i = 0; i < kThreads / kWarp; i++) f(have[i]);
            },
            a.top);
        if (kth > ordered(-kInf)) {
          bound = static_cast<uint64_t>(kth) << 32;
          bound_v = value_of(kth);
        }
      }
      if (top >= bound_v) {
#pragma unroll
        for (int j = 0; j < kUnroll; j++) {
          const uint32_t v = base + t + j * kThreads;
          if (v >= v1 || tops[j] < bound_v) continue;
          // (nothing more is worth noting once one had no room)
          if (*static_cast<volatile int*>(&sh.lost)) continue;
          const int at = atomicAdd(&sh.count, 1);
          if (at < kList)
            sh.list[at] = static_cast<uint64_t>(ordered(tops[j])) << 32 | v;
          else
            sh.lost = 1;
        }
      }
    }
  }
  if (rank == 0 && (part.head | part.tail)) {
    if (extra_at < a.vocab) s = join(s, Stats{extra, extra == -kInf ? 0.0f : 1.0f, 0.0f}, c);
    if (!(extra < kInf)) s.l = extra - extra;  // a NaN or +inf: no probabilities
  }

  // the block's statistics, in a fixed order
#pragma unroll
  for (int d = kWarp / 2; d > 0; d >>= 1) {
    const Stats o{__shfl_xor_sync(0xFFFFFFFFu, s.m, d), __shfl_xor_sync(0xFFFFFFFFu, s.l, d),
                  __shfl_xor_sync(0xFFFFFFFFu, s.e, d)};
    s = (t & d) ? join(o, s, c) : join(s, o, c);
  }
  if (t % kWarp == 0) sh.stats[t / kWarp] = s;
  __syncthreads();
  if (TOP) {
    if (t < kWarp && !sh.lost)
      read_noted<T>(sh, body, part.head, Extra{extra, extra_at}, a.top);
    __syncthreads();
    if (sh.lost)
      collect_again<T>(sh, body, part.head, v0, v1, Extra{extra, extra_at}, bound, a.top);
  }
  if (t < kWarp) {
    s = sh.stats[0];
    for (int i = 1; i < kThreads / kWarp; i++) s = join(s, sh.stats[i], c);
    if (TOP && sh.lost) take_largest(sh.list, min(sh.count, kList), a.top, sh.best);
    if (t == 0) sh.total = s;
  }
  if (ranks > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (rank == 0 && t < kWarp) {
      for (uint32_t r = 1; r < ranks; r++)
        s = join(s, *cluster.map_shared_rank(&sh.total, r), c);
      if (TOP) {
        const int n = static_cast<int>(ranks) * a.top;
        for (int i = t; i < n; i += kWarp) {
          const int r = i / a.top;
          sh.list[i] = *cluster.map_shared_rank(&sh.best[i - r * a.top], r);
        }
        __syncwarp();
        take_largest(sh.list, n, a.top, sh.best);
      }
    }
    cluster.sync();  // the others' shared memory is read until here
  }
  if (rank != 0 || t >= kWarp) return;
  const bool none = s.m == -kInf && s.l == 0.0f;  // every logit is -inf
  const float ln_l = kLn2 * log2f(s.l);
  auto logprob = [&](float v) { return none ? -kInf : fmaf(v - s.m, a.inv_t, -ln_l); };
  if (t == 0) {
    a.lse[row] = none ? -kInf : fmaf(s.m, a.inv_t, ln_l);
    a.entropy[row] = none ? 0.0f : fmaf(-__fdiv_rn(s.e, s.l), a.inv_t, ln_l);
    a.logprob[row] = token >= 0 && token < a.vocab ? logprob(at_token) : 0.0f;
  }
  if (TOP) {
    __syncwarp();
    for (int i = t; i < a.top; i += kWarp) {
      const uint64_t k = sh.best[i];
      const bool bad = s.l != s.l;  // a NaN in the row
      const int64_t at = static_cast<int64_t>(row) * a.top + i;
      a.top_ids[at] = bad || k == 0 ? -1 : static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(k));
      a.top_logprob[at] = bad ? s.l : logprob(value_of(static_cast<uint32_t>(k >> 32)));
    }
  }
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------
struct LogprobGradArgs {
  void* dlogits;
  const float* dlogprob;  // or null
  const float* dentropy;  // or null
  const void* logits;
  const int64_t* tokens;
  const float* lse;
  const float* entropy;
  int64_t stride, out_stride;
  uint32_t vocab;
  uint32_t blocks;  // blocks a row
  float inv_t;
};

// dz of a pair of logits without the token's own term: p = e^(z - lse),
// -p (g + h (ln p + H)), all times 1 / T.
struct GradRow {
  F2 inv_t, neg_lse, a, b;  // dz = p (a + b ln p)
  __device__ __forceinline__ F2 operator()(F2 x) const {
    const F2 lp = fma2(x, inv_t, neg_lse);
    float u[2];
    split(lp, u[0], u[1]);
    // p = 0 far above this; a masked logit's 0 * -inf would be a NaN, and 0 times what leaves f32's
    // range with a large gradient of the entropy too
    u[0] = fmaxf(u[0], -1e3f);
    u[1] = fmaxf(u[1], -1e3f);
    const F2 p = f2(exp2_fast(u[0] * kLog2e), exp2_fast(u[1] * kLog2e));
    return mul2(p, fma2(b, f2(u[0], u[1]), a));
  }
};

template <typename T, bool SAME>
__global__ void __launch_bounds__(kThreads) token_logprobs_grad_kernel(const LogprobGradArgs a) {
  constexpr int N = Vec<T>::N;
  const int t = threadIdx.x;
  const uint32_t row = blockIdx.x / a.blocks, chunk = blockIdx.x - row * a.blocks;
  const T* x = static_cast<const T*>(a.logits) + static_cast<int64_t>(row) * a.stride;
  T* out = static_cast<T*>(a.dlogits) + static_cast<int64_t>(row) * a.out_stride;
  const RowParts part = parts_of(out, a.vocab);  // whole vectors of the output
  const T* body = x + part.head;
  T* out_body = out + part.head;
  const uint32_t v0 = chunk * kChunk + t;
  pdl_enter();  // before any global read: the previous kernel may still run
  uint4 raw[kUnroll];
#pragma unroll
  for (int j = 0; j < kUnroll; j++) {
    const uint32_t v = v0 + j * kThreads;
    if (v >= part.vecs) continue;
    if (SAME) {
      raw[j] = ld_stream(reinterpret_cast<const uint4*>(body) + v);
    } else {  // x lies otherwise against 16 bytes than the output does
      float f[N];
#pragma unroll
      for (int i = 0; i < N; i++) f[i] = widen(body[static_cast<int64_t>(v) * N + i]);
      raw[j] = Vec<T>::pack(f);
    }
  }
  uint32_t extra_at = 0xFFFFFFFFu;
  if (chunk == 0) {
    if (static_cast<uint32_t>(t) < part.head) extra_at = t;
    if (t >= 8 && static_cast<uint32_t>(t - 8) < part.tail)
      extra_at = a.vocab - part.tail + (t - 8);
  }
  const float extra = extra_at < a.vocab ? widen(x[extra_at]) : 0.0f;
  const int64_t token = a.tokens[row];
  const float lse = a.lse[row];
  const bool given = token >= 0 && token < a.vocab && a.dlogprob != nullptr;
  // a row of -inf alone has no probabilities: its gradient is 0
  const bool none = lse == -kInf;
  const float g = given && !none ? a.dlogprob[row] : 0.0f;
  const float h = a.dentropy != nullptr && !none ? a.dentropy[row] : 0.0f;
  const float ent = a.dentropy != nullptr ? a.entropy[row] : 0.0f;
  const float ca = -(g + h * ent) * a.inv_t, cb = -h * a.inv_t, own = g * a.inv_t;
  const float neg = none ? 0.0f : -lse;
  const GradRow grad{f2(a.inv_t, a.inv_t), f2(neg, neg), f2(ca, ca), f2(cb, cb)};
  const uint32_t tok = given ? static_cast<uint32_t>(token) : 0xFFFFFFFFu;
#pragma unroll
  for (int j = 0; j < kUnroll; j++) {
    const uint32_t v = v0 + j * kThreads;
    if (v >= part.vecs) continue;
    F2 f[N / 2];
    Pairs<T>::unpack(raw[j], f);
#pragma unroll
    for (int i = 0; i < N / 2; i++) f[i] = grad(f[i]);
    float u[N];
    from_pairs(f, u);
    const uint32_t at = part.head + v * N;
    if (tok - at < N) {
#pragma unroll
      for (int i = 0; i < N; i++)
        if (tok == at + i) u[i] += own;
    }
    st_stream(reinterpret_cast<uint4*>(out_body) + v, Vec<T>::pack(u));
  }
  if (extra_at < a.vocab) {
    float lo, hi;
    split(grad(f2(extra, extra)), lo, hi);
    if (extra_at == tok) lo += own;
    out[extra_at] = static_cast<T>(lo);
  }
}

template <typename T, bool TOP>
cudaError_t launch_rows(const LogprobArgs& a, int64_t rows, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * a.ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(a.ranks);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.ranks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, TOP>, a);
}

}  // namespace

cudaError_t launch_token_logprobs(float* logprob, float* entropy, float* lse, float* top_logprob,
                                  int64_t* top_ids, const void* logits, const int64_t* tokens,
                                  int64_t rows, int64_t vocab, int64_t stride, int top,
                                  float inv_t, int is_bf16, cudaStream_t stream) {
  LogprobArgs a = {logits, tokens, logprob, entropy, lse, top_logprob, top_ids, stride,
                   static_cast<uint32_t>(vocab), top, 1, inv_t};
  int device = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return e;
  // Few rows are split while blocks find room at once and keep half a chunk each.
  const int64_t vecs = vocab / (is_bf16 ? 8 : 4);
  while (a.ranks < 8 && rows * a.ranks * 2 <= 2 * sms && vecs >= a.ranks * kChunk) a.ranks *= 2;
  if (is_bf16)
    return top > 0 ? launch_rows<__nv_bfloat16, true>(a, rows, stream)
                   : launch_rows<__nv_bfloat16, false>(a, rows, stream);
  return top > 0 ? launch_rows<float, true>(a, rows, stream)
                 : launch_rows<float, false>(a, rows, stream);
}

cudaError_t launch_token_logprobs_backward(void* dlogits, const float* dlogprob,
                                           const float* dentropy, const void* logits,
                                           const int64_t* tokens, const float* lse,
                                           const float* entropy, int64_t rows, int64_t vocab,
                                           int64_t stride, int64_t out_stride, float inv_t,
                                           int is_bf16, cudaStream_t stream) {
  LogprobGradArgs a = {dlogits, dlogprob, dentropy, logits, tokens, lse, entropy, stride,
                       out_stride, static_cast<uint32_t>(vocab), 0, inv_t};
  const int64_t n = is_bf16 ? 8 : 4, es = is_bf16 ? 2 : 4;
  a.blocks = static_cast<uint32_t>((vocab / n + kChunk - 1) / kChunk);
  if (a.blocks == 0) a.blocks = 1;
  // every row of both at the same distance from a 16-byte boundary
  const bool same = ((reinterpret_cast<uintptr_t>(logits) ^ reinterpret_cast<uintptr_t>(dlogits)) &
                     15u) == 0 &&
                    (stride - out_stride) * es % 16 == 0;
  const dim3 grid(static_cast<unsigned>(rows * a.blocks));
  const dim3 block(kThreads);
  if (is_bf16)
    return same ? launch_pdl(token_logprobs_grad_kernel<__nv_bfloat16, true>, grid, block, 0,
                             stream, a)
                : launch_pdl(token_logprobs_grad_kernel<__nv_bfloat16, false>, grid, block, 0,
                             stream, a);
  return same ? launch_pdl(token_logprobs_grad_kernel<float, true>, grid, block, 0, stream, a)
              : launch_pdl(token_logprobs_grad_kernel<float, false>, grid, block, 0, stream, a);
}

}  // namespace nr
