// Attention over the quantised paged cache with many query rows an item: trees and chains of
// drafted tokens, prompts (sm_103a, tcgen05).  The arithmetic is cache_attention.cu's; a row's largest weight
// times V scale is held at 2^7.5 or more, so f16's end takes at most 2^-32 of it from another.
//
// A block owns an SM and up to 128 query rows of one K/V head, and walks its share's positions in
// tiles of 128.  Eight warps read the codes and write them as f16 into shared memory in
// the layout that the tensor core wants (K and V alike, rows of 128 bytes with the 128-byte
// swizzle); one thread issues the products; four warps do the softmax, a row a thread:
//     S = Q K^T    A and B from shared memory, S in tensor memory, two buffers
//     O += P V     A = P (f16) in tensor memory, beside the S it came from; B = V as it lies
//                  (the dimension runs fastest); O stays in tensor memory
// so that Q K^T of the next tile runs under the softmax of this one.  A row's references (its largest
// score, and its largest weight times V scale) move only when a tile's weights sum to more than 2^8 or
// one of them times its V scale leaves f16's range, 2^6.5 above what the largest is held at or more;
// then the warp multiplies its rows of O.  So a tile's weights are taken with the references that are
// there, and once more where these have to move (a pass of its own for the maximum in each tile took 131 us
// where one pass took 121).
//
// What bounds it: the products take 1076 cycles a tile (D = 128), the operands 160 KB of shared
// memory a tile (1250 cycles).  The softmax's warps are alone on their schedulers and wait for their own
// results most of the time: that is what a tile takes now, about twice the products.  Trees of up to 61
// tokens of 6 sequences with 60013 cached tokens, 32 query and 8 cache heads of 128 in FP8: 124 us, 467
// TFLOP/s (mma.sync, 16 rows an item: 790 us).
#include "attn_plan.cuh"
#include "nr_internal.h"

namespace nr {
namespace {

constexpr int kRows = 128;
constexpr int kPos = 128;  // positions a tile
constexpr int kSoftWarps = 4, kLoadWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kLoadWarps;
constexpr int kRowsThreads = (kMmaWarp + 1) * kWarp;
constexpr int kRowsShares = 152;   // one block an SM
constexpr int kPer = kPos / kLoadWarps;  // positions a loading warp
constexpr int kItemCost = 8;       // tiles that an item costs besides its own
constexpr int kMeta = 4;           // tiles whose scales are kept
constexpr int kItems = 8;          // items whose row scales are kept
constexpr float kMostSum = 256.0f;  // of a tile's weights, relative to the row's reference
constexpr int kHold = 9;            // what a row holds for f16 starts between 2^7.5 and 2^9.5,
constexpr float kMostHeld = 65504.0f;  // and may rise to f16's largest
constexpr long long kWaitCycles = 1ll << 31;
constexpr float kNone = -__builtin_huge_valf();

// --- tcgen05
__device__ __forceinline__ void tmem_alloc(unsigned dst, unsigned cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(unsigned at, unsigned cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Everything this thread has issued arrives on `bar` when it is done.
__device__ __forceinline__ void tc_commit(unsigned bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void mma_ss(unsigned d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<int>(add))
      : "memory");
}
__device__ __forceinline__ void mma_ts(unsigned d, unsigned a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<int>(add))
      : "memory");
}
// 32 columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_load(unsigned at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
      "[%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
// The loads' registers are there behind this; they pass through it so that no use moves in front.
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; i++) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_store32(unsigned at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
          at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_store16(unsigned at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_stored() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(unsigned bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A shared-memory operand in rows of 128 bytes with the 128-byte swizzle, eight rows 1024 bytes.
// `wide`: bytes between blocks of 64 elements of the fast axis, where that is not the axis
// summed over (V).
__device__ __forceinline__ uint64_t operand(unsigned at, unsigned wide) {
  return static_cast<uint64_t>((at >> 4) & 0x3FFFu) | static_cast<uint64_t>((wide >> 4) & 0x3FFFu) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// f16 operands, f32 sums, M = 128; `fast_n`: B's fast axis is N.
constexpr uint32_t product_of(int n, bool fast_n) {
  return 1u << 4 | (fast_n ? 1u << 16 : 0u) | static_cast<uint32_t>(n >> 3) << 17 | (128u >> 4) << 24;
}

template <bool FP4, int DIM>
struct RowsShared {
  static constexpr int kBlocks = DIM / 64;          // of 64 dimensions
  static constexpr int kBlockBytes = kPos * 128;    // (Q: kRows rows)
  static constexpr int kTileBytes = kBlocks * kBlockBytes;
  static constexpr int kGroups = FP4 ? DIM / 32 : 1;
  unsigned char q[kTileBytes];
  unsigned char k[2][kTileBytes];
  unsigned char v[2][kTileBytes];
  // barriers
  unsigned long long q_full, q_empty, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2],
      o_full[2], meta_full[kMeta], done;
  alignas(16) float ks[kMeta][kPos];
  alignas(16) float vs[kMeta][kPos];
  alignas(16) float vk[kMeta][kPos];  // exponents of V's scales
  alignas(16) uint16_t there[kMeta][kLoadWarps];       // positions that are in the cache
  alignas(16) unsigned char clean[kMeta][kLoadWarps];  // every position there, seen by every row
  float row_scale[kItems][kRows];
  int nan_lo[kItems], nan_hi[kItems];      // positions whose V holds a NaN that was left out
  alignas(16) int64_t at[kLoadWarps][2][kPer];
  uint16_t km[kLoadWarps][2][kPer][kGroups], vm[kLoadWarps][2][kPer][kGroups];
  unsigned tmem;
  int dead;
  AttnPlan<kRowsThreads> plan;
};

// A loading lane's codes of some positions: position n * kAtOnce + lane / kLanes of the warp's, 16
// bytes of its head from 16 * (lane % kLanes) on.
template <bool FP4, int DIM>
struct RowsLane {
  static constexpr int kLanes = (FP4 ? DIM / 2 : DIM) / 16;  // of a position
  static constexpr int kAtOnce = kWarp / kLanes;             // positions an instruction
  static constexpr int kLoads = kPer / kAtOnce;
  static constexpr int kChunks = FP4 ? 4 : 2;                // of 16 bytes that 16 bytes of codes widen to
  uint4 x[kLoads];

  __device__ __forceinline__ void load(const unsigned char* codes, const int64_t* at, int lane) {
#pragma unroll
    for (int n = 0; n < kLoads; n++) {
      const int64_t from = at[n * kAtOnce + lane / kLanes];
      x[n] = make_uint4(0u, 0u, 0u, 0u);
      if (from >= 0)
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x[n].x), "=r"(x[n].y), "=r"(x[n].z), "=r"(x[n].w)
                     : "l"(codes + from));
    }
  }

  // Widened into a tile, from its row row0 on.  TIDY: halves that are NaN become 0; bit n of the
  // result: the n-th position had one.
  template <bool TIDY>
  __device__ __forceinline__ uint32_t store(unsigned char* dst, const uint16_t* mult, int row0,
                                            int lane) const {
    using Sh = RowsShared<FP4, DIM>;
    const int lr = lane / kLanes, lc = lane % kLanes;
    uint32_t found = 0;
#pragma unroll
    for (int n = 0; n < kLoads; n++) {
      const int pos = n * kAtOnce + lr, row = row0 + pos;
      const uint32_t word[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
      uint4 half[kChunks];
      if constexpr (!FP4) {
#pragma unroll
        for (int e = 0; e < 2; e++)
          half[e] = make_uint4(half2_of_e4m3(word[2 * e]), half2_of_e4m3(word[2 * e] >> 16),
                               half2_of_e4m3(word[2 * e + 1]), half2_of_e4m3(word[2 * e + 1] >> 16));
      } else {
        const uint32_t f = mult[pos * Sh::kGroups + lc] * 0x10001u;
#pragma unroll
        for (int e = 0; e < 4; e++) {
          uint32_t h[4];
          half2_of_e2m1(word[e], h);
          half[e] =
              make_uint4(mul_half2(h[0], f), mul_half2(h[1], f), mul_half2(h[2], f), mul_half2(h[3], f));
        }
      }
      if (TIDY) {
        uint32_t any = 0;
#pragma unroll
        for (int e = 0; e < kChunks; e++)
          any |= tidy(half[e].x) | tidy(half[e].y) | tidy(half[e].z) | tidy(half[e].w);
        if (any) found |= 1u << n;
      }
      // Chunk c of 16 bytes of a row lies at c ^ (row % 8) of its block of 128 bytes.  The order in
      // which the lanes of a row write theirs keeps eight neighbouring lanes in different banks.
      const int turn = FP4 ? (DIM == 128 ? (lc >> 1) | (row & 1) << 1 : (row >> 1 & 1) | (row & 1) << 1)
                           : (DIM == 128 ? lc >> 2 : 0);
#pragma unroll
      for (int s = 0; s < kChunks; s++) {
        const int e = s ^ turn, c = lc * kChunks + e;
        uint4 h = half[0];
#pragma unroll
        for (int o = 1; o < kChunks; o++)
          if (e == o) h = half[o];
        *reinterpret_cast<uint4*>(dst + c / 8 * Sh::kBlockBytes + row * 128 + ((c % 8) ^ (row & 7)) * 16) = h;
      }
    }
    return found;
  }

  __device__ __forceinline__ static uint32_t tidy(uint32_t& h) {
    const uint32_t nan = ((h & 0x7FFFu) > 0x7C00u ? 0xFFFFu : 0u) |
                         ((h & 0x7FFF0000u) > 0x7C000000u ? 0xFFFF0000u : 0u);
    h &= ~nan;
    return nan;
  }
};

// One thread's row of a tile of scores, over the positions whose bits are set (ALL: every one): the
// largest score, and the largest sum of a score and the exponent of its V scale.
template <bool ALL>
__device__ __forceinline__ void rows_find(unsigned s_at, const float* ks, const float* vk,
                                          const uint32_t (&see)[4], float rs, float& mx, float& tx) {
  const F2 rs2 = f2(rs, rs);
  mx = tx = kNone;
  uint32_t x[32];
#pragma unroll 1
  for (int j = 0; j < 4; j++) {
    tmem_load(s_at + 32 * j, x);
    tmem_loaded(x);
    const float2* k2 = reinterpret_cast<const float2*>(ks + 32 * j);
    const float2* v2 = reinterpret_cast<const float2*>(vk + 32 * j);
    const uint32_t bits = j == 0 ? see[0] : j == 1 ? see[1] : j == 2 ? see[2] : see[3];
#pragma unroll
    for (int e = 0; e < 16; e++) {
      const float2 k = k2[e], v = v2[e];
      const bool s0 = ALL || (bits >> (2 * e) & 1u), s1 = ALL || (bits >> (2 * e + 1) & 1u);
      const F2 score = mul2(f2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])),
                            mul2(f2(k.x, k.y), rs2));
      float u[2];
      split(score, u[0], u[1]);
      mx = fmaxf(mx, fmaxf(s0 ? u[0] : kNone, s1 ? u[1] : kNone));
      split(add2(score, f2(v.x, v.y)), u[0], u[1]);
      tx = fmaxf(tx, fmaxf(s0 ? u[0] : kNone, s1 ? u[1] : kNone));
    }
  }
}

// The same row's weights e^(score - m), summed; times `up` and V's scales as f16 to p_at.  `most`: the
// largest magnitude of these.
template <bool ALL>
__device__ __forceinline__ float rows_weigh(unsigned s_at, unsigned p_at, const float* ks,
                                            const float* vs, const uint32_t (&see)[4], float rs,
                                            float neg, float up, float& most) {
  const F2 rs2 = f2(rs, rs), neg2 = f2(neg, neg), up2 = f2(up, up);
  F2 l2 = f2(0.0f, 0.0f);
  most = 0.0f;
  uint32_t x[32];
#pragma unroll 1
  for (int j = 0; j < 4; j++) {
    tmem_load(s_at + 32 * j, x);
    tmem_loaded(x);
    const float4* k4 = reinterpret_cast<const float4*>(ks + 32 * j);
    const float4* v4 = reinterpret_cast<const float4*>(vs + 32 * j);
    const uint32_t bits = j == 0 ? see[0] : j == 1 ? see[1] : j == 2 ? see[2] : see[3];
    uint32_t p[16];
#pragma unroll
    for (int e = 0; e < 16; e++) {
      const float4 k = k4[e / 2], v = v4[e / 2];
      const F2 kk = e % 2 ? f2(k.z, k.w) : f2(k.x, k.y);
      const F2 vv = e % 2 ? f2(v.z, v.w) : f2(v.x, v.y);
      const bool s0 = ALL || (bits >> (2 * e) & 1u), s1 = ALL || (bits >> (2 * e + 1) & 1u);
      float u[2];  // (the products with Q first times K's scale could leave f32's range)
      split(fma2(f2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), mul2(kk, rs2), neg2), u[0],
            u[1]);
      u[0] = attn_exp2(u[0]);
      u[1] = attn_exp2(u[1]);
      if (!s0) u[0] = 0.0f;
      if (!s1) u[1] = 0.0f;
      const F2 weight = f2(u[0], u[1]);
      l2 = add2(l2, weight);
      split(mul2(mul2(weight, up2), vv), u[0], u[1]);  // (a scale times `up` may be infinite)
      if (!s0) u[0] = 0.0f;  // whatever its scale
      if (!s1) u[1] = 0.0f;
      most = fmaxf(most, fmaxf(fabsf(u[0]), fabsf(u[1])));
      p[e] = half2_of(u[0], u[1]);
    }
    tmem_store16(p_at + 16 * j, p);
  }
  tmem_stored();  // the next stores may go to the same columns, and nothing orders two but this
  float lo, hi;
  split(l2, lo, hi);
  return lo + hi;
}

// Waits for the phase; once a wait has run out, no further one waits: every role runs through its
// loop, the outputs are not valid, and the status word says so.
struct Waiter {
  int* dead;
  unsigned* status;
  __device__ __forceinline__ void operator()(unsigned bar, unsigned parity) const {
    if (mbar_test_wait(bar, parity)) return;
    const long long t0 = clock64();
    for (;;) {
      __nanosleep(20);
      if (mbar_test_wait(bar, parity)) return;
      if (*static_cast<volatile int*>(dead)) return;
      if (clock64() - t0 > kWaitCycles) {
        *static_cast<volatile int*>(dead) = 1;
        atomicOr(status, kStatusBitAttnWait);
        return;
      }
    }
  }
};

// A walk through a share: its items, and how many tiles of each.
struct Walk {
  int64_t unit, end;
  AttnItem it;
};

template <bool FP4, int DIM>
__global__ void __launch_bounds__(kRowsThreads, 1)
    cache_attention_rows_kernel(const AttnArgs a, unsigned* status) {
  using T = __nv_bfloat16;
  using Sh = RowsShared<FP4, DIM>;
  constexpr int kCodeRow = FP4 ? DIM / 2 : DIM;  // bytes of a head
  constexpr unsigned kCols = 512;                // S twice 128, O 128, the weights twice 64
  extern __shared__ __align__(16) unsigned char smem_raw[];
  // the swizzle goes by address: operands start at multiples of 1024
  auto& sh = *reinterpret_cast<Sh*>(
      smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  const int t = threadIdx.x, warp = t / kWarp, lane = t % kWarp;

  if (t == 0) {
    auto init = [](unsigned long long& b, unsigned n) { mbar_init(smem_addr(&b), n); };
    init(sh.q_full, kLoadWarps);
    init(sh.q_empty, 1);
    for (int i = 0; i < 2; i++) {
      init(sh.k_full[i], kLoadWarps);
      init(sh.k_empty[i], 1);
      init(sh.v_full[i], kLoadWarps);
      init(sh.v_empty[i], 1);
      init(sh.s_full[i], 1);
      init(sh.p_full[i], kSoftWarps * kWarp);
      init(sh.o_full[i], 1);
    }
    for (int i = 0; i < kMeta; i++) init(sh.meta_full[i], kLoadWarps);
    init(sh.done, 1);
    fence_mbar_init();
    sh.dead = 0;
    for (int i = 0; i < kItems; i++) sh.nan_lo[i] = 0x7FFFFFFF, sh.nan_hi[i] = -1;
  }
  if (warp == kMmaWarp) tmem_alloc(smem_addr(&sh.tmem), kCols);
  pdl_enter();  // before any global read: the previous kernel may still run
  make_plan<kRows, kPos, kItemCost>(a, sh.plan);  // (its barriers make the above visible)
  tc_before();
  __syncthreads();
  tc_after();
  const unsigned tmem = *static_cast<volatile unsigned*>(&sh.tmem);
  const int64_t total = sh.plan.at[kRowsThreads];
  const int64_t share = share_size(total, gridDim.x);
  Walk w;
  w.unit = blockIdx.x * share;
  w.end = min(w.unit + share, total);
  if (t == 0) a.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
  const Waiter wait{&sh.dead, status};

  if (w.unit < w.end) {
    w.it = locate<kRows, kPos, kItemCost>(a, sh.plan, w.unit);
    int64_t tile = 0;  // of this block, over all its items
    int item = 0;
    while (w.unit < w.end) {
      const AttnSeq<kPos> seq(a, w.it.seq);
      const int rows = min(seq.queries * static_cast<int>(a.group.div) - w.it.rb * kRows, kRows);
      const int steps = static_cast<int>(min(static_cast<int64_t>(seq.tiles - w.it.tile), w.end - w.unit));
      const bool from_start = w.it.tile == 0, to_end = w.it.tile + steps == seq.tiles;

      if (warp < kSoftWarps) {
        // ------------------------------------------------------------ softmax
        const int r = t;  // row of the block, lane of tensor memory
        const unsigned mine = tmem + (static_cast<unsigned>(warp * kWarp) << 16);
        const bool busy = warp * kWarp < rows;
        const int row = w.it.rb * kRows + r;
        const int tok = a.group.quot(row);
        float m = kNone, vm = kNone, l = 0.0f, rs = 0.0f;  // (vm: as hold_factor's t)
        for (int i = 0; i < steps; i++) {
          const int64_t g = tile + i;
          const int b = g & 1;
          const unsigned s_at = mine + b * kPos;
          wait(smem_addr(&sh.meta_full[g % kMeta]), (g / kMeta) & 1);
          wait(smem_addr(&sh.s_full[b]), (g >> 1) & 1);
          // (a phase that is not waited for in its turn could be taken for the one behind it)
          if (g >= 2) wait(smem_addr(&sh.o_full[b]), ((g >> 1) - 1) & 1);
          __syncwarp();
          tc_after();
          if (busy) {
            if (i == 0) rs = sh.row_scale[item % kItems][r];
            const float* ks = sh.ks[g % kMeta];
            const float* vs = sh.vs[g % kMeta];
            const bool clean = *reinterpret_cast<const volatile uint64_t*>(sh.clean[g % kMeta]) ==
                               0x0101010101010101ull;
            uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
            if (!clean) {
              const int p0 = (w.it.tile + i) * kPos;
#pragma unroll
              for (int j = 0; j < 4; j++) {
                uint32_t bits = 0;
                const uint32_t there = *reinterpret_cast<const uint32_t*>(&sh.there[g % kMeta][2 * j]);
                if (r < rows) {
                  const int first = p0 + 32 * j - seq.context;  // of the word's first position
                  if (first <= -32) {
                    bits = ~0u;
                  } else if (a.tree == nullptr) {
                    const int n = tok - first + 1;
                    bits = n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
                  } else {  // the context in front of the words is seen
                    auto word = [&](int i) {
                      if (i < 0) return ~0u;
                      return i < a.words
                                 ? a.tree[static_cast<int64_t>(seq.first + tok) * a.words + i]
                                 : 0u;
                    };
                    bits = __funnelshift_r(word(first >> 5), word((first >> 5) + 1), first & 31);
                  }
                  bits &= there;
                }
                see[j] = bits;
              }
            }
            __syncwarp();
            // With the references that the row has, and once more where they have to move: at an item's
            // first tile, where there are none, at once; seldom after it.
            float lt;
            bool need = i == 0;
#pragma unroll 1
            for (int turn = i == 0 ? 1 : 0;; turn++) {
              if (turn == 1) {
                float mx, tx, f = 1.0f;
                if (clean)
                  rows_find<true>(s_at, ks, sh.vk[g % kMeta], see, rs, mx, tx);
                else
                  rows_find<false>(s_at, ks, sh.vk[g % kMeta], see, rs, mx, tx);
                if (need) {
                  const float to = fmaxf(m, mx), vto = fmaxf(vm, tx);
                  const float fl = m == kNone ? 0.0f : attn_exp2(m - to);
                  l *= fl;
                  f = fl * hold_factor<kHold>(vto, to) * power_reciprocal(hold_factor<kHold>(vm, m));
                  m = to;
                  vm = vto;
                }
                __syncwarp();
                if (i > 0) {  // the row of O moves with them
                  wait(smem_addr(&sh.o_full[b ^ 1]), ((g - 1) >> 1) & 1);
                  __syncwarp();
                  tc_after();
                  uint32_t x[32];
#pragma unroll 1
                  for (int j = 0; j < DIM / 32; j++) {
                    tmem_load(mine + 2 * kPos + 32 * j, x);
                    tmem_loaded(x);
#pragma unroll
                    for (int e = 0; e < 32; e++) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                    tmem_store32(mine + 2 * kPos + 32 * j, x);
                  }
                  tmem_stored();
                }
              }
              const float neg = m == kNone ? 0.0f : -m;
              const float up = hold_factor<kHold>(vm, m);
              const unsigned p_at = mine + 3 * kPos + b * (kPos / 2);
              float most;
              lt = clean ? rows_weigh<true>(s_at, p_at, ks, vs, see, rs, neg, up, most)
                         : rows_weigh<false>(s_at, p_at, ks, vs, see, rs, neg, up, most);
              // (a sum above 2^8 has a weight above 2: the reference moves)
              need = lt > kMostSum || most > kMostHeld ||
                     (m == kNone && (see[0] | see[1] | see[2] | see[3]) != 0u);
              if (turn == 1 || !__any_sync(0xFFFFFFFFu, need)) break;
            }
            l += lt;
          }
          tc_before();
          mbar_arrive(smem_addr(&sh.p_full[b]));
        }
        // the item's result
        const int64_t last = tile + steps - 1;
        wait(smem_addr(&sh.o_full[last & 1]), (last >> 1) & 1);
        __syncwarp();
        tc_after();
        if (busy) {
          const int lo = *static_cast<volatile int*>(&sh.nan_lo[item % kItems]);
          const int hi = *static_cast<volatile int*>(&sh.nan_hi[item % kItems]);
          const float back = power_reciprocal(hold_factor<kHold>(vm, m));
          const bool whole = from_start && to_end;
          const float scale = whole ? (l != 0.0f ? __fdiv_rn(back, l) : 0.0f) : back;
          const int64_t head = static_cast<int64_t>(seq.first + tok) * a.heads * a.group.div +
                               w.it.head * a.group.div + (row - tok * a.group.div);
          float* part = a.partial +
                        (2 * static_cast<int64_t>(blockIdx.x) + (from_start ? 1 : 0)) * kRows * (DIM + 2);
          T* out = static_cast<T*>(a.out) + head * DIM;
          uint32_t x[32];
#pragma unroll 1
          for (int j = 0; j < DIM / 32; j++) {
            tmem_load(mine + 2 * kPos + 32 * j, x);
            tmem_loaded(x);
            if (r < rows && whole) {
#pragma unroll
              for (int e = 0; e < 4; e++) {
                float f[8];
#pragma unroll
                for (int h = 0; h < 8; h++) f[h] = __uint_as_float(x[8 * e + h]) * scale;
                *reinterpret_cast<uint4*>(out + 32 * j + 8 * e) = Vec<T>::pack(f);
              }
            } else if (r < rows) {
#pragma unroll
              for (int e = 0; e < 8; e++) {
                const float4 f = make_float4(
                    __uint_as_float(x[4 * e]) * scale, __uint_as_float(x[4 * e + 1]) * scale,
                    __uint_as_float(x[4 * e + 2]) * scale, __uint_as_float(x[4 * e + 3]) * scale);
                *reinterpret_cast<float4*>(part + r * DIM + 32 * j + 4 * e) = f;
              }
            }
            __syncwarp();
          }
          if (r < rows) {
            if (whole) {
              if (a.lse != nullptr) a.lse[head] = l != 0.0f ? (m + log2f(l)) * kAttnLn2 : kNone;
            } else {
              part[kRows * DIM + 2 * r] = m;
              part[kRows * DIM + 2 * r + 1] = l;
            }
            // V's NaN, left out of the products (0 times one is one): they reach the rows that see
            // their position
            for (int p = lo; p <= hi; p++) {
              if (p >= seq.length || !attn_sees(a, seq, tok, p)) continue;
              const int64_t page = a.page.quot(p);
              const int blk = page < a.width ? a.table[w.it.seq * a.width + page] : -1;
              if (blk < 0 || blk >= a.blocks) continue;
              const int64_t in = p - page * a.page.div;
              const unsigned char* code = a.side[1].codes + blk * a.geo.code_block_stride +
                                          in * a.geo.code_row + w.it.head * kCodeRow;
              const unsigned char* sc = a.side[1].scales + blk * a.geo.scale_block_stride +
                                        in * a.geo.scale_row + w.it.head * (DIM / 32);
              for (int d = 0; d < DIM; d++) {
                if (FP4 ? sc[d / 32] != 255 : (code[d] & 0x7F) != 0x7F) continue;
                if (whole)
                  out[d] = narrow<T>(__uint_as_float(0x7FC00000u));
                else
                  part[r * DIM + d] = __uint_as_float(0x7FC00000u);
              }
            }
          }
        }
        __syncwarp();
        if (t == 0) {
          if (from_start && !to_end) {
            const int64_t item_end = w.unit + seq.tiles;
            a.joins[blockIdx.x] = make_int4(w.it.seq, w.it.head, w.it.rb,
                                            static_cast<int>((item_end - 1) / share - blockIdx.x + 1));
          }
          // the place of an item that nobody loads yet
          sh.nan_lo[(item + 4) % kItems] = 0x7FFFFFFF;
          sh.nan_hi[(item + 4) % kItems] = -1;
        }
        __syncwarp();
        tc_before();
      } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------ loading
        const int lw = warp - kSoftWarps;
        RowsLane<FP4, DIM> k, v;
        const int64_t from = w.it.head * kCodeRow + 16 * (lane % k.kLanes);
        const unsigned char* kc = a.side[0].codes + from;
        const unsigned char* vc = a.side[1].codes + from;
        const int base0 = w.it.tile * kPos + lw * kPer;
        auto lookup = [&](int i) {
          // what the table says, looked at a step later: a comparison here would wait for it
          const int p = base0 + i * kPos + lane;
          if (lane >= kPer || i >= steps || p >= seq.length) return -1;
          const int64_t page = a.page.quot(p);
          return page < a.width ? a.table[w.it.seq * a.width + page] : -1;
        };
        float ks = 0.0f, vs = 0.0f;
        uint64_t kb = 0, vb = 0;
        // offsets of step i, its scales on their way
        auto place = [&](int i, int blk) {
          if (lane >= kPer) return;
          const int p = base0 + i * kPos + lane;
          int64_t at = -1;
          ks = vs = 0.0f;
          kb = vb = 0;
          if (blk >= 0 && blk < a.blocks) {
            const int64_t in = p - static_cast<int64_t>(a.page.quot(p)) * a.page.div;
            at = blk * a.geo.code_block_stride + in * a.geo.code_row;
            const int64_t sc = blk * a.geo.scale_block_stride + in * a.geo.scale_row;
            if constexpr (!FP4) {
              ks = reinterpret_cast<const float*>(a.side[0].scales + sc)[w.it.head];
              vs = reinterpret_cast<const float*>(a.side[1].scales + sc)[w.it.head];
            } else {
              const unsigned char* pk = a.side[0].scales + sc + w.it.head * Sh::kGroups;
              const unsigned char* pv = a.side[1].scales + sc + w.it.head * Sh::kGroups;
              if (a.wide_scales) {
                if constexpr (Sh::kGroups == 2)
                  kb = *reinterpret_cast<const uint16_t*>(pk), vb = *reinterpret_cast<const uint16_t*>(pv);
                else
                  kb = *reinterpret_cast<const uint32_t*>(pk), vb = *reinterpret_cast<const uint32_t*>(pv);
              } else {
#pragma unroll
                for (int e = 0; e < Sh::kGroups; e++) {
                  kb |= static_cast<uint64_t>(pk[e]) << (8 * e);
                  vb |= static_cast<uint64_t>(pv[e]) << (8 * e);
                }
              }
            }
          }
          sh.at[lw][i & 1][lane] = at;
        };
        int blk = lookup(0);
        place(0, blk);
        blk = lookup(1);
        __syncwarp();
        k.load(kc, sh.at[lw][0], lane);
        v.load(vc, sh.at[lw][0], lane);

        // Q: two threads a row
        if (item > 0) wait(smem_addr(&sh.q_empty), (item - 1) & 1);
        {
          const int lt = t - kSoftWarps * kWarp, r = lt / 2, part = lt % 2;
          constexpr int N = DIM / 16;  // vectors a thread
          const int row = w.it.rb * kRows + r;
          const int tok = a.group.quot(row), head = w.it.head * a.group.div + (row - tok * a.group.div);
          const T* p = static_cast<const T*>(a.q) + (seq.first + tok) * a.q_stride +
                       static_cast<int64_t>(head) * DIM + part * (DIM / 2);
          uint4 raw[N];
          float top = 0.0f;
#pragma unroll
          for (int n = 0; n < N; n++) {
            raw[n] = r < rows ? ld_param(p + 8 * n) : make_uint4(0u, 0u, 0u, 0u);
            float f[8];
            Vec<T>::unpack(raw[n], f);
            top = fmaxf(top, max_abs(f));
          }
          top = group_max<2>(top);
          // as in cache_attention.cu; a negative scale of the scores turns Q's sign
          const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 27), 254) - 127;
          const float up = copysignf(__uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23), a.scale_log2);
          if (part == 0)
            sh.row_scale[item % kItems][r] =
                fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
#pragma unroll
          for (int n = 0; n < N; n++) {
            float f[8];
            Vec<T>::unpack(raw[n], f);
            const int c = part * N + n;
            *reinterpret_cast<uint4*>(sh.q + c / 8 * Sh::kBlockBytes + r * 128 + ((c % 8) ^ (r & 7)) * 16) =
                make_uint4(half2_of(f[0] * up, f[1] * up), half2_of(f[2] * up, f[3] * up),
                           half2_of(f[4] * up, f[5] * up), half2_of(f[6] * up, f[7] * up));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.q_full));
        }

        for (int i = 0; i < steps; i++) {
          const int64_t g = tile + i;
          const int b = g & 1;
          const int p0 = base0 + i * kPos;
          // the step's scales
          bool clean;
          {
            const bool in = lane < kPer && sh.at[lw][i & 1][lane % kPer] >= 0;
            if (FP4 && lane < kPer) {
              uint16_t m[Sh::kGroups];
              ks = mx_multipliers(kb, m);
#pragma unroll
              for (int e = 0; e < Sh::kGroups; e++) sh.km[lw][i & 1][lane][e] = m[e];
              vs = mx_multipliers(vb, m);
#pragma unroll
              for (int e = 0; e < Sh::kGroups; e++) sh.vm[lw][i & 1][lane][e] = m[e];
            }
            clean = __all_sync(0xFFFFFFFFu, lane >= kPer || (in && p0 + lane < seq.context));
            const unsigned there = __ballot_sync(0xFFFFFFFFu, in);
            if (lane < kPer) {
              sh.ks[g % kMeta][lw * kPer + lane] = ks;
              sh.vs[g % kMeta][lw * kPer + lane] = vs;
              sh.vk[g % kMeta][lw * kPer + lane] = scale_exponent(vs);
            }
            if (lane == 0) {
              sh.there[g % kMeta][lw] = static_cast<uint16_t>(there);
              sh.clean[g % kMeta][lw] = clean ? 1 : 0;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.meta_full[g % kMeta]));
          }
          const bool more = i + 1 < steps;
          if (more) {
            place(i + 1, blk);
            blk = lookup(i + 2);
            __syncwarp();
          }
          if (g >= 2) wait(smem_addr(&sh.k_empty[b]), ((g >> 1) - 1) & 1);
          k.template store<false>(sh.k[b], &sh.km[lw][i & 1][0][0], lw * kPer, lane);
          if (more) k.load(kc, sh.at[lw][(i + 1) & 1], lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.k_full[b]));
          if (g >= 2) wait(smem_addr(&sh.v_empty[b]), ((g >> 1) - 1) & 1);
          if (clean) {
            v.template store<false>(sh.v[b], &sh.vm[lw][i & 1][0][0], lw * kPer, lane);
          } else {
            uint32_t found = v.template store<true>(sh.v[b], &sh.vm[lw][i & 1][0][0], lw * kPer, lane);
            for (; found != 0; found &= found - 1) {
              const int pos = p0 + (__ffs(found) - 1) * v.kAtOnce + lane / v.kLanes;
              atomicMin(&sh.nan_lo[item % kItems], pos);
              atomicMax(&sh.nan_hi[item % kItems], pos);
            }
          }
          if (more) v.load(vc, sh.at[lw][(i + 1) & 1], lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.v_full[b]));
        }
      } else if (lane == 0) {
        // ------------------------------------------------------------ products
        const uint64_t q = operand(smem_addr(sh.q), 16);
        auto scores = [&](int i) {
          const int64_t g = tile + i;
          const int b = g & 1;
          wait(smem_addr(&sh.k_full[b]), (g >> 1) & 1);
          // S goes where the weights of two tiles ago were read from
          if (g >= 2) wait(smem_addr(&sh.o_full[b]), ((g >> 1) - 1) & 1);
          tc_after();
          const uint64_t k = operand(smem_addr(sh.k[b]), 16);
#pragma unroll
          for (int s = 0; s < DIM / 16; s++) {
            const uint64_t step = (s / 4 * Sh::kBlockBytes + s % 4 * 32) >> 4;
            mma_ss(tmem + b * kPos, q + step, k + step, product_of(kPos, false), s > 0);
          }
          tc_commit(smem_addr(&sh.s_full[b]));
          tc_commit(smem_addr(&sh.k_empty[b]));
          if (i + 1 == steps) tc_commit(smem_addr(&sh.q_empty));
        };
        wait(smem_addr(&sh.q_full), item & 1);
        scores(0);
        for (int i = 0; i < steps; i++) {
          const int64_t g = tile + i;
          const int b = g & 1;
          if (i + 1 < steps) scores(i + 1);
          wait(smem_addr(&sh.v_full[b]), (g >> 1) & 1);
          wait(smem_addr(&sh.p_full[b]), (g >> 1) & 1);
          tc_after();
          const uint64_t v = operand(smem_addr(sh.v[b]), Sh::kBlockBytes);
#pragma unroll
          for (int s = 0; s < kPos / 16; s++)
            mma_ts(tmem + 2 * kPos, tmem + 3 * kPos + b * (kPos / 2) + s * 8, v + (s * 2048 >> 4), product_of(DIM, true),
                   i > 0 || s > 0);
          tc_commit(smem_addr(&sh.v_empty[b]));
          tc_commit(smem_addr(&sh.o_full[b]));
        }
      }

      w.unit += steps + kItemCost;
      tile += steps;
      item++;
      if (w.unit < w.end) next_item<kRows, kPos>(a, w.it, seq.queries);
    }
    if (warp == kMmaWarp && lane == 0) {
      // nothing may be in flight when the tensor memory goes
      tc_commit(smem_addr(&sh.done));
      const long long t0 = clock64();
      while (!mbar_test_wait(smem_addr(&sh.done), 0) && clock64() - t0 <= kWaitCycles) {
      }
    }
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == kMmaWarp) tmem_free(tmem, kCols);
}

template <bool FP4, int DIM>
cudaError_t rows_go(AttnArgs a, void* workspace, cudaStream_t s) {
  constexpr size_t shared = sizeof(RowsShared<FP4, DIM>) + 1024;
  constexpr int percent = 86;  // 196 of 228 KB: the rest is L1, for what the registers do not hold
  static_assert(shared <= 195 * 1024, "one block an SM");
  static std::atomic<int> done[64], done_join[64];
  unsigned* status = nullptr;
  cudaError_t e = status_word(&status);
  if (e == cudaSuccess) e = allow_shared(cache_attention_rows_kernel<FP4, DIM>, shared, done, percent);
  if (e == cudaSuccess)
    e = allow_shared(cache_attention_join_kernel<__nv_bfloat16, kRows, DIM, FP4>, 0, done_join, percent);
  if (e != cudaSuccess) return e;
  a.joins = static_cast<int4*>(workspace);
  a.partial = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) +
                                       attn_joins_bytes(kRowsShares));
  e = launch_pdl(cache_attention_rows_kernel<FP4, DIM>, dim3(kRowsShares), dim3(kRowsThreads), shared, s,
                 a, status);
  if (e != cudaSuccess) return e;
  return launch_pdl(cache_attention_join_kernel<__nv_bfloat16, kRows, DIM, FP4>,
                    dim3(kRowsShares, kRows / kJoinRows), dim3(DIM / 4, kJoinRows), 0, s, a);
}

}  // namespace

int64_t attn_rows_bytes(int64_t head_dim) {
  return head_dim <= 128 ? attn_bytes(kRowsShares, kRows, head_dim) : 0;
}

cudaError_t launch_attn_rows(const AttnArgs& a, bool fp4, int64_t head_dim, void* workspace,
                             cudaStream_t stream) {
  if (head_dim == 64)
    return fp4 ? rows_go<true, 64>(a, workspace, stream) : rows_go<false, 64>(a, workspace, stream);
  return fp4 ? rows_go<true, 128>(a, workspace, stream) : rows_go<false, 128>(a, workspace, stream);
}

}  // namespace nr
