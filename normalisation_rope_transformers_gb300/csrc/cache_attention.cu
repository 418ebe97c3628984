// Attention over the quantised paged cache (sm_103a): one token, a chain or a tree of drafted
// tokens of each sequence against everything cached for it.
//
// Scores, weights and sums are f32, one pass over K and V with the running maximum and sum of
// the softmax.  Codes become f16 exactly (e4m3 has 4 significant bits, e2m1 2), and each row of
// Q is brought to f16's range by a power of two, so products of Q and K are exact and summed in
// f32.  A token's K scale multiplies its scores, its V scale its weights.  MXFP4 has a scale for
// 32 elements: relative to the token's largest they are powers of two that f16 holds down to
// 2^-37 of it; what is smaller counts as zero.  Weights times V's scales are rounded to f16 (11 bits), the
// one rounding that is not f32's: it is eight times finer than the bf16 output's.  A row's largest of them
// is held at 2^9.5 or more, whatever the weight or the scale alone, so f16's end takes at most 2^-34 of it from
// another.  With f32 tensors Q and these products are two f16 parts each (22 bits).
//
// Few queries a sequence: each code read once for 8, 16 or 24 query rows.  A warp reads 16 or 32
// positions' codes straight into the registers where mma.sync wants them (positions and dimensions
// are the rows of its first operand, query rows the columns of its second): which dimensions a
// lane's vector holds is free as long as Q (and the output's order) agree.  K of the next positions is
// on its way during softmax and the second product, V during the first.  A row's reference follows its
// maximum only when that is 2^4 above, so most steps reduce nothing across lanes.  Every share of
// the positions is as long: shares that end inside a sequence leave parts that a second kernel joins.
//
// Measured: one token of 48 sequences with 400009 cached tokens, 32 query and 8 cache heads of 128 in
// FP8: 152 us, 0.82 of the copy rate, bound by what 12 warps an SM have under way (168 registers).
// Up to 5 tokens of 29 sequences with 150001, 24 and 6 heads, MXFP4: 89 us, 0.20 of it, bound by
// instructions (52% of the issue slots; widening a code costs as much as FP8's twice as many bytes).
// One sequence of 1501 tokens: 10.7 us, latency: two launches, a plan, one step, joining.
#include <type_traits>

#include "attn_plan.cuh"
#include "nr_internal.h"

namespace nr {
namespace {

// NT: tiles of eight query rows an item has.  A warp's step is 16 SUB positions: 32 where a lane's
// codes of them fit in the registers beside O.  (One token, heads of 128 in FP8, 400009 positions in
// 48 sequences: 16 at a time, four blocks an SM 188 us, 32 at a time, three 159 us.)
template <bool FP4, int DIM, int NT>
constexpr int kSub = DIM == 256 || (NT == 3 && DIM == 128 && !FP4) ? 1 : 2;
// A share for each block that fits at once on 152 SMs (any number is right).
// (32 query and 8 cache heads of 64, one token, 300009 positions in 48 sequences: four blocks an SM instead
// of three 97 -> 96 us in FP8, 93 -> 85 in MXFP4; heads of 128 in MXFP4 124 with four, 122 with three.)
template <int DIM, int NT>
constexpr int attn_blocks = DIM == 256 || NT > 1 ? 2 : DIM == 64 ? 4 : 3;
constexpr int kSms = 152;

constexpr int kAttnThreads = 128;
constexpr int kAttnWarps = kAttnThreads / kWarp;
constexpr int kItemCost = 3;  // tiles that an item costs besides its own
constexpr float kSlack = 4.0f;  // a row's reference is behind its maximum by up to 2^4,
constexpr int kHold = 11;       // and what it holds for f16 starts between 2^9.5 and 2^11.5, up to 2^15.5

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// The fragment of an 8 x 8 matrix of halves turned into the fragment of its transpose.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// N bytes (4, 8 or a multiple of 16) from global memory, or zeros.
template <int N>
struct Words {
  uint32_t w[N / 4];
  __device__ __forceinline__ void load(const unsigned char* p, int64_t step, bool in) {
    if constexpr (N >= 16) {
#pragma unroll
      for (int i = 0; i < N / 16; i++) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        // no wider prefetch into L2: the neighbouring head's codes are another block's
        if (in)
          asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "l"(p + i * step));
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else if constexpr (N == 8) {
      uint2 v = make_uint2(0u, 0u);
      if (in)
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = 0u;
      if (in) asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
    }
  }
};

// Which dimensions a lane's codes hold.
template <bool FP4, int DIM>
struct Layout {
  static constexpr int kPieceK = FP4 && DIM >= 128 ? 32 : 16;  // dimensions a vector of K
  static constexpr int kBytesK = FP4 ? DIM / 8 : DIM / 4;      // a lane and position
  static constexpr int kBytesV = FP4 ? DIM / 16 : DIM / 8;
  static constexpr int kStepsK = DIM / 16;
  static constexpr int kTilesV = DIM / 8;
  static constexpr int kGroups = DIM / 32;
  static constexpr int kCodeRow = FP4 ? DIM / 2 : DIM;  // bytes of a head
  // lane c (of 4) of product step k has dimensions k_dim .. k_dim + 3
  __host__ __device__ static constexpr int k_dim(int c, int k) {
    constexpr int n = kPieceK / 4;
    return k / n * 4 * kPieceK + kPieceK * c + 4 * (k % n);
  }
  // column g (of 8) of output tile j is dimension v_dim
  static constexpr int kPieceV = FP4 ? DIM / 8 : (DIM >= 128 ? 16 : 8);
  __host__ __device__ static constexpr int v_dim(int g, int j) {
    return j / kPieceV * 8 * kPieceV + kPieceV * g + j % kPieceV;
  }
  // Where shared memory holds dimension v_dim(g, j) of a row of O: lanes g side by side, rows two
  // apart eight banks apart, and so that 32 lanes with 4 dimensions each read different banks.
  static constexpr int kPitchO = DIM / 4 * 5 + 4;
  __host__ __device__ static constexpr int o_at(int g, int j) { return 8 * j + 8 * (j / 4) + g; }
  __device__ static int o_first(int d) {  // of dimension d, a multiple of 4; the next three 8 further each
    return o_at(d % (8 * kPieceV) / kPieceV, d / (8 * kPieceV) * kPieceV + d % kPieceV);
  }
};

template <typename T, bool FP4, int DIM, int NT, int STEP>
struct AttnShared {
  static constexpr int SPLIT = sizeof(T) == 4 ? 2 : 1;
  using L = Layout<FP4, DIM>;
  static constexpr int ROWS = 8 * NT;
  union {
    uint2 q[SPLIT][NT][L::kStepsK][kWarp];  // fragments
    alignas(16) float o[kAttnWarps][ROWS][L::kPitchO];  // when Q is done with
  };
  alignas(16) float row_scale[ROWS];
  alignas(16) int64_t at[kAttnWarps][2][STEP];        // code offsets, -1: no such position
  float ks[kAttnWarps][STEP];             // scales of K, of V
  float vs[kAttnWarps][STEP];
  uint16_t km[kAttnWarps][STEP][FP4 ? L::kGroups : 1];
  uint16_t vm[kAttnWarps][STEP][FP4 ? L::kGroups : 1];
  float m[kAttnWarps][ROWS], l[kAttnWarps][ROWS];
  float top[ROWS], sum[ROWS];
  AttnPlan<kAttnThreads> plan;
};

template <typename T, bool FP4, int DIM, int NT>
__global__ void __launch_bounds__(kAttnThreads, (attn_blocks<DIM, NT>))
    cache_attention_kernel(const AttnArgs a) {
  using L = Layout<FP4, DIM>;
  constexpr int SPLIT = sizeof(T) == 4 ? 2 : 1, SUB = kSub<FP4, DIM, NT>, ROWS = 8 * NT;
  constexpr int kStep = 16 * SUB, kAttnTile = kStep * kAttnWarps;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  auto& sh = *reinterpret_cast<AttnShared<T, FP4, DIM, NT, kStep>*>(smem_raw);
  const int t = threadIdx.x, warp = t / kWarp, lane = t % kWarp, g = lane / 4, c = lane % 4;
  pdl_enter();  // before any global read: the previous kernel may still run
  make_plan<ROWS, kAttnTile, kItemCost>(a, sh.plan);
  const int64_t total = sh.plan.at[kAttnThreads];
  const int64_t share = share_size(total, gridDim.x);
  int64_t unit = blockIdx.x * share;
  const int64_t end = min(unit + share, total);
  if (t == 0) a.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (unit >= end) return;
  AttnItem it = locate<ROWS, kAttnTile, kItemCost>(a, sh.plan, unit);

  while (unit < end) {
    const AttnSeq<kAttnTile> seq(a, it.seq);
    const int rows_left = seq.queries * static_cast<int>(a.group.div) - it.rb * ROWS;
    const int rows = min(rows_left, ROWS);
    const int steps = static_cast<int>(min(static_cast<int64_t>(seq.tiles - it.tile), end - unit));

    // --- the pipeline's stages
    const unsigned char* kc = a.side[0].codes + it.head * L::kCodeRow;
    const unsigned char* vc = a.side[1].codes + it.head * L::kCodeRow;
    const int base0 = it.tile * kAttnTile + warp * kStep;
    // What the table says for position `lane` of step i, or -1.  (It is looked at a step later: a
    // comparison here would wait for it.)
    const int32_t* table = a.table + it.seq * a.width;
    auto lookup = [&](int i) {
      const int p = base0 + i * kAttnTile + lane;
      int b = -1;
      if (lane < kStep && i < steps && p < seq.length) {
        const uint32_t page = a.page.quot(p);
        if (page < a.width) b = table[page];
      }
      return b;
    };
    float ks = 0.0f, vs = 0.0f;        // FP8 scales of this lane's position
    uint64_t kb = 0, vb = 0;           // MXFP4 scale bytes
    // offsets of step i into buffer i & 1, its scales on their way; true: every position of
    // it is there and seen by every query
    auto place = [&](int i, int block) {
      const int p = base0 + i * kAttnTile + lane;
      if (lane < kStep) {
        int64_t at = -1;
        ks = vs = 0.0f;
        kb = vb = 0;
        if (block >= 0 && block < a.blocks) {
          const uint32_t in = p - a.page.quot(p) * a.page.div;
          at = block * a.geo.code_block_stride + in * a.geo.code_row;
          const int64_t sc = block * a.geo.scale_block_stride + in * a.geo.scale_row;
          if constexpr (!FP4) {
            ks = reinterpret_cast<const float*>(a.side[0].scales + sc)[it.head];
            vs = reinterpret_cast<const float*>(a.side[1].scales + sc)[it.head];
          } else {
            const unsigned char* pk = a.side[0].scales + sc + it.head * L::kGroups;
            const unsigned char* pv = a.side[1].scales + sc + it.head * L::kGroups;
            if (a.wide_scales) {
              if constexpr (L::kGroups == 2)
                kb = *reinterpret_cast<const uint16_t*>(pk), vb = *reinterpret_cast<const uint16_t*>(pv);
              else if constexpr (L::kGroups == 4)
                kb = *reinterpret_cast<const uint32_t*>(pk), vb = *reinterpret_cast<const uint32_t*>(pv);
              else
                kb = *reinterpret_cast<const uint64_t*>(pk), vb = *reinterpret_cast<const uint64_t*>(pv);
            } else {
#pragma unroll
              for (int e = 0; e < L::kGroups; e++) {
                kb |= static_cast<uint64_t>(pk[e]) << (8 * e);
                vb |= static_cast<uint64_t>(pv[e]) << (8 * e);
              }
            }
          }
        }
        sh.at[warp][i & 1][lane] = at;
      }
      return __all_sync(0xFFFFFFFFu,
                        lane >= kStep || (block >= 0 && block < a.blocks && p < seq.context));
    };
    Words<L::kBytesK> k[SUB][2];
    Words<L::kBytesV> v[SUB][4];
    auto load_k = [&](int i) {
#pragma unroll
      for (int n = 0; n < 2 * SUB; n++) {
        const int64_t at = sh.at[warp][i & 1][8 * n + g];
        constexpr int bytes = L::kPieceK * (FP4 ? 1 : 2) / 2;  // of a vector
        k[n / 2][n % 2].load(kc + at + bytes * c, 4 * bytes, at >= 0);
      }
    };
    auto load_v = [&](int i) {
#pragma unroll
      for (int n = 0; n < 4 * SUB; n++) {
        const int64_t at = sh.at[warp][i & 1][(n / 2) * 8 + 2 * c + n % 2];
        constexpr int bytes = L::kPieceV * (FP4 ? 1 : 2) / 2;
        v[n / 4][n % 4].load(vc + at + bytes * g, 8 * bytes, at >= 0);
      }
    };

    int block = lookup(0);
    const int after = lookup(1);
    // Q's rows, eight threads a row, each DIM / 8 elements: on their way
    constexpr int kPasses = (NT + 1) / 2, N = DIM / 8;
    uint4 qx[kPasses][N / Vec<T>::N];
    const int eighth = t % 8;
#pragma unroll
    for (int pass = 0; pass < kPasses; pass++) {
      const int r = 16 * pass + t / 8;
      const int row = it.rb * ROWS + (r < rows ? r : 0);
      const int tok = a.group.quot(row), head = it.head * a.group.div + (row - tok * a.group.div);
      const T* p = static_cast<const T*>(a.q) + (seq.first + tok) * a.q_stride +
                   static_cast<int64_t>(head) * DIM + eighth * N;
#pragma unroll
      for (int i = 0; i < N / Vec<T>::N; i++)
        qx[pass][i] = r < rows ? ld_param(p + i * Vec<T>::N) : make_uint4(0u, 0u, 0u, 0u);
    }
    bool clean = place(0, block);
    block = after;
    __syncwarp();
    load_k(0);
    load_v(0);
    // as fragments
#pragma unroll
    for (int pass = 0; pass < kPasses; pass++) {
      const int r = 16 * pass + t / 8;
      float x[N], top = 0.0f;
#pragma unroll
      for (int i = 0; i < N / Vec<T>::N; i++) {
        float v[Vec<T>::N];
        Vec<T>::unpack(qx[pass][i], v);
#pragma unroll
        for (int e = 0; e < Vec<T>::N; e++) x[i * Vec<T>::N + e] = v[e];
      }
      top = group_max<8>(max_abs(x));
      // times 2^(14 - e) for top in [2^e, 2^(e + 1)) (rows below 2^-100: 2^114)
      const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 27), 254) - 127;
      const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
      if (r < ROWS) {
        if (eighth == 0)
          sh.row_scale[r] =
              a.scale_log2 * __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
#pragma unroll
        for (int i = 0; i < N; i++) {
          const int d = eighth * N + i;
          constexpr int P = L::kPieceK;
          const int k = d / (4 * P) * (P / 4) + d % P / 4, lc = d % (4 * P) / P;
          const int at = (r % 8 * 4 + lc) * 4 + d % 4;  // halves
          const float v = x[i] * up;
          const __half hi = __float2half_rn(v);
          reinterpret_cast<__half*>(sh.q[0][r / 8][k])[at] = hi;
          if (SPLIT == 2)
            reinterpret_cast<__half*>(sh.q[SPLIT - 1][r / 8][k])[at] =
                __float2half_rn(v - __half2float(hi));
        }
      }
    }
    __syncthreads();

    // A lane's rows: 8 n + 2 c + e, e 0 or 1.  Positions are the rows of a fragment of scores, query
    // rows its columns: of 16 positions a lane has g and g + 8.
    float rs[NT][2];
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int e = 0; e < 2; e++) rs[n][e] = sh.row_scale[8 * n + 2 * c + e];
    constexpr int kTilesO = DIM / 16;
    float o[NT][kTilesO][4];
    float m[NT][2], l[NT][2];
    // The same of scores and the exponents of V's scales: what hold_factor takes (a power of two, so
    // that a step's result does not depend on it but where weights leave f16's range).
    float vm[NT][2];
#pragma unroll
    for (int n = 0; n < NT; n++) {
#pragma unroll
      for (int j = 0; j < kTilesO; j++) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; e++) m[n][e] = vm[n][e] = -__builtin_huge_valf(), l[n][e] = 0.0f;
    }

    for (int i = 0; i < steps; i++) {
      // scales of this step to shared memory, the next one's on their way
      if (FP4 && lane < kStep) {
        uint16_t mul[L::kGroups];
        ks = mx_multipliers(kb, mul);
#pragma unroll
        for (int e = 0; e < L::kGroups; e++) sh.km[warp][lane][FP4 ? e : 0] = mul[e];
        vs = mx_multipliers(vb, mul);
#pragma unroll
        for (int e = 0; e < L::kGroups; e++) sh.vm[warp][lane][FP4 ? e : 0] = mul[e];
      }
      if (lane < kStep) sh.ks[warp][lane] = ks, sh.vs[warp][lane] = vs;
      const bool was_clean = clean;
      const bool more = i + 1 < steps;
      if (more) {
        clean = place(i + 1, block);
        block = lookup(i + 2);
      }
      __syncwarp();

      // Scores: s[u][n][e], position 16 u + g + 8 (e / 2), row 8 n + 2 c + e % 2.
      float s[SUB][NT][4];
#pragma unroll
      for (int u = 0; u < SUB; u++)
#pragma unroll
        for (int n = 0; n < NT; n++) s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.0f;
#pragma unroll
      for (int q = 0; q < L::kStepsK; q++) {
        uint2 x[SPLIT][NT];
#pragma unroll
        for (int part = 0; part < SPLIT; part++)
#pragma unroll
          for (int n = 0; n < NT; n++) x[part][n] = sh.q[part][n][q][lane];
#pragma unroll
        for (int u = 0; u < SUB; u++) {
          uint32_t h[2][2];  // of position 8 n + g: dimensions k_dim, + 1 and + 2, + 3
#pragma unroll
          for (int n = 0; n < 2; n++) {
            if constexpr (!FP4) {
              h[n][0] = half2_of_e4m3(k[u][n].w[q]);
              h[n][1] = half2_of_e4m3(k[u][n].w[q] >> 16);
            } else {
              uint32_t w[4];
              half2_of_e2m1(k[u][n].w[q / 2], w);
              const uint32_t f = sh.km[warp][16 * u + 8 * n + g][L::k_dim(0, q) / 32 +
                                                                 (L::kPieceK == 32 ? c : c / 2)] *
                                 0x10001u;
              h[n][0] = mul_half2(w[q % 2 * 2], f);
              h[n][1] = mul_half2(w[q % 2 * 2 + 1], f);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int part = 0; part < SPLIT; part++)
              mma_f16(s[u][n], make_uint4(h[0][0], h[1][0], h[0][1], h[1][1]), x[part][n].x,
                      x[part][n].y);
        }
      }
      if (more) load_k(i + 1);

      // in units of log2
      float sv[SUB][2];  // V's scales of the lane's positions
#pragma unroll
      for (int u = 0; u < SUB; u++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
          sv[u][h] = sh.vs[warp][16 * u + 8 * h + g];
          const float sk = sh.ks[warp][16 * u + 8 * h + g];
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) s[u][n][2 * h + e] *= sk * rs[n][e];
        }
      uint32_t hidden[SUB];  // bit 4 n + e: not seen
#pragma unroll
      for (int u = 0; u < SUB; u++) hidden[u] = 0u;
      if (!was_clean) {
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const int r = 8 * n + 2 * c + e, tok = a.group.quot(it.rb * ROWS + r);
#pragma unroll
            for (int u = 0; u < SUB; u++)
#pragma unroll
              for (int h = 0; h < 2; h++) {
                const int at = 16 * u + 8 * h + g;
                if (!(r < rows && sh.at[warp][i & 1][at] >= 0 &&
                      attn_sees(a, seq, tok, base0 + i * kAttnTile + at))) {
                  hidden[u] |= 1u << (4 * n + 2 * h + e);
                  s[u][n][2 * h + e] = -__builtin_huge_valf();
                }
              }
          }
      }
      // The largest exponent of the lane's V scales: with the largest score it is at least what any
      // position of the lane holds.
      float big = 0.0f;
#pragma unroll
      for (int u = 0; u < SUB; u++) big = fmaxf(big, fmaxf(fabsf(sv[u][0]), fabsf(sv[u][1])));
      const float most = static_cast<float>(static_cast<int>(__float_as_uint(big) >> 23) - 126);
      bool higher = false;
      float mx[NT][2];
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          mx[n][e] = fmaxf(s[0][n][e], s[0][n][2 + e]);
#pragma unroll
          for (int u = 1; u < SUB; u++)
            mx[n][e] = fmaxf(mx[n][e], fmaxf(s[u][n][e], s[u][n][2 + e]));
          higher = higher || mx[n][e] > m[n][e] + kSlack || mx[n][e] + most > vm[n][e] + kSlack;
        }
      // Seldom after an item's first step: references stay until a maximum is 2^kSlack above.
      if (__any_sync(0xFFFFFFFFu, higher)) {
        float vk[SUB][2];
#pragma unroll
        for (int u = 0; u < SUB; u++)
#pragma unroll
          for (int h = 0; h < 2; h++) vk[u][h] = scale_exponent(sv[u][h]);
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            float top = fmaxf(mx[n][e], m[n][e]), vtop = vm[n][e];
#pragma unroll
            for (int u = 0; u < SUB; u++)
#pragma unroll
              for (int h = 0; h < 2; h++) vtop = fmaxf(vtop, s[u][n][2 * h + e] + vk[u][h]);
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) {  // the lanes that share a row
              top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
              vtop = fmaxf(vtop, __shfl_xor_sync(0xFFFFFFFFu, vtop, d));
            }
            float f = top == m[n][e] ? 1.0f : attn_exp2(m[n][e] - top);
            l[n][e] *= f;
            // (at most 2: what the row has met is below both references)
            f = f * hold_factor<kHold>(vtop, top) * power_reciprocal(hold_factor<kHold>(vm[n][e], m[n][e]));
#pragma unroll
            for (int j = 0; j < kTilesO; j++) {
              o[n][j][e] *= f;
              o[n][j][2 + e] *= f;
            }
            m[n][e] = top;
            vm[n][e] = vtop;
          }
      }
      // The weights as the second product's fragments: p[u][n][part], pairs of positions of a row.
      uint32_t p[SUB][NT][SPLIT][2];
#pragma unroll
      for (int n = 0; n < NT; n++) {
        float use[2], up[2];
#pragma unroll
        for (int e = 0; e < 2; e++) {
          use[e] = m[n][e] == -__builtin_huge_valf() ? 0.0f : m[n][e];
          up[e] = hold_factor<kHold>(vm[n][e], m[n][e]);
        }
#pragma unroll
        for (int u = 0; u < SUB; u++)
#pragma unroll
          for (int h = 0; h < 2; h++) {
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
              w[e] = attn_exp2(s[u][n][2 * h + e] - use[e]);
              l[n][e] += w[e];
              w[e] = w[e] * up[e] * sv[u][h];  // (in this order: a scale times the factor may be infinite)
              if (!was_clean && (hidden[u] >> (4 * n + 2 * h + e) & 1u)) w[e] = 0.0f;  // whatever its scale
            }
            const uint32_t first = half2_of(w[0], w[1]);
            p[u][n][0][h] = transposed(first);
            if (SPLIT == 2) {
              const float2 f = floats_of_half2(first);
              p[u][n][SPLIT - 1][h] = transposed(half2_of(w[0] - f.x, w[1] - f.y));
            }
          }
      }

      // The second product, for dimensions' tiles 2 j and 2 j + 1: x and y pairs of positions (2 c,
      // 2 c + 1; 8 further) of each one's dimension.
      bool nans = false;  // in V, where someone does not see all
      if (!was_clean) {
        if constexpr (FP4) {  // of a scale
#pragma unroll
          for (int e = 0; e < L::kGroups; e++) nans = nans || (lane < kStep && sh.vm[warp][lane % kStep][FP4 ? e : 0] == 0x7E00);
        } else {
          uint32_t full = 0u;
#pragma unroll
          for (int u = 0; u < SUB; u++)
#pragma unroll
            for (int n = 0; n < 4; n++)
#pragma unroll
              for (int q = 0; q < L::kBytesV / 4; q++)
                full |= (v[u][n].w[q] & 0x7F7F7F7Fu) + 0x01010101u;
          nans = (full & 0x80808080u) != 0u;
        }
        nans = __any_sync(0xFFFFFFFFu, nans);
      }
      auto product = [&](int u, int j, uint32_t x0, uint32_t y0, uint32_t x1, uint32_t y1) {
        if (nans) {
          // A NaN of V reaches those who see its position and nobody else: it leaves the
          // product (0 * NaN is a NaN), and is counted.
          auto nan_halves = [](uint32_t h) {
            return ((h & 0x7FFFu) > 0x7C00u ? 0xFFFFu : 0u) |
                   ((h & 0x7FFF0000u) > 0x7C000000u ? 0xFFFF0000u : 0u);
          };
          const uint32_t a0 = nan_halves(x0), b0 = nan_halves(y0), a1 = nan_halves(x1), b1 = nan_halves(y1);
          constexpr uint32_t one = 0x3C003C00u;
#pragma unroll
          for (int n = 0; n < NT; n++) {
            uint32_t seen[2];  // ones where a weight may be
#pragma unroll
            for (int h = 0; h < 2; h++)
              seen[h] = transposed((hidden[u] >> (4 * n + 2 * h) & 1u ? 0u : 0x3C00u) |
                                   (hidden[u] >> (4 * n + 2 * h + 1) & 1u ? 0u : 0x3C000000u));
            float count[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_f16(count, make_uint4(a0 & one, a1 & one, b0 & one, b1 & one), seen[0], seen[1]);
#pragma unroll
            for (int e = 0; e < 4; e++)
              if (count[e] > 0.0f) o[n][j][e] = __uint_as_float(0x7FC00000u);
          }
          x0 &= ~a0, y0 &= ~b0, x1 &= ~a1, y1 &= ~b1;
        }
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int part = 0; part < SPLIT; part++)
            mma_f16(o[n][j], make_uint4(x0, x1, y0, y1), p[u][n][part][0], p[u][n][part][1]);
      };
#pragma unroll
      for (int u = 0; u < SUB; u++) {
        if constexpr (!FP4) {
#pragma unroll
          for (int q = 0; q < L::kTilesV / 4; q++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
              const uint32_t x = __byte_perm(v[u][0].w[q], v[u][1].w[q], h ? 0x7362 : 0x5140);
              const uint32_t y = __byte_perm(v[u][2].w[q], v[u][3].w[q], h ? 0x7362 : 0x5140);
              product(u, 2 * q + h, half2_of_e4m3(x), half2_of_e4m3(y), half2_of_e4m3(x >> 16),
                      half2_of_e4m3(y >> 16));
            }
        } else {
          constexpr int per = 32 / L::kPieceV;  // lanes g that share a scale
          const uint16_t* f = &sh.vm[warp][16 * u][FP4 ? g / per : 0];
          constexpr int G = FP4 ? L::kGroups : 1;
          const uint32_t f0 = f[2 * c * G] | static_cast<uint32_t>(f[(2 * c + 1) * G]) << 16;
          const uint32_t f1 = f[(8 + 2 * c) * G] | static_cast<uint32_t>(f[(9 + 2 * c) * G]) << 16;
#pragma unroll
          for (int q = 0; q < L::kTilesV / 8; q++) {
            auto even = [](uint32_t lo, uint32_t hi) {
              return (lo & 0x0F0F0F0Fu) | (hi & 0x0F0F0F0Fu) << 4;
            };
            auto odd = [](uint32_t lo, uint32_t hi) {
              return (lo >> 4 & 0x0F0F0F0Fu) | (hi & 0xF0F0F0F0u);
            };
            uint32_t x0[4], y0[4], x1[4], y1[4];
            half2_of_e2m1(even(v[u][0].w[q], v[u][1].w[q]), x0);
            half2_of_e2m1(even(v[u][2].w[q], v[u][3].w[q]), y0);
            half2_of_e2m1(odd(v[u][0].w[q], v[u][1].w[q]), x1);
            half2_of_e2m1(odd(v[u][2].w[q], v[u][3].w[q]), y1);
#pragma unroll
            for (int h = 0; h < 4; h++)
              product(u, 4 * q + h, mul_half2(x0[h], f0), mul_half2(y0[h], f1), mul_half2(x1[h], f0),
                      mul_half2(y1[h], f1));
          }
        }
      }
      if (more) load_v(i + 1);
      __syncwarp();  // the step's scales are read until here
    }

    // --- the warps' results joined, in order
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], d);
        if (g == 0) {
          sh.m[warp][8 * n + 2 * c + e] = m[n][e];
          sh.l[warp][8 * n + 2 * c + e] = l[n][e];
        }
      }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const int r = 8 * n + 2 * c + e;
        float top = sh.m[0][r];
#pragma unroll
        for (int w = 1; w < kAttnWarps; w++) top = fmaxf(top, sh.m[w][r]);
        const float f = m[n][e] == -__builtin_huge_valf() ? 0.0f : attn_exp2(m[n][e] - top);
        const float back = power_reciprocal(hold_factor<kHold>(vm[n][e], m[n][e]));
#pragma unroll
        for (int j = 0; j < kTilesO; j++)
#pragma unroll
          for (int h = 0; h < 2; h++)
            sh.o[warp][r][L::o_at(g, 2 * j + h)] = o[n][j][2 * h + e] * back * f;
      }
    if (t < ROWS) {
      float top = sh.m[0][t], sum = 0.0f;
#pragma unroll
      for (int w = 1; w < kAttnWarps; w++) top = fmaxf(top, sh.m[w][t]);
#pragma unroll
      for (int w = 0; w < kAttnWarps; w++)
        if (sh.l[w][t] != 0.0f) sum += sh.l[w][t] * attn_exp2(sh.m[w][t] - top);
      sh.top[t] = top;
      sh.sum[t] = sum;
    }
    __syncthreads();
    const bool from_start = it.tile == 0, to_end = it.tile + steps == seq.tiles;
    float* part = a.partial +
                  (2 * static_cast<int64_t>(blockIdx.x) + (from_start ? 1 : 0)) * ROWS * (DIM + 2);
    for (int i = t; i < rows * (DIM / 4); i += kAttnThreads) {
      const int r = i / (DIM / 4), d = i % (DIM / 4) * 4;
      const int at = L::o_first(d);
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kAttnWarps; w++) {
        const float* y = &sh.o[w][r][at];
        x.x += y[0], x.y += y[8], x.z += y[16], x.w += y[24];
      }
      const float sum = sh.sum[r];
      if (from_start && to_end) {
        const int row = it.rb * ROWS + r;
        const int tok = a.group.quot(row), i_head = row - tok * a.group.div;
        const int64_t head = static_cast<int64_t>(seq.first + tok) * a.heads * a.group.div +
                             it.head * a.group.div + i_head;
        // nothing seen: zeros
        const float inv = sum != 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
        T* out = static_cast<T*>(a.out) + head * DIM + d;
        out[0] = narrow<T>(x.x * inv);
        out[1] = narrow<T>(x.y * inv);
        out[2] = narrow<T>(x.z * inv);
        out[3] = narrow<T>(x.w * inv);
        if (d == 0 && a.lse != nullptr)
          a.lse[head] = sum != 0.0f ? (sh.top[r] + log2f(sum)) * kAttnLn2 : -__builtin_huge_valf();
      } else {
        *reinterpret_cast<float4*>(part + r * DIM + d) = x;
        if (d == 0) {
          part[ROWS * DIM + 2 * r] = sh.top[r];
          part[ROWS * DIM + 2 * r + 1] = sum;
        }
      }
    }
    if (from_start && !to_end && t == 0) {
      // the shares that the item reaches into
      const int64_t item_end = unit + seq.tiles;
      const int64_t last = (item_end - 1) / share;
      a.joins[blockIdx.x] = make_int4(it.seq, it.head, it.rb, static_cast<int>(last - blockIdx.x + 1));
    }
    __syncthreads();  // the shared memory is written anew

    unit += steps + kItemCost;
    if (unit >= end) break;
    next_item<ROWS, kAttnTile>(a, it, seq.queries);
  }
}

// Of an SM's memory what holds `bytes` of shared memory, in percent of the most; the rest is L1, through
// which the codes come: 400009 tokens of 48 sequences take 154 us with three blocks' room, 188 us with 55
// percent and four blocks, 216 us with all of it.
constexpr int room(size_t bytes) {
  for (size_t kb : {8, 16, 32, 64, 100, 132, 164, 196})
    if (bytes <= kb * 1024) return static_cast<int>((kb * 100 + 227) / 228);
  return 100;
}

template <typename T, bool FP4, int DIM, int NT>
cudaError_t attn_go(AttnArgs a, void* workspace, cudaStream_t s) {
  constexpr int blocks = attn_blocks<DIM, NT>, ROWS = 8 * NT;
  constexpr size_t shared = sizeof(AttnShared<T, FP4, DIM, NT, 16 * kSub<FP4, DIM, NT>>);
  constexpr int percent = room(blocks * (shared + 1024));
  constexpr unsigned shares = kSms * blocks;
  static std::atomic<int> done[64], done_join[64];
  auto* kernel = cache_attention_kernel<T, FP4, DIM, NT>;
  auto* join = cache_attention_join_kernel<T, ROWS, DIM, FP4>;
  cudaError_t e = allow_shared(kernel, shared, done, percent);
  if (e == cudaSuccess) e = allow_shared(join, 0, done_join, percent);
  if (e != cudaSuccess) return e;
  a.joins = static_cast<int4*>(workspace);
  a.partial = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) +
                                       attn_joins_bytes(shares));
  e = launch_pdl(kernel, dim3(shares), dim3(kAttnThreads), shared, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(join, dim3(shares, ROWS / kJoinRows), dim3(DIM / 4, kJoinRows), 0, s, a);
}

// How many tiles of eight rows an item has, of at most `most`.  A step costs about 5 + 7 tiles (one
// token, heads of 128 in FP8, 100009 tokens in 16 sequences: 16 rows take 81 us as two items of one
// tile, 65 us as one of two; 24 rows 114 us as three of one, 87 us as one of three); a sequence with
// fewer rows than an item pays for them all.  With as
// many new tokens in each sequence its rows are known here; otherwise anything up to twice the average is
// taken to be as likely (4 to 24 rows, 13 on average: one tile 72 us, two 76; in MXFP4 74 and 83).
int row_tiles(int64_t average, bool even, int most) {
  int best = 1;
  int64_t least = 0;
  for (int nt = 1; nt <= most; nt++) {
    const int64_t rows = 8 * nt, top = 2 * average - 1, whole = top / rows;
    const int64_t items = even ? (average + rows - 1) / rows
                               : rows * whole * (whole + 1) / 2 + top % rows * (whole + 1);
    if (nt == 1 || items * (5 + 7 * nt) < least) best = nt, least = items * (5 + 7 * nt);
  }
  return best;
}

template <typename T, bool FP4, int DIM, int MOST>
cudaError_t attn_dim(int64_t average, bool even, const AttnArgs& a, void* ws, cudaStream_t s) {
  const int tiles = row_tiles(average, even, MOST);
  if constexpr (MOST >= 3)
    if (tiles == 3) return attn_go<T, FP4, DIM, 3>(a, ws, s);
  if constexpr (MOST >= 2)
    if (tiles == 2) return attn_go<T, FP4, DIM, 2>(a, ws, s);
  return attn_go<T, FP4, DIM, 1>(a, ws, s);
}

// Heads of 256: three tiles of O do not fit in the registers, nor do two beside FP8's codes (16 rows of
// one token, 50009 tokens in 8 sequences: one tile 49 us, two 59; MXFP4 58 and 45).
template <typename T, bool FP4>
cudaError_t attn_few(int64_t average, bool even, int64_t dim, const AttnArgs& a, void* ws, cudaStream_t s) {
  if (dim == 64) return attn_dim<T, FP4, 64, 3>(average, even, a, ws, s);
  if (dim == 128) return attn_dim<T, FP4, 128, 3>(average, even, a, ws, s);
  return attn_dim<T, FP4, 256, FP4 ? 2 : 1>(average, even, a, ws, s);
}

AttnArgs attn_args(const KvCacheArgs& c, const CacheAttentionArgs& p) {
  const int64_t groups = c.head_dim / 32;
  return AttnArgs{p.q,
                  p.out,
                  p.lse,
                  {{c.k_codes, c.k_scales}, {c.v_codes, c.v_scales}},
                  cache_geometry(c),
                  p.block_table,
                  p.seq_lens,
                  p.cu_q,
                  reinterpret_cast<const uint32_t*>(p.tree),
                  p.table_width,
                  c.blocks,
                  p.q_stride,
                  p.tokens,
                  static_cast<int>(p.seqs),
                  static_cast<int>(c.heads),
                  FastDiv(static_cast<uint32_t>(p.q_heads / c.heads)),
                  FastDiv(static_cast<uint32_t>(c.block_size)),
                  static_cast<int>(p.tree_words),
                  p.scale * kAttnLog2e,
                  c.fp4 && ((reinterpret_cast<uintptr_t>(c.k_scales) |
                             reinterpret_cast<uintptr_t>(c.v_scales) |
                             static_cast<uintptr_t>(c.scale_block_stride)) %
                            static_cast<uintptr_t>(groups)) == 0,
                  nullptr,
                  nullptr};
}

}  // namespace

int64_t cache_attention_workspace(int64_t head_dim) {
  const int64_t few = head_dim == 256
                          ? attn_bytes(kSms * attn_blocks<256, 2>, 16, head_dim)
                          : attn_bytes(kSms * attn_blocks<128, 3>, 24, head_dim);
  const int64_t many = attn_rows_bytes(head_dim);
  return few > many ? few : many;
}

// Query rows a sequence and head of the cache, on average, that the kernel for few rows takes where there
// is one for many: three tiles.  (24 rows of one token, heads of 128 in FP8, 100009 tokens in 16 sequences:
// 87 us here, 105 there; here every 24 more take as long again.)
constexpr int64_t kFewRows = 24;

cudaError_t launch_cache_attention(const KvCacheArgs& c, const CacheAttentionArgs& p, int is_bf16,
                                   cudaStream_t stream) {
  const AttnArgs a = attn_args(c, p);
  // (what each sequence has is known on the device alone)
  const int64_t average = (p.tokens * (p.q_heads / c.heads) + p.seqs - 1) / p.seqs;
  const bool even = p.tokens % p.seqs == 0;
  if (is_bf16 && c.head_dim <= 128 && average > kFewRows)
    return launch_attn_rows(a, c.fp4, c.head_dim, p.workspace, stream);
  if (is_bf16)
    return c.fp4 ? attn_few<__nv_bfloat16, true>(average, even, c.head_dim, a, p.workspace, stream)
                 : attn_few<__nv_bfloat16, false>(average, even, c.head_dim, a, p.workspace, stream);
  return c.fp4 ? attn_few<float, true>(average, even, c.head_dim, a, p.workspace, stream)
               : attn_few<float, false>(average, even, c.head_dim, a, p.workspace, stream);
}

}  // namespace nr
