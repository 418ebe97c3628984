// Attention over the quantised paged cache (sm_103a): one token, a chain or a tree of drafted
// tokens of each sequence against everything cached for it.
//
// Scores, weights and sums are f32, one pass over K and V with the running maximum and sum of
// the softmax.  Codes become f16 exactly (e4m3 has 4 significant bits, e2m1 2), and each row of
// Q is brought to f16's range by a power of two, so products of Q and K are exact and summed in
// f32.  A token's K scale multiplies its scores, its V scale its weights.  MXFP4 has a scale for
// 32 elements: relative to the token's largest they are powers of two that f16 holds down to
// 2^-37 of it; what is smaller counts as zero.  Weights are rounded to f16 (11 bits, relative
// to the largest V scale met), the one rounding that is not f32's: it is four times finer than the
// bf16 output's.  With f32 tensors Q and the weights are two f16 parts each (22 bits).
//
// Few queries a sequence: bound by HBM, each code read once for up to 16 query rows.  A warp
// reads 16 positions' codes straight into the registers where mma.sync wants them: which
// dimensions a lane's vector holds is free as long as Q (and the output's order) agree.  K of the
// next positions is on its way during softmax and the second product, V during the first.
#include <type_traits>

#include "attn_plan.cuh"
#include "nr_internal.h"

namespace nr {
namespace {

// A share for each block that fits at once on 152 SMs (any number is right).
template <int DIM, int ROWS>
constexpr int attn_blocks = DIM == 256 ? 2 : ROWS == 8 ? 4 : 3;
constexpr int kSms = 152;

constexpr int kAttnThreads = 128;
constexpr int kAttnWarps = kAttnThreads / kWarp;
constexpr int kStep = 16;          // positions a warp handles at a time
constexpr int kAttnTile = kStep * kAttnWarps;  // positions of a block's step
constexpr int kItemCost = 3;  // tiles that an item costs besides its own
constexpr float kWeightUp = 16384.0f;  // weights are held times 2^14

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
};

template <typename T, bool FP4, int DIM, int ROWS>
struct AttnShared {
  static constexpr int SPLIT = sizeof(T) == 4 ? 2 : 1;
  using L = Layout<FP4, DIM>;
  // fragments: 16 rows are the first operand, 8 rows the second
  using Fragment = typename std::conditional<ROWS == 16, uint4, uint2>::type;
  Fragment q[SPLIT][L::kStepsK][kWarp];
  alignas(16) float row_scale[ROWS];
  alignas(16) int64_t at[kAttnWarps][2][kStep];        // code offsets, -1: no such position
  float ks[kAttnWarps][kStep];             // scales of K, of V
  float vs[kAttnWarps][kStep];
  uint16_t km[kAttnWarps][kStep][FP4 ? L::kGroups : 1];
  uint16_t vm[kAttnWarps][kStep][FP4 ? L::kGroups : 1];
  float m[kAttnWarps][ROWS], l[kAttnWarps][ROWS];
  float top[ROWS], sum[ROWS];
  alignas(16) float o[kAttnWarps][ROWS][DIM + 4];
  AttnPlan<kAttnThreads> plan;
};

template <typename T, bool FP4, int DIM, int ROWS>
__global__ void __launch_bounds__(kAttnThreads, attn_blocks<DIM, ROWS>)
    cache_attention_kernel(const AttnArgs a) {
  using L = Layout<FP4, DIM>;
  constexpr int SPLIT = sizeof(T) == 4 ? 2 : 1;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  auto& sh = *reinterpret_cast<AttnShared<T, FP4, DIM, ROWS>*>(smem_raw);
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

    // Q's rows as fragments: eight threads a row, each DIM / 8 elements
    {
      const int r = t / 8, part = t % 8;
      constexpr int N = DIM / 8;
      float x[N], top = 0.0f;
      const int row = it.rb * ROWS + r;
      const int tok = a.group.quot(row), head = it.head * a.group.div + (row - tok * a.group.div);
      const T* p = static_cast<const T*>(a.q) + (seq.first + tok) * a.q_stride +
                   static_cast<int64_t>(head) * DIM + part * N;
#pragma unroll
      for (int i = 0; i < N / Vec<T>::N; i++) {
        float v[Vec<T>::N];
        Vec<T>::unpack(r < rows ? ld_param(p + i * Vec<T>::N) : make_uint4(0u, 0u, 0u, 0u), v);
#pragma unroll
        for (int e = 0; e < Vec<T>::N; e++) x[i * Vec<T>::N + e] = v[e];
      }
      top = group_max<8>(max_abs(x));
      // times 2^(14 - e) for top in [2^e, 2^(e + 1)) (rows below 2^-100: 2^114)
      const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 27), 254) - 127;
      const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
      if (part == 0 && r < ROWS)
        sh.row_scale[r] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
#pragma unroll
      for (int i = 0; i < N; i++) {
        const int d = part * N + i;
        constexpr int P = L::kPieceK;
        const int k = d / (4 * P) * (P / 4) + d % P / 4, lc = d % (4 * P) / P, sub = d % 4;
        const int at = ROWS == 16 ? ((r % 8) * 4 + lc) * 8 + ((sub / 2) * 2 + r / 8) * 2 + sub % 2
                                  : (r * 4 + lc) * 4 + sub;  // halves
        if (r >= ROWS) continue;
        const float v = x[i] * up;
        const __half hi = __float2half_rn(v);
        reinterpret_cast<__half*>(sh.q[0][k])[at] = hi;
        if (SPLIT == 2)
          reinterpret_cast<__half*>(sh.q[SPLIT - 1][k])[at] = __float2half_rn(v - __half2float(hi));
      }
    }
    __syncthreads();
    // A lane's two rows: with 16 they are rows of the scores' fragment (positions its columns),
    // with 8 its columns (positions its rows): half the products, and half of O.
    const int r0 = ROWS == 16 ? g : 2 * c, r1 = ROWS == 16 ? g + 8 : 2 * c + 1;
    const float rs0 = sh.row_scale[r0], rs1 = sh.row_scale[r1];
    const int row0 = it.rb * ROWS + r0, row1 = it.rb * ROWS + r1;
    const int tok0 = a.group.quot(row0), tok1 = a.group.quot(row1);

    constexpr int kTilesO = L::kTilesV * ROWS / 16;
    float o[kTilesO][4];
#pragma unroll
    for (int j = 0; j < kTilesO; j++) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    float m0 = -__builtin_huge_valf(), m1 = m0, l0 = 0.0f, l1 = 0.0f;
    // A row's weights are held relative to the largest V scale that it has met, as a power of two
    // (so that a step's result does not depend on it but where weights leave f16's range).
    float vref0 = 0.0f, vref1 = 0.0f;

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
    Words<L::kBytesK> k[2];
    Words<L::kBytesV> v[4];
    auto load_k = [&](int i) {
#pragma unroll
      for (int n = 0; n < 2; n++) {
        const int64_t at = sh.at[warp][i & 1][8 * n + g];
        constexpr int bytes = L::kPieceK * (FP4 ? 1 : 2) / 2;  // of a vector
        k[n].load(kc + at + bytes * c, 4 * bytes, at >= 0);
      }
    };
    auto load_v = [&](int i) {
#pragma unroll
      for (int n = 0; n < 4; n++) {
        const int64_t at = sh.at[warp][i & 1][(n / 2) * 8 + 2 * c + n % 2];
        constexpr int bytes = L::kPieceV * (FP4 ? 1 : 2) / 2;
        v[n].load(vc + at + bytes * g, 8 * bytes, at >= 0);
      }
    };

    int block = lookup(0);
    bool clean = place(0, block);
    block = lookup(1);
    __syncwarp();
    load_k(0);
    load_v(0);

    for (int i = 0; i < steps; i++) {
      // scales of this step to shared memory, the next one's on their way
      if (FP4 && lane < kStep) {
        uint16_t m[L::kGroups];
        ks = mx_multipliers(kb, m);
#pragma unroll
        for (int e = 0; e < L::kGroups; e++) sh.km[warp][lane][FP4 ? e : 0] = m[e];
        vs = mx_multipliers(vb, m);
#pragma unroll
        for (int e = 0; e < L::kGroups; e++) sh.vm[warp][lane][FP4 ? e : 0] = m[e];
      }
      if (lane < kStep) sh.ks[warp][lane] = ks, sh.vs[warp][lane] = vs;
      const float vs_now = vs;
      const bool was_clean = clean;
      const bool more = i + 1 < steps;
      if (more) {
        clean = place(i + 1, block);
        block = lookup(i + 2);
      }
      __syncwarp();

      // Scores: s[n][e], element e of position fragment n (16 rows: n-th eight positions; 8 rows: one
      // fragment of all 16).
      constexpr int kN = ROWS / 8;
      float s[kN][4];
#pragma unroll
      for (int n = 0; n < kN; n++) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
      for (int q = 0; q < L::kStepsK; q++) {
        uint32_t h[2][2];  // of position 8 n + g: dimensions k_dim, + 1 and + 2, + 3
#pragma unroll
        for (int n = 0; n < 2; n++) {
          if constexpr (!FP4) {
            h[n][0] = half2_of_e4m3(k[n].w[q]);
            h[n][1] = half2_of_e4m3(k[n].w[q] >> 16);
          } else {
            uint32_t w[4];
            half2_of_e2m1(k[n].w[q / 2], w);
            const uint32_t f = sh.km[warp][8 * n + g][L::k_dim(0, q) / 32 +
                                                     (L::kPieceK == 32 ? c : c / 2)] *
                               0x10001u;
            h[n][0] = mul_half2(w[q % 2 * 2], f);
            h[n][1] = mul_half2(w[q % 2 * 2 + 1], f);
          }
        }
#pragma unroll
        for (int part = 0; part < SPLIT; part++) {
          const auto x = sh.q[part][q][lane];
          if constexpr (ROWS == 16) {
            mma_f16(s[0], x, h[0][0], h[0][1]);
            mma_f16(s[1], x, h[1][0], h[1][1]);
          } else {
            mma_f16(s[0], make_uint4(h[0][0], h[1][0], h[0][1], h[1][1]), x.x, x.y);
          }
        }
      }
      if (more) load_k(i + 1);

      // In units of log2.  Element e of fragment n: row r0 or r1, position at(n, e).
      auto at = [&](int n, int e) { return ROWS == 16 ? 8 * n + 2 * c + e % 2 : g + 8 * (e / 2); };
      auto second = [](int e) { return ROWS == 16 ? e >= 2 : e % 2 == 1; };  // of r1
      float mx0 = m0, mx1 = m1;
      float sv[kN][2];  // V's scales of the lane's positions
      {
        float sk[kN][2];
#pragma unroll
        for (int n = 0; n < kN; n++) {
          if (ROWS == 16) {
            const float2 x = *reinterpret_cast<const float2*>(&sh.ks[warp][8 * n + 2 * c]);
            const float2 y = *reinterpret_cast<const float2*>(&sh.vs[warp][8 * n + 2 * c]);
            sk[n][0] = x.x, sk[n][1] = x.y, sv[n][0] = y.x, sv[n][1] = y.y;
          } else {
            sk[n][0] = sh.ks[warp][g], sk[n][1] = sh.ks[warp][g + 8];
            sv[n][0] = sh.vs[warp][g], sv[n][1] = sh.vs[warp][g + 8];
          }
#pragma unroll
          for (int e = 0; e < 4; e++)
            s[n][e] *= sk[n][ROWS == 16 ? e % 2 : e / 2] * (second(e) ? rs1 : rs0);
        }
      }
      uint32_t hidden = 0;  // bit 4 n + e: not seen
      if (!was_clean) {
        const int rows_end = it.rb * ROWS + rows;
#pragma unroll
        for (int n = 0; n < kN; n++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const int p = base0 + i * kAttnTile + at(n, e);
            const bool there = sh.at[warp][i & 1][at(n, e)] >= 0;
            if (!(there && (second(e) ? row1 : row0) < rows_end &&
                  attn_sees(a, seq, second(e) ? tok1 : tok0, p))) {
              hidden |= 1u << (4 * n + e);
              s[n][e] = -__builtin_huge_valf();
            }
          }
      }
#pragma unroll
      for (int n = 0; n < kN; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          if (second(e)) mx1 = fmaxf(mx1, s[n][e]);
          else mx0 = fmaxf(mx0, s[n][e]);
        }
      // the lanes that share a row
      constexpr int kFirst = ROWS == 16 ? 1 : 4, kLast = ROWS == 16 ? 2 : 16;
#pragma unroll
      for (int d = kFirst; d <= kLast; d <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xFFFFFFFFu, mx0, d));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xFFFFFFFFu, mx1, d));
      }
      float vt0, vt1;
      if (was_clean) {
        const float own = lane < kStep ? scale_reference(vs_now) : 0.0f;
        vt0 = vt1 = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(own)));
      } else {
        vt0 = vt1 = 0.0f;
#pragma unroll
        for (int n = 0; n < kN; n++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            if (hidden >> (4 * n + e) & 1u) continue;
            const float x = scale_reference(sv[n][ROWS == 16 ? e % 2 : e / 2]);
            if (second(e)) vt1 = fmaxf(vt1, x);
            else vt0 = fmaxf(vt0, x);
          }
#pragma unroll
        for (int d = kFirst; d <= kLast; d <<= 1) {
          vt0 = fmaxf(vt0, __shfl_xor_sync(0xFFFFFFFFu, vt0, d));
          vt1 = fmaxf(vt1, __shfl_xor_sync(0xFFFFFFFFu, vt1, d));
        }
      }
      vt0 = fmaxf(vt0, vref0);
      vt1 = fmaxf(vt1, vref1);
      const float use0 = mx0 == -__builtin_huge_valf() ? 0.0f : mx0;
      const float use1 = mx1 == -__builtin_huge_valf() ? 0.0f : mx1;
      if (__any_sync(0xFFFFFFFFu, mx0 > m0 || mx1 > m1 || vt0 > vref0 || vt1 > vref1)) {
        float f0 = attn_exp2(m0 - use0), f1 = attn_exp2(m1 - use1);
        l0 *= f0;
        l1 *= f1;
        f0 *= vref0 * power_reciprocal(vt0);
        f1 *= vref1 * power_reciprocal(vt1);
#pragma unroll
        for (int j = 0; j < kTilesO; j++)
#pragma unroll
          for (int e = 0; e < 4; e++) o[j][e] *= second(e) ? f1 : f0;
        m0 = mx0;
        m1 = mx1;
        vref0 = vt0;
        vref1 = vt1;
      }
      const float winv0 = kWeightUp * power_reciprocal(vref0);
      const float winv1 = kWeightUp * power_reciprocal(vref1);
      float w[kN][4];
#pragma unroll
      for (int n = 0; n < kN; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          w[n][e] = attn_exp2(s[n][e] - (second(e) ? use1 : use0));
          if (second(e)) l1 += w[n][e];
          else l0 += w[n][e];
          w[n][e] *= sv[n][ROWS == 16 ? e % 2 : e / 2] * (second(e) ? winv1 : winv0);
          if (!was_clean && (hidden >> (4 * n + e) & 1u)) w[n][e] = 0.0f;  // whatever its scale
        }
      // As fragments of the second product: 16 rows its first operand as they are, 8 rows its second,
      // turned around.  p[part][0 .. 3] or [0 .. 1].
      uint32_t p[SPLIT][2 * kN];
#pragma unroll
      for (int n = 0; n < kN; n++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const float x = w[n][2 * h], y = w[n][2 * h + 1];
          p[0][2 * n + h] = half2_of(x, y);
          if (SPLIT == 2) {
            const float2 f = floats_of_half2(p[0][2 * n + h]);
            p[SPLIT - 1][2 * n + h] = half2_of(x - f.x, y - f.y);
          }
        }
      uint32_t seen[2 * kN];  // ones where a weight may be
#pragma unroll
      for (int n = 0; n < 2 * kN; n++)
        seen[n] = (hidden >> (2 * n) & 1u ? 0u : 0x3C00u) | (hidden >> (2 * n + 1) & 1u ? 0u : 0x3C000000u);
      if constexpr (ROWS == 8) {
#pragma unroll
        for (int n = 0; n < 2; n++) {
#pragma unroll
          for (int part = 0; part < SPLIT; part++) p[part][n] = transposed(p[part][n]);
          if (!was_clean) seen[n] = transposed(seen[n]);
        }
      }

      // The second product, for output tiles j and j + 1: x and y pairs of positions (2 c, 2 c + 1; 8
      // further) of each one's dimension.
      auto product = [&](int j, uint32_t x0, uint32_t y0, uint32_t x1, uint32_t y1) {
        auto both = [&](float (&d)[4], float (&d2)[4], const uint32_t (&f)[2 * kN], uint32_t x0, uint32_t y0,
                        uint32_t x1, uint32_t y1) {
          if constexpr (ROWS == 16) {
            const uint4 rows16 = make_uint4(f[0], f[1], f[2 * kN - 2], f[2 * kN - 1]);
            mma_f16(d, rows16, x0, y0);
            mma_f16(d2, rows16, x1, y1);
          } else {
            mma_f16(d, make_uint4(x0, x1, y0, y1), f[0], f[1]);
          }
        };
        constexpr int kPer = ROWS == 16 ? 1 : 2;  // output tiles a fragment
        float(&d)[4] = o[j / kPer];
        float(&d2)[4] = o[(j + 1) / kPer];
        if (!was_clean) {
          // A NaN of V reaches those who see its position and nobody else: it leaves the
          // product (0 * NaN is a NaN), and is counted.
          auto nan_halves = [](uint32_t h) {
            return ((h & 0x7FFFu) > 0x7C00u ? 0xFFFFu : 0u) |
                   ((h & 0x7FFF0000u) > 0x7C000000u ? 0xFFFF0000u : 0u);
          };
          const uint32_t a0 = nan_halves(x0), b0 = nan_halves(y0), a1 = nan_halves(x1), b1 = nan_halves(y1);
          if (__any_sync(0xFFFFFFFFu, (a0 | b0 | a1 | b1) != 0)) {
            float n0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, n1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            constexpr uint32_t one = 0x3C003C00u;
            both(n0, n1, seen, a0 & one, b0 & one, a1 & one, b1 & one);
            x0 &= ~a0, y0 &= ~b0, x1 &= ~a1, y1 &= ~b1;
#pragma unroll
            for (int e = 0; e < 4; e++) {
              if (n0[e] > 0.0f) d[e] = __uint_as_float(0x7FC00000u);
              if (ROWS == 16 && n1[e] > 0.0f) d2[e] = __uint_as_float(0x7FC00000u);
            }
          }
        }
#pragma unroll
        for (int part = 0; part < SPLIT; part++) both(d, d2, p[part], x0, y0, x1, y1);
      };
      if constexpr (!FP4) {
#pragma unroll
        for (int q = 0; q < L::kTilesV / 4; q++) {
#pragma unroll
          for (int h = 0; h < 2; h++) {
            const uint32_t x = __byte_perm(v[0].w[q], v[1].w[q], h ? 0x7362 : 0x5140);
            const uint32_t y = __byte_perm(v[2].w[q], v[3].w[q], h ? 0x7362 : 0x5140);
            product(4 * q + 2 * h, half2_of_e4m3(x), half2_of_e4m3(y), half2_of_e4m3(x >> 16),
                    half2_of_e4m3(y >> 16));
          }
        }
      } else {
        constexpr int per = 32 / L::kPieceV;  // lanes g that share a scale
        const uint16_t* f = &sh.vm[warp][0][FP4 ? g / per : 0];
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
          half2_of_e2m1(even(v[0].w[q], v[1].w[q]), x0);
          half2_of_e2m1(even(v[2].w[q], v[3].w[q]), y0);
          half2_of_e2m1(odd(v[0].w[q], v[1].w[q]), x1);
          half2_of_e2m1(odd(v[2].w[q], v[3].w[q]), y1);
#pragma unroll
          for (int h = 0; h < 4; h++)
            product(8 * q + 2 * h, mul_half2(x0[h], f0), mul_half2(y0[h], f1), mul_half2(x1[h], f0),
                    mul_half2(y1[h], f1));
        }
      }
      if (more) load_v(i + 1);
      __syncwarp();  // the step's scales are read until here
    }

    // --- the warps' results joined, in order
    constexpr int kFirst = ROWS == 16 ? 1 : 4, kLast = ROWS == 16 ? 2 : 16;
#pragma unroll
    for (int d = kFirst; d <= kLast; d <<= 1) {
      l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, d);
      l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, d);
    }
    if ((ROWS == 16 ? c : g) == 0) {
      sh.m[warp][r0] = m0;
      sh.m[warp][r1] = m1;
      sh.l[warp][r0] = l0;
      sh.l[warp][r1] = l1;
    }
    __syncthreads();
    float top0 = sh.m[0][r0], top1 = sh.m[0][r1];
#pragma unroll
    for (int w = 1; w < kAttnWarps; w++) {
      top0 = fmaxf(top0, sh.m[w][r0]);
      top1 = fmaxf(top1, sh.m[w][r1]);
    }
    const float f0 = m0 == -__builtin_huge_valf() ? 0.0f : attn_exp2(m0 - top0);
    const float f1 = m1 == -__builtin_huge_valf() ? 0.0f : attn_exp2(m1 - top1);
    const float back0 = vref0 * (1.0f / kWeightUp), back1 = vref1 * (1.0f / kWeightUp);
#pragma unroll
    for (int j = 0; j < kTilesO; j++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const bool two = ROWS == 16 ? e >= 2 : e % 2 == 1;
        const int d = ROWS == 16 ? L::v_dim(2 * c + e % 2, j) : L::v_dim(g, 2 * j + e / 2);
        sh.o[warp][two ? r1 : r0][d] = o[j][e] * (two ? back1 : back0) * (two ? f1 : f0);
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
      float4 x = *reinterpret_cast<const float4*>(&sh.o[0][r][d]);
#pragma unroll
      for (int w = 1; w < kAttnWarps; w++) {
        const float4 y = *reinterpret_cast<const float4*>(&sh.o[w][r][d]);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
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

template <typename T, bool FP4, int DIM, int ROWS>
cudaError_t attn_go(AttnArgs a, void* workspace, cudaStream_t s) {
  constexpr size_t shared = sizeof(AttnShared<T, FP4, DIM, ROWS>);
  constexpr unsigned shares = kSms * attn_blocks<DIM, ROWS>;
  static std::atomic<int> done[64], done_join[64];
  cudaError_t e = allow_shared(cache_attention_kernel<T, FP4, DIM, ROWS>, shared, done);
  if (e == cudaSuccess) e = allow_shared(cache_attention_join_kernel<T, ROWS, DIM>, 0, done_join);
  if (e != cudaSuccess) return e;
  a.joins = static_cast<int4*>(workspace);
  a.partial = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) +
                                       attn_joins_bytes(shares));
  e = launch_pdl(cache_attention_kernel<T, FP4, DIM, ROWS>, dim3(shares), dim3(kAttnThreads), shared,
                 s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(cache_attention_join_kernel<T, ROWS, DIM>, dim3(shares, ROWS / kJoinRows),
                    dim3(DIM / 4, kJoinRows), 0, s, a);
}

template <typename T, bool FP4, int ROWS>
cudaError_t attn_dim(int64_t dim, const AttnArgs& a, void* ws, cudaStream_t s) {
  if (dim == 64) return attn_go<T, FP4, 64, ROWS>(a, ws, s);
  if (dim == 128) return attn_go<T, FP4, 128, ROWS>(a, ws, s);
  return attn_go<T, FP4, 256, ROWS>(a, ws, s);
}

template <typename T, bool FP4>
cudaError_t attn_rows(int64_t average, int64_t dim, const AttnArgs& a, void* ws, cudaStream_t s) {
  return average <= 8 ? attn_dim<T, FP4, 8>(dim, a, ws, s) : attn_dim<T, FP4, 16>(dim, a, ws, s);
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
  const bool wide = head_dim == 256;
  const int64_t rows8 =
      attn_bytes(kSms * (wide ? attn_blocks<256, 8> : attn_blocks<128, 8>), 8, head_dim);
  const int64_t rows16 =
      attn_bytes(kSms * (wide ? attn_blocks<256, 16> : attn_blocks<128, 16>), 16, head_dim);
  const int64_t many = attn_rows_bytes(head_dim), few = rows8 > rows16 ? rows8 : rows16;
  return few > many ? few : many;
}

cudaError_t launch_cache_attention(const KvCacheArgs& c, const CacheAttentionArgs& p, int is_bf16,
                                   cudaStream_t stream) {
  const AttnArgs a = attn_args(c, p);
  // Query rows an item on average (what each sequence has is known on the device alone).  More than
  // 16: the kernel whose tile of products has 128.  Up to 8: the form with half the products.
  const int64_t average = (p.tokens * (p.q_heads / c.heads) + p.seqs - 1) / p.seqs;
  if (is_bf16 && c.head_dim <= 128 && average > 16)
    return launch_attn_rows(a, c.fp4, c.head_dim, p.workspace, stream);
  if (is_bf16)
    return c.fp4 ? attn_rows<__nv_bfloat16, true>(average, c.head_dim, a, p.workspace, stream)
                 : attn_rows<__nv_bfloat16, false>(average, c.head_dim, a, p.workspace, stream);
  return c.fp4 ? attn_rows<float, true>(average, c.head_dim, a, p.workspace, stream)
               : attn_rows<float, false>(average, c.head_dim, a, p.workspace, stream);
}

}  // namespace nr
