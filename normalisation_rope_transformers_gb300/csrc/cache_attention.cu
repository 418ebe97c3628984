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
template <int DIM>
constexpr int attn_blocks = DIM == 256 ? 2 : 3;
constexpr int kSms = 152;

constexpr int kAttnThreads = 128;
constexpr int kAttnWarps = kAttnThreads / kWarp;
constexpr int kAttnRows = 16;
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

template <typename T, bool FP4, int DIM>
struct AttnShared {
  static constexpr int SPLIT = sizeof(T) == 4 ? 2 : 1;
  using L = Layout<FP4, DIM>;
  uint4 q[SPLIT][L::kStepsK][kWarp];       // fragments
  float row_scale[kAttnRows];
  int64_t at[kAttnWarps][2][kStep];        // code offsets, -1: no such position
  float ks[kAttnWarps][kStep];             // scales of K, of V
  float vs[kAttnWarps][kStep];
  uint16_t km[kAttnWarps][kStep][FP4 ? L::kGroups : 1];
  uint16_t vm[kAttnWarps][kStep][FP4 ? L::kGroups : 1];
  float m[kAttnWarps][kAttnRows], l[kAttnWarps][kAttnRows];
  float top[kAttnRows], sum[kAttnRows];
  float o[kAttnWarps][kAttnRows][DIM + 4];
  AttnPlan<kAttnThreads> plan;
};

template <typename T, bool FP4, int DIM>
__global__ void __launch_bounds__(kAttnThreads, attn_blocks<DIM>)
    cache_attention_kernel(const AttnArgs a) {
  using L = Layout<FP4, DIM>;
  constexpr int SPLIT = sizeof(T) == 4 ? 2 : 1;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  auto& sh = *reinterpret_cast<AttnShared<T, FP4, DIM>*>(smem_raw);
  const int t = threadIdx.x, warp = t / kWarp, lane = t % kWarp, g = lane / 4, c = lane % 4;
  pdl_enter();  // before any global read: the previous kernel may still run
  make_plan<kAttnRows, kAttnTile, kItemCost>(a, sh.plan);
  const int64_t total = sh.plan.at[kAttnThreads];
  const int64_t share = share_size(total, gridDim.x);
  int64_t unit = blockIdx.x * share;
  const int64_t end = min(unit + share, total);
  if (t == 0) a.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (unit >= end) return;
  AttnItem it = locate<kAttnRows, kAttnTile, kItemCost>(a, sh.plan, unit);

  while (unit < end) {
    const AttnSeq<kAttnTile> seq(a, it.seq);
    const int rows_left = seq.queries * static_cast<int>(a.group.div) - it.rb * kAttnRows;
    const int rows = min(rows_left, kAttnRows);
    const int steps = static_cast<int>(min(static_cast<int64_t>(seq.tiles - it.tile), end - unit));

    // Q's rows as fragments: eight threads a row, each DIM / 8 elements
    {
      const int r = t / 8, part = t % 8;
      constexpr int N = DIM / 8;
      float x[N], top = 0.0f;
      const int row = it.rb * kAttnRows + r;
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
      if (part == 0)
        sh.row_scale[r] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
#pragma unroll
      for (int i = 0; i < N; i++) {
        const int d = part * N + i;
        constexpr int P = L::kPieceK;
        const int k = d / (4 * P) * (P / 4) + d % P / 4, lc = d % (4 * P) / P, sub = d % 4;
        const int at = ((r % 8) * 4 + lc) * 8 + ((sub / 2) * 2 + r / 8) * 2 + sub % 2;  // halves
        const float v = x[i] * up;
        const __half hi = __float2half_rn(v);
        reinterpret_cast<__half*>(sh.q[0][k])[at] = hi;
        if (SPLIT == 2)
          reinterpret_cast<__half*>(sh.q[SPLIT - 1][k])[at] = __float2half_rn(v - __half2float(hi));
      }
    }
    __syncthreads();
    const float rs0 = sh.row_scale[g], rs1 = sh.row_scale[g + 8];
    const int row0 = it.rb * kAttnRows + g;
    const int tok0 = a.group.quot(row0), tok1 = a.group.quot(row0 + 8);

    float o[L::kTilesV][4];
#pragma unroll
    for (int j = 0; j < L::kTilesV; j++) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    float m0 = -__builtin_huge_valf(), m1 = m0, l0 = 0.0f, l1 = 0.0f;
    // A row's weights are held relative to the largest V scale that it has met, as a power of two
    // (so that a step's result does not depend on it but where weights leave f16's range).
    float vref0 = 0.0f, vref1 = 0.0f;

    // --- the pipeline's stages
    const unsigned char* kc = a.side[0].codes + it.head * L::kCodeRow;
    const unsigned char* vc = a.side[1].codes + it.head * L::kCodeRow;
    const int base0 = it.tile * kAttnTile + warp * kStep;
    auto lookup = [&](int i) {  // the block of position `lane` of step i, or -1
      const int p = base0 + i * kAttnTile + lane;
      if (lane >= kStep || i >= steps || p >= seq.length) return -1;
      const int64_t page = a.page.quot(p);
      if (page >= a.width) return -1;
      const int b = a.table[it.seq * a.width + page];
      return b >= 0 && b < a.blocks ? b : -1;
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
        if (block >= 0) {
          const int64_t in = p - static_cast<int64_t>(a.page.quot(p)) * a.page.div;
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
      return __all_sync(0xFFFFFFFFu, lane >= kStep || (block >= 0 && p < seq.context));
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

      float s[2][4];
#pragma unroll
      for (int n = 0; n < 2; n++) {
        s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
        for (int q = 0; q < L::kStepsK; q++) {
          uint32_t b0, b1;
          if constexpr (!FP4) {
            b0 = half2_of_e4m3(k[n].w[q]);
            b1 = half2_of_e4m3(k[n].w[q] >> 16);
          } else {
            uint32_t h[4];
            half2_of_e2m1(k[n].w[q / 2], h);
            const uint32_t f = sh.km[warp][8 * n + g][L::k_dim(0, q) / 32 +
                                                     (L::kPieceK == 32 ? c : c / 2)] *
                               0x10001u;
            b0 = mul_half2(h[q % 2 * 2], f);
            b1 = mul_half2(h[q % 2 * 2 + 1], f);
          }
          mma_f16(s[n], sh.q[0][q][lane], b0, b1);
          if (SPLIT == 2) mma_f16(s[n], sh.q[SPLIT - 1][q][lane], b0, b1);
        }
      }
      if (more) load_k(i + 1);

      // scores in units of log2
      float mx0 = m0, mx1 = m1;
      float2 sv[2];
#pragma unroll
      for (int n = 0; n < 2; n++) {
        const float2 sk = *reinterpret_cast<const float2*>(&sh.ks[warp][8 * n + 2 * c]);
        sv[n] = *reinterpret_cast<const float2*>(&sh.vs[warp][8 * n + 2 * c]);
        s[n][0] *= sk.x * rs0;
        s[n][1] *= sk.y * rs0;
        s[n][2] *= sk.x * rs1;
        s[n][3] *= sk.y * rs1;
      }
      uint32_t hidden = 0;  // bit 4 n + e: not seen
      if (!was_clean) {
#pragma unroll
        for (int n = 0; n < 2; n++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const int p = base0 + i * kAttnTile + 8 * n + 2 * c + e;
            const bool there = sh.at[warp][i & 1][8 * n + 2 * c + e] >= 0;
            if (!(there && row0 < it.rb * kAttnRows + rows && attn_sees(a, seq, tok0, p))) {
              hidden |= 1u << (4 * n + e);
              s[n][e] = -__builtin_huge_valf();
            }
            if (!(there && row0 + 8 < it.rb * kAttnRows + rows && attn_sees(a, seq, tok1, p))) {
              hidden |= 1u << (4 * n + 2 + e);
              s[n][2 + e] = -__builtin_huge_valf();
            }
          }
      }
#pragma unroll
      for (int n = 0; n < 2; n++) {
        mx0 = fmaxf(mx0, fmaxf(s[n][0], s[n][1]));
        mx1 = fmaxf(mx1, fmaxf(s[n][2], s[n][3]));
      }
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
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
        for (int n = 0; n < 2; n++) {
          const float x = scale_reference(sv[n].x), y = scale_reference(sv[n].y);
          if (!(hidden >> (4 * n) & 1u)) vt0 = fmaxf(vt0, x);
          if (!(hidden >> (4 * n + 1) & 1u)) vt0 = fmaxf(vt0, y);
          if (!(hidden >> (4 * n + 2) & 1u)) vt1 = fmaxf(vt1, x);
          if (!(hidden >> (4 * n + 3) & 1u)) vt1 = fmaxf(vt1, y);
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
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
        for (int j = 0; j < L::kTilesV; j++) {
          o[j][0] *= f0;
          o[j][1] *= f0;
          o[j][2] *= f1;
          o[j][3] *= f1;
        }
        m0 = mx0;
        m1 = mx1;
        vref0 = vt0;
        vref1 = vt1;
      }
      const float winv0 = kWeightUp * power_reciprocal(vref0);
      const float winv1 = kWeightUp * power_reciprocal(vref1);
      float w[2][4];
#pragma unroll
      for (int n = 0; n < 2; n++) {
#pragma unroll
        for (int e = 0; e < 4; e++) w[n][e] = attn_exp2(s[n][e] - (e < 2 ? use0 : use1));
        l0 += w[n][0] + w[n][1];
        l1 += w[n][2] + w[n][3];
        w[n][0] *= sv[n].x * winv0;
        w[n][1] *= sv[n].y * winv0;
        w[n][2] *= sv[n].x * winv1;
        w[n][3] *= sv[n].y * winv1;
        if (!was_clean) {
#pragma unroll
          for (int e = 0; e < 4; e++)
            if (hidden >> (4 * n + e) & 1u) w[n][e] = 0.0f;  // whatever its scale
        }
      }
      uint4 p[SPLIT];
      p[0] = make_uint4(half2_of(w[0][0], w[0][1]), half2_of(w[0][2], w[0][3]),
                        half2_of(w[1][0], w[1][1]), half2_of(w[1][2], w[1][3]));
      if (SPLIT == 2) {
        const uint32_t hi[4] = {p[0].x, p[0].y, p[0].z, p[0].w};
        uint32_t lo[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float2 f = floats_of_half2(hi[e]);
          lo[e] = half2_of(w[e / 2][e % 2 * 2] - f.x, w[e / 2][e % 2 * 2 + 1] - f.y);
        }
        p[SPLIT - 1] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }

      // the second product: pairs of positions of one dimension
      const uint4 seen =
          make_uint4((hidden & 1 ? 0u : 0x3C00u) | (hidden & 2 ? 0u : 0x3C000000u),
                     (hidden & 4 ? 0u : 0x3C00u) | (hidden & 8 ? 0u : 0x3C000000u),
                     (hidden & 16 ? 0u : 0x3C00u) | (hidden & 32 ? 0u : 0x3C000000u),
                     (hidden & 64 ? 0u : 0x3C00u) | (hidden & 128 ? 0u : 0x3C000000u));
      auto product = [&](int j, uint32_t b0, uint32_t b1) {
        if (!was_clean) {
          // A NaN of V reaches those who see its position and nobody else: it leaves the
          // product (0 * NaN is a NaN), and is counted.
          auto nan_halves = [](uint32_t h) {
            return ((h & 0x7FFFu) > 0x7C00u ? 0xFFFFu : 0u) |
                   ((h & 0x7FFF0000u) > 0x7C000000u ? 0xFFFF0000u : 0u);
          };
          const uint32_t n0 = nan_halves(b0), n1 = nan_halves(b1);
          if (__any_sync(0xFFFFFFFFu, (n0 | n1) != 0)) {
            float count[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_f16(count, seen, n0 & 0x3C003C00u, n1 & 0x3C003C00u);
            b0 &= ~n0;
            b1 &= ~n1;
#pragma unroll
            for (int e = 0; e < 4; e++)
              if (count[e] > 0.0f) o[j][e] = __uint_as_float(0x7FC00000u);
          }
        }
        mma_f16(o[j], p[0], b0, b1);
        if (SPLIT == 2) mma_f16(o[j], p[SPLIT - 1], b0, b1);
      };
      if constexpr (!FP4) {
#pragma unroll
        for (int q = 0; q < L::kTilesV / 4; q++) {
#pragma unroll
          for (int h = 0; h < 2; h++) {
            const uint32_t x = __byte_perm(v[0].w[q], v[1].w[q], h ? 0x7362 : 0x5140);
            const uint32_t y = __byte_perm(v[2].w[q], v[3].w[q], h ? 0x7362 : 0x5140);
            product(4 * q + 2 * h, half2_of_e4m3(x), half2_of_e4m3(y));
            product(4 * q + 2 * h + 1, half2_of_e4m3(x >> 16), half2_of_e4m3(y >> 16));
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
          uint32_t x[4], y[4];
          auto even = [](uint32_t lo, uint32_t hi) {
            return (lo & 0x0F0F0F0Fu) | (hi & 0x0F0F0F0Fu) << 4;
          };
          auto odd = [](uint32_t lo, uint32_t hi) {
            return (lo >> 4 & 0x0F0F0F0Fu) | (hi & 0xF0F0F0F0u);
          };
          half2_of_e2m1(even(v[0].w[q], v[1].w[q]), x);
          half2_of_e2m1(even(v[2].w[q], v[3].w[q]), y);
#pragma unroll
          for (int h = 0; h < 4; h++) product(8 * q + 2 * h, mul_half2(x[h], f0), mul_half2(y[h], f1));
          half2_of_e2m1(odd(v[0].w[q], v[1].w[q]), x);
          half2_of_e2m1(odd(v[2].w[q], v[3].w[q]), y);
#pragma unroll
          for (int h = 0; h < 4; h++)
            product(8 * q + 2 * h + 1, mul_half2(x[h], f0), mul_half2(y[h], f1));
        }
      }
      if (more) load_v(i + 1);
      __syncwarp();  // the step's scales are read until here
    }

    // --- the warps' results joined, in order
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, d);
      l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, d);
    }
    if (c == 0) {
      sh.m[warp][g] = m0;
      sh.m[warp][g + 8] = m1;
      sh.l[warp][g] = l0;
      sh.l[warp][g + 8] = l1;
    }
    __syncthreads();
    float top0 = sh.m[0][g], top1 = sh.m[0][g + 8];
#pragma unroll
    for (int w = 1; w < kAttnWarps; w++) {
      top0 = fmaxf(top0, sh.m[w][g]);
      top1 = fmaxf(top1, sh.m[w][g + 8]);
    }
    const float f0 = m0 == -__builtin_huge_valf() ? 0.0f : attn_exp2(m0 - top0);
    const float f1 = m1 == -__builtin_huge_valf() ? 0.0f : attn_exp2(m1 - top1);
    const float back0 = vref0 * (1.0f / kWeightUp), back1 = vref1 * (1.0f / kWeightUp);
#pragma unroll
    for (int j = 0; j < L::kTilesV; j++) {
      const int d0 = L::v_dim(2 * c, j), d1 = L::v_dim(2 * c + 1, j);
      sh.o[warp][g][d0] = o[j][0] * back0 * f0;
      sh.o[warp][g][d1] = o[j][1] * back0 * f0;
      sh.o[warp][g + 8][d0] = o[j][2] * back1 * f1;
      sh.o[warp][g + 8][d1] = o[j][3] * back1 * f1;
    }
    if (t < kAttnRows) {
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
                  (2 * static_cast<int64_t>(blockIdx.x) + (from_start ? 1 : 0)) * kAttnRows * (DIM + 2);
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
        const int row = it.rb * kAttnRows + r;
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
          part[kAttnRows * DIM + 2 * r] = sh.top[r];
          part[kAttnRows * DIM + 2 * r + 1] = sum;
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
    next_item<kAttnRows, kAttnTile>(a, it, seq.queries);
  }
}

template <typename T, bool FP4, int DIM>
cudaError_t attn_go(AttnArgs a, void* workspace, cudaStream_t s) {
  constexpr size_t shared = sizeof(AttnShared<T, FP4, DIM>);
  constexpr unsigned shares = kSms * attn_blocks<DIM>;
  static std::atomic<int> done[64], done_join[64];
  cudaError_t e = allow_shared(cache_attention_kernel<T, FP4, DIM>, shared, done);
  if (e == cudaSuccess) e = allow_shared(cache_attention_join_kernel<T, kAttnRows, DIM>, 0, done_join);
  if (e != cudaSuccess) return e;
  a.joins = static_cast<int4*>(workspace);
  a.partial = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) +
                                       attn_joins_bytes(shares));
  e = launch_pdl(cache_attention_kernel<T, FP4, DIM>, dim3(shares), dim3(kAttnThreads), shared, s,
                 a);
  if (e != cudaSuccess) return e;
  return launch_pdl(cache_attention_join_kernel<T, kAttnRows, DIM>,
                    dim3(shares, kAttnRows / kJoinRows), dim3(DIM / 4, kJoinRows), 0, s, a);
}

template <typename T, bool FP4>
cudaError_t attn_dim(int64_t dim, const AttnArgs& a, void* ws, cudaStream_t s) {
  if (dim == 64) return attn_go<T, FP4, 64>(a, ws, s);
  if (dim == 128) return attn_go<T, FP4, 128>(a, ws, s);
  return attn_go<T, FP4, 256>(a, ws, s);
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
  const int64_t shares = kSms * (head_dim == 256 ? attn_blocks<256> : attn_blocks<128>);
  const int64_t few = attn_bytes(shares, kAttnRows, head_dim), many = attn_rows_bytes(head_dim);
  return few > many ? few : many;
}

cudaError_t launch_cache_attention(const KvCacheArgs& c, const CacheAttentionArgs& p, int is_bf16,
                                   cudaStream_t stream) {
  const AttnArgs a = attn_args(c, p);
  // More than 16 rows an item on average: the kernel whose tile of products has 128.
  if (is_bf16 && c.head_dim <= 128 && p.tokens * (p.q_heads / c.heads) > kAttnRows * p.seqs)
    return launch_attn_rows(a, c.fp4, c.head_dim, p.workspace, stream);
  if (is_bf16)
    return c.fp4 ? attn_dim<__nv_bfloat16, true>(c.head_dim, a, p.workspace, stream)
                 : attn_dim<__nv_bfloat16, false>(c.head_dim, a, p.workspace, stream);
  return c.fp4 ? attn_dim<float, true>(c.head_dim, a, p.workspace, stream)
               : attn_dim<float, false>(c.head_dim, a, p.workspace, stream);
}

}  // namespace nr
