// Q/K RMSNorm + rotary embedding with K and V going straight into the
// quantised paged cache, for sm_103a.
//
// Per token: q_out = rope(norm(q)) rounded once to its storage type; the same
// of K and the plain V are quantised from their f32 values, never rounded in
// between, so K is read once and only its codes are written.  Against the
// two-call form (norm + rope, then the cache write) this saves writing and
// re-reading K.
//
// Design.  A token's head rows (Q, then K, then V) are one list, cut into
// items of whole warp passes; a warp takes items w, w + W, ... and works on its
// own: it copies its rows RING passes ahead into a ring of its own (cp.async),
// computes an item's angles once into a table of its own, and no block barrier
// follows the set-up.  A group of L lanes owns one head row, a lane the two
// vectors that rotate into one another; the arithmetic is on pairs of f32
// values.  Calls of many tokens take whole tokens as items; small ones cut them
// until every warp has work.  Angles are the exact turns of the Q/K kernels.
//
// At [26598, 24 + 24 + 24, 128] bf16 -> fp8 a block of four warps with bulk-copy
// stages and one barrier an item took 166 us (whole tokens) to 307 us (items
// of a third): about 2 us an item whatever its rows, in the chain from the
// barrier through the angles to the next barrier.
#include <type_traits>

#include "quant.cuh"

namespace nr {
namespace {

constexpr int kFusedThreads = 128;
constexpr int kFusedWarps = kFusedThreads / kWarp;
// Passes in flight of a warp: 3, 5 and 8 ran [26598, 24 + 24 + 24, 128] in 135,
// 133 and 133 us (129.0 us, 0.94 of the measured copy rate, with row addresses
// formed per token and not per pass).
constexpr int kRing = 5;
constexpr int kFusedPerSm = 4;  // resident blocks (three: 144 us)

struct FusedArgs {
  void* q_out;
  const void* q;
  const void* k;
  const void* v;
  const void* wq;
  const void* wk;
  const int32_t* pos;
  const int64_t* slots;
  CacheSide side[2];
  CacheGeom geo;
  int64_t tokens;
  int64_t q_stride, k_stride, v_stride;
  int hq, hk;
  int chunk;  // rows of an item
  int items;  // items of a token
  float eps, inv_d, w_add;
  int rot_vec, interleaved, mrope;
};

__device__ __forceinline__ float weight_of(const float* w, int i) { return w[i]; }
__device__ __forceinline__ float weight_of(const __nv_bfloat16* w, int i) {
  return __bfloat162float(w[i]);
}

template <typename T, int L>
struct FusedSmem {
  static constexpr int N = Vec<T>::N;
  static constexpr int HALF = L * N;
  static constexpr int D = 2 * HALF;
  // a warp: ring of two vectors a lane, angle table (cos, sin); a block: turns, axes
  static constexpr int kWarpBytes =
      kRing * kWarp * 2 * static_cast<int>(sizeof(uint4)) + HALF * static_cast<int>(sizeof(float2));
  static constexpr int kBytes = kFusedWarps * kWarpBytes +
                                HALF * static_cast<int>(sizeof(unsigned long long)) + HALF;
};

// GEN: partial rotation, GPT-J pairs and M-RoPE, chosen at run time.
template <typename T, typename WT, int L, bool FP4, bool GEN>
__global__ void __launch_bounds__(kFusedThreads, kFusedPerSm)
    qk_cache_kernel(const FusedArgs a, const RopeTurns turns) {
  using S = FusedSmem<T, L>;
  constexpr int N = S::N, P = N / 2;
  constexpr int HALF = S::HALF;
  constexpr int D = S::D;
  constexpr int GW = kWarp / L;               // head rows of a pass
  constexpr int W = 32 / N < L ? 32 / N : L;  // lanes of one 32-element group

  extern __shared__ __align__(16) unsigned char smem[];
  const int warp = threadIdx.x / kWarp, lane32 = threadIdx.x % kWarp;
  uint4* ring = reinterpret_cast<uint4*>(smem + warp * S::kWarpBytes) + lane32;  // [kRing][2][32]
  float2* table = reinterpret_cast<float2*>(smem + warp * S::kWarpBytes +
                                            kRing * kWarp * 2 * sizeof(uint4));
  unsigned long long* turn_sm =
      reinterpret_cast<unsigned long long*>(smem + kFusedWarps * S::kWarpBytes);
  unsigned char* axis_sm = reinterpret_cast<unsigned char*>(turn_sm + HALF);
  for (int i = threadIdx.x; i < HALF; i += kFusedThreads) {
    turn_sm[i] = turns.turn[i];
    if (GEN) axis_sm[i] = turns.axis[i];
  }
  __syncthreads();  // the only block-level barrier
  pdl_enter();      // before any global read: the previous kernel may still run

  const int g = lane32 / L, l = lane32 % L;
  // The two vectors of this lane: rotate-half partners, the halves of what is
  // not rotated, or (GPT-J pairs, which lie inside a vector) l and l + L.
  int va = l, vb = l + L;
  bool rotates = true;
  if (GEN && !a.interleaved) {
    const int half_rot = a.rot_vec / 2;
    if (l < half_rot) {
      vb = l + half_rot;
    } else {
      va = a.rot_vec + l - half_rot;
      vb = va + L - half_rot;
      rotates = false;
    }
  }
  const int rows = a.hq + 2 * a.hk;

  // An item: its token and first row.  A cursor walks this warp's items pass by pass.
  struct Cursor {
    int64_t tok;
    int row, end;  // next pass's first row, end of the item's rows
    int c;         // item of the token
  };
  const int64_t W_items = static_cast<int64_t>(gridDim.x) * kFusedWarps;
  const int64_t step_tok = W_items / a.items;
  const int step_c = static_cast<int>(W_items % a.items);
  auto open = [&](Cursor& u) {
    u.row = u.c * a.chunk;
    u.end = min(u.row + a.chunk, rows);
  };
  auto next_item = [&](Cursor& u) {
    u.tok += step_tok;
    u.c += step_c;
    if (u.c >= a.items) {
      u.c -= a.items;
      u.tok++;
    }
    open(u);
  };
  Cursor cur;
  {
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kFusedWarps + warp;
    cur.tok = first / a.items;
    cur.c = static_cast<int>(first - cur.tok * a.items);
    open(cur);
  }
  if (cur.tok >= a.tokens) return;
  Cursor cp = cur;
  // Where the copy cursor's token has its rows, each list as if it began at row 0.
  const T *pq, *pk, *pv;
  auto sources = [&]() {
    pq = static_cast<const T*>(a.q) + cp.tok * a.q_stride;
    pk = static_cast<const T*>(a.k) + cp.tok * a.k_stride - a.hq * D;
    pv = static_cast<const T*>(a.v) + cp.tok * a.v_stride - (a.hq + a.hk) * D;
  };
  sources();
  // Starts the copies of the copy cursor's pass into a ring slot, one group.
  auto issue = [&](int slot) {
    if (cp.tok < a.tokens) {
      const int row = cp.row + g;
      if (row < cp.end) {
        const T* p = (row < a.hq ? pq : row < a.hq + a.hk ? pk : pv) + row * D;
        cp_async16(smem_addr(ring + slot * 2 * kWarp), p + va * N);
        cp_async16(smem_addr(ring + (slot * 2 + 1) * kWarp), p + vb * N);
      }
      cp.row += GW;
      if (cp.row >= cp.end) {
        next_item(cp);
        sources();
      }
    }
    cp_async_commit();  // possibly empty: keeps one group a pass
  };
  for (int s = 0; s < kRing; s++) issue(s);

  // This lane's weights.
  F2 wqa[P], wqb[P], wka[P], wkb[P];
  {
    const WT* wq = static_cast<const WT*>(a.wq);
    const WT* wk = static_cast<const WT*>(a.wk);
    auto get = [&](const WT* w, int vec, F2 (&o)[P]) {
#pragma unroll
      for (int i = 0; i < P; i++) {
        const int e = vec * N + 2 * i;
        o[i] = f2(weight_of(w, e) + a.w_add, weight_of(w, e + 1) + a.w_add);
      }
    };
    get(wq, va, wqa);
    get(wq, vb, wqb);
    get(wk, va, wka);
    get(wk, vb, wkb);
  }

  // Position and slot of an item's token, loaded one item ahead.
  constexpr int NPOS = GEN ? 3 : 1;
  int pos[NPOS];
  int64_t slot_of_token = -1;
  auto fetch = [&](const Cursor& u) {
    slot_of_token = -1;
    if (u.tok < a.tokens) {
      slot_of_token = a.slots[u.tok];
#pragma unroll
      for (int ax = 0; ax < NPOS; ax++)
        pos[ax] = (ax == 0 || a.mrope) ? a.pos[ax * a.tokens + u.tok] : 0;
    }
  };
  fetch(cur);
  const int pairs = GEN ? a.rot_vec * N / 2 : HALF;

  int slot = 0;
  while (cur.tok < a.tokens) {
    // A new item: its angles, once a warp, then this lane's; its place in the
    // cache (a slot outside it keeps nothing).
    __syncwarp();
    for (int i = lane32; i < pairs; i += kWarp) {
      long long p = pos[0];
      if (GEN && a.mrope) {
        if (axis_sm[i] == 1) p = pos[NPOS > 1 ? 1 : 0];
        if (axis_sm[i] == 2) p = pos[NPOS > 2 ? 2 : 0];
      }
      // the angle in turns, mod 1, times 2^32: exact for any int32 position
      const unsigned long long prod = static_cast<unsigned long long>(p) * turn_sm[i];
      // The nearest quarter turn comes off before the conversion to 24 bits, which
      // then round an eighth of a turn and not a half: K's codes are made from the
      // f32 value, with no bf16 rounding to hide the angle's.  At [26598, 24, 128],
      // eight inputs, 1118 of 654 million e4m3 codes of K differ from those of exact
      // values (1108 with cosines rounded once from 64 bits, 1921 with an angle
      // rounded over half a turn), for 0.4 us of the 129.0.
      const unsigned t = static_cast<unsigned>(prod >> 32) + (1u << 29);
      const int rest = static_cast<int>(t & 0x3FFFFFFFu) - (1 << 29);  // of quarter t >> 30
      float sn, cn;
      sincospif(static_cast<float>(rest) * 0x1p-31f, &sn, &cn);
      const bool odd = (t & 0x40000000u) != 0;
      // cos is negative in quarters 1 and 2, sin in 2 and 3
      table[i] = make_float2(
          __uint_as_float(__float_as_uint(odd ? sn : cn) ^ ((t + 0x40000000u) & 0x80000000u)),
          __uint_as_float(__float_as_uint(odd ? cn : sn) ^ (t & 0x80000000u)));
    }
    __syncwarp();
    // rotate-half: cos and sin of the lane's N pairs; GPT-J: of the pairs inside
    // its two vectors, N / 2 each
    F2 co[P], si[P];
    if (!GEN || !a.interleaved) {
      if (rotates) {
#pragma unroll
        for (int i = 0; i < P; i++) {
          const float2 x = table[l * N + 2 * i], y = table[l * N + 2 * i + 1];
          co[i] = f2(x.x, y.x);
          si[i] = f2(x.y, y.y);
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < P; h++) {  // co[h]: (cos, sin) in va, si[h]: in vb
        if (va < a.rot_vec) co[h] = f2(table[va * P + h].x, table[va * P + h].y);
        if (vb < a.rot_vec) si[h] = f2(table[vb * P + h].x, table[vb * P + h].y);
      }
    }
    const bool kept = slot_of_token >= 0 && slot_of_token < a.geo.slots;
    int64_t code_off = 0, scale_off = 0;
    if (kept) {
      const int64_t block = a.geo.block_of(slot_of_token);
      const int64_t place = slot_of_token - block * a.geo.block_size;
      code_off = block * a.geo.code_block_stride + place * a.geo.code_row;
      scale_off = block * a.geo.scale_block_stride + place * a.geo.scale_row;
    }
    T* const q_row = static_cast<T*>(a.q_out) + cur.tok * a.q_stride;
    Cursor after = cur;
    next_item(after);
    fetch(after);

    // One pass of GW rows.  KIND 0: all Q, 1: all K, 2: all V, 3: any mix, or
    // past the last row (those lanes still join the shuffles).
    auto pass = [&](auto kind, int first) {
      constexpr int KIND = decltype(kind)::value;
      const int row = first + g;
      const bool valid = KIND != 3 || row < cur.end;
      const bool is_q = KIND == 0 || (KIND == 3 && row < a.hq);
      const bool is_v = KIND == 2 || (KIND == 3 && row >= a.hq + a.hk);
      F2 xa[P], xb[P];
      if (valid) {
        Pairs<T>::unpack(lds128(ring + slot * 2 * kWarp), xa);
        Pairs<T>::unpack(lds128(ring + (slot * 2 + 1) * kWarp), xb);
      } else {
#pragma unroll
        for (int i = 0; i < P; i++) xa[i] = xb[i] = f2(0.0f, 0.0f);
      }
      if (KIND != 2) {
        F2 sq = mul2(xa[0], xa[0]);
#pragma unroll
        for (int i = 1; i < P; i++) sq = fma2(xa[i], xa[i], sq);
#pragma unroll
        for (int i = 0; i < P; i++) sq = fma2(xb[i], xb[i], sq);
        float s0, s1;
        split(sq, s0, s1);
        const float ss = group_sum<L>(s0 + s1);
        if (KIND != 3 || !is_v) {
          const float inv = rsqrtf(fmaf(ss, a.inv_d, a.eps));
          const F2 inv2 = f2(inv, inv);
#pragma unroll
          for (int i = 0; i < P; i++) {
            const bool q_row = KIND == 0 || (KIND == 3 && is_q);
            xa[i] = mul2(mul2(xa[i], inv2), KIND == 3 ? (q_row ? wqa[i] : wka[i])
                                                      : KIND == 0 ? wqa[i] : wka[i]);
            xb[i] = mul2(mul2(xb[i], inv2), KIND == 3 ? (q_row ? wqb[i] : wkb[i])
                                                      : KIND == 0 ? wqb[i] : wkb[i]);
          }
          if (!GEN || (!a.interleaved && rotates)) {
#pragma unroll
            for (int i = 0; i < P; i++) {
              const F2 na = xa[i], nb = xb[i];
              xa[i] = sub2(mul2(na, co[i]), mul2(nb, si[i]));
              xb[i] = fma2(na, si[i], mul2(nb, co[i]));
            }
          } else if (a.interleaved) {
#pragma unroll
            for (int h = 0; h < P; h++) {
              auto turn = [](F2& x, F2 cs) {
                float x0, x1, c, s;
                split(x, x0, x1);
                split(cs, c, s);
                x = f2(fmaf(x0, c, -x1 * s), fmaf(x0, s, x1 * c));
              };
              if (va < a.rot_vec) turn(xa[h], co[h]);
              if (vb < a.rot_vec) turn(xb[h], si[h]);
            }
          }
        }
      }
      if (KIND == 0 || (KIND == 3 && is_q && valid)) {
        T* o = q_row + row * D;
        st_stream(o + va * N, Pairs<T>::pack(xa));
        st_stream(o + vb * N, Pairs<T>::pack(xb));
      }
      if (KIND == 0) return;
      const int head = row - a.hq - (is_v ? a.hk : 0);
      const CacheSide side = is_v ? a.side[1] : a.side[0];
      const bool write = kept && valid && !is_q;
      float fa[N], fb[N];
      if constexpr (!FP4) {
        from_pairs<P>(xa, fa);
        from_pairs<P>(xb, fb);
        const float top = clamp_scale(group_max<L>(fmaxf(max_abs(fa), max_abs(fb))));
        if (!write) return;
        const float inv = fp8_inverse(top);
        const F2 inv2 = f2(inv, inv);
#pragma unroll
        for (int i = 0; i < P; i++) {
          xa[i] = mul2(xa[i], inv2);
          xb[i] = mul2(xb[i], inv2);
        }
        from_pairs<P>(xa, fa);
        from_pairs<P>(xb, fb);
        unsigned char* o = side.codes + code_off + head * D;
        uint32_t ca[N / 4], cb[N / 4];
        fp8_codes_scaled(fa, ca);
        fp8_codes_scaled(fb, cb);
        if constexpr (N == 8) {
          st_stream8(o + va * N, make_uint2(ca[0], ca[N / 4 - 1]));
          st_stream8(o + vb * N, make_uint2(cb[0], cb[N / 4 - 1]));
        } else {
          st_stream4(o + va * N, ca[0]);
          st_stream4(o + vb * N, cb[0]);
        }
        if (l == 0) reinterpret_cast<float*>(side.scales + scale_off)[head] = fp8_scale(top);
      } else {
        from_pairs<P>(xa, fa);
        from_pairs<P>(xb, fb);
        const uint32_t ba = mx_scale_byte(clamp_scale(group_max<W>(max_abs(fa))));
        const uint32_t bb = mx_scale_byte(clamp_scale(group_max<W>(max_abs(fb))));
        if (!write) return;
        unsigned char* o = side.codes + code_off + head * (D / 2);
        unsigned char* s = side.scales + scale_off + head * (D / 32);
        const uint32_t ca = fp4_codes(fa, mx_inverse(ba)), cb = fp4_codes(fb, mx_inverse(bb));
        if constexpr (N == 8) {
          st_stream4(o + va * 4, ca);
          st_stream4(o + vb * 4, cb);
        } else {
          *reinterpret_cast<uint16_t*>(o + va * 2) = static_cast<uint16_t>(ca);
          *reinterpret_cast<uint16_t*>(o + vb * 2) = static_cast<uint16_t>(cb);
        }
        if (va % W == 0) {  // vb lies at the same place of its group
          s[va / W] = static_cast<unsigned char>(ba);
          s[vb / W] = static_cast<unsigned char>(bb);
        }
      }
    };
    for (int first = cur.row; first < cur.end; first += GW) {  // warp-uniform
      cp_async_wait<kRing - 1>();  // this pass's group has landed
      const int last = first + GW;
      if (last <= cur.end && last <= a.hq)
        pass(std::integral_constant<int, 0>(), first);
      else if (last <= cur.end && first >= a.hq && last <= a.hq + a.hk)
        pass(std::integral_constant<int, 1>(), first);
      else if (last <= cur.end && first >= a.hq + a.hk)
        pass(std::integral_constant<int, 2>(), first);
      else
        pass(std::integral_constant<int, 3>(), first);
      issue(slot);  // the slot's values have been used
      slot = slot + 1 == kRing ? 0 : slot + 1;
    }
    cur = after;
  }
  cp_async_wait<0>();  // nothing may land after the block's shared memory is released
}

// Warps that reside on the GPU: an SM holds four blocks (128 registers a thread).
constexpr int64_t kFusedResident = 152 * kFusedPerSm;

template <typename T, typename WT, int L, bool FP4, bool GEN>
cudaError_t fused_launch(FusedArgs& a, const RopeTurns& turns, cudaStream_t s) {
  constexpr int GW = kWarp / L;
  constexpr int smem = FusedSmem<T, L>::kBytes;
  auto kernel = qk_cache_kernel<T, WT, L, FP4, GEN>;
  static_assert(smem <= 48 * 1024, "no opt-in to more shared memory is needed");
  // Whole tokens from four rounds of every warp on; below that they are cut.
  const int rows = a.hq + 2 * a.hk;
  const int passes = (rows + GW - 1) / GW;
  constexpr int64_t warps = kFusedResident * kFusedWarps;
  int64_t items = (4 * warps + a.tokens - 1) / a.tokens;
  items = items < passes ? items : passes;
  const int per = static_cast<int>((passes + items - 1) / items);  // passes of an item
  a.chunk = per * GW;
  a.items = (passes + per - 1) / per;
  const int64_t blocks = (a.tokens * a.items + kFusedWarps - 1) / kFusedWarps;
  return launch_pdl(kernel,
                    dim3(static_cast<unsigned>(blocks < kFusedResident ? blocks : kFusedResident)),
                    dim3(kFusedThreads), smem, s, a, turns);
}

template <typename T, typename WT, int L>
cudaError_t fused_l(FusedArgs& a, bool fp4, const RopeTurns& turns, cudaStream_t s) {
  const bool gen = a.rot_vec != 2 * L || a.interleaved || a.mrope;
  if (fp4)
    return gen ? fused_launch<T, WT, L, true, true>(a, turns, s)
               : fused_launch<T, WT, L, true, false>(a, turns, s);
  return gen ? fused_launch<T, WT, L, false, true>(a, turns, s)
             : fused_launch<T, WT, L, false, false>(a, turns, s);
}

template <typename T, typename WT>
cudaError_t fused_w(FusedArgs& a, bool fp4, int lanes, const RopeTurns& turns, cudaStream_t s) {
  switch (lanes) {
    case 4: return fused_l<T, WT, 4>(a, fp4, turns, s);
    case 8: return fused_l<T, WT, 8>(a, fp4, turns, s);
    case 16: return fused_l<T, WT, 16>(a, fp4, turns, s);
    case 32: return fused_l<T, WT, 32>(a, fp4, turns, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope_cache(const KvCacheArgs& c, void* q_out, const void* q,
                                      const void* k, const void* v, const void* wq,
                                      const void* wk, int w_is_bf16, const int32_t* positions,
                                      const int64_t* slots, int64_t tokens, int64_t hq,
                                      int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                      float eps, const RopeTurns& turns, int gemma,
                                      int64_t rotary_dim, int interleaved, int mrope, int is_bf16,
                                      cudaStream_t stream) {
  const int n = is_bf16 ? 8 : 4;
  FusedArgs a;
  a.q_out = q_out;
  a.q = q;
  a.k = k;
  a.v = v;
  a.wq = wq;
  a.wk = wk;
  a.pos = positions;
  a.slots = slots;
  a.side[0] = CacheSide{c.k_codes, c.k_scales};
  a.side[1] = CacheSide{c.v_codes, c.v_scales};
  a.geo = cache_geometry(c);
  a.tokens = tokens;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.hq = static_cast<int>(hq);
  a.hk = static_cast<int>(c.heads);
  a.eps = eps;
  a.inv_d = 1.0f / static_cast<float>(c.head_dim);
  a.w_add = gemma ? 1.0f : 0.0f;
  a.rot_vec = static_cast<int>(rotary_dim / n);
  a.interleaved = interleaved;
  a.mrope = mrope;
  const int lanes = static_cast<int>(c.head_dim / (2 * n));
  if (is_bf16)
    return w_is_bf16 ? fused_w<__nv_bfloat16, __nv_bfloat16>(a, c.fp4, lanes, turns, stream)
                     : fused_w<__nv_bfloat16, float>(a, c.fp4, lanes, turns, stream);
  return w_is_bf16 ? fused_w<float, __nv_bfloat16>(a, c.fp4, lanes, turns, stream)
                   : fused_w<float, float>(a, c.fp4, lanes, turns, stream);
}

}  // namespace nr
