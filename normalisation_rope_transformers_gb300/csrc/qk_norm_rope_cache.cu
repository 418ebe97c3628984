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
// items of `chunk` rows (about 8 KB); an item may span the tensors.  A block
// of four warps takes items b, b + grid, ...: bulk copies bring an item's rows
// (up to three contiguous pieces) into one of NST shared-memory stages ahead
// of time, the warps work on it, Q rows are written back in place and leave by
// one bulk copy, codes and scales leave from registers.  A group of L lanes
// owns one head row, a lane the two vectors that rotate into one another.
// The next item's angles are computed beside the current rows, into the other
// of two tables, with the exact turn arithmetic of the Q/K kernels.  Waits on
// the copies are bounded and report through the device status word.  Small
// items keep many blocks busy for single tokens and fit any number of heads.
#include <atomic>
#include <type_traits>

#include "quant.cuh"

namespace nr {
namespace {

constexpr int kFusedThreads = 128;
constexpr int kFusedWarps = kFusedThreads / kWarp;
constexpr int kStages = 3;
// Bytes of an item: calls of many tokens take whole tokens where they fit (one
// barrier and one angle table for more rows), small calls spread their rows.
constexpr int kItemBytesMany = 20 * 1024;
constexpr int kItemBytesFew = 8 * 1024;
constexpr long long kFusedWaitLimit = 1LL << 31;  // SM cycles, about one second

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
  unsigned stage_bytes;
  float eps, inv_d, w_add;
  int rot_vec, interleaved, mrope;
  unsigned* status;
};

__device__ __forceinline__ float weight_of(const float* w, int i) { return __ldg(w + i); }
__device__ __forceinline__ float weight_of(const __nv_bfloat16* w, int i) {
  return __bfloat162float(w[i]);
}

template <typename T, int L>
struct FusedSmem {
  static constexpr int N = Vec<T>::N;
  static constexpr int HALF = L * N;
  static constexpr int D = 2 * HALF;
  // [kStages stages][2 angle tables of HALF float2][2D weights][HALF turns][mbarriers][flag]
  static size_t bytes(unsigned stage_bytes) {
    return static_cast<size_t>(kStages) * stage_bytes + 2 * HALF * sizeof(float2) +
           2 * D * sizeof(float) + HALF * sizeof(unsigned long long) +
           kStages * sizeof(unsigned long long) + 16;
  }
};

// GEN: partial rotation, GPT-J pairs and M-RoPE, chosen at run time.
template <typename T, typename WT, int L, bool FP4, bool GEN>
__global__ void __launch_bounds__(kFusedThreads) qk_cache_kernel(const FusedArgs a,
                                                                 const RopeTurns turns) {
  using S = FusedSmem<T, L>;
  constexpr int N = S::N;
  constexpr int HALF = S::HALF;
  constexpr int D = S::D;
  constexpr int GW = kWarp / L;           // head rows of a warp pass
  constexpr int W = 32 / N < L ? 32 / N : L;  // lanes of one 32-element group

  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char* stages = smem;
  float2* table = reinterpret_cast<float2*>(stages + kStages * static_cast<size_t>(a.stage_bytes));
  float* wsm = reinterpret_cast<float*>(table + 2 * HALF);
  unsigned long long* turn_sm = reinterpret_cast<unsigned long long*>(wsm + 2 * D);
  unsigned long long* bars = turn_sm + HALF;
  int* abort_flag = reinterpret_cast<int*>(bars + kStages);

  const int tid = threadIdx.x;
  const int warp = tid / kWarp, lane32 = tid % kWarp;
  for (int i = tid; i < HALF; i += kFusedThreads) turn_sm[i] = turns.turn[i];
  if (tid == 0) {
    for (int st = 0; st < kStages; st++) mbar_init(smem_addr(bars + st), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }

  const int rows = a.hq + 2 * a.hk;
  const T* q = static_cast<const T*>(a.q);
  const T* k = static_cast<const T*>(a.k);
  const T* v = static_cast<const T*>(a.v);

  // An item: token and first row.  A block's items are `step` apart.
  struct Item {
    int64_t tok;
    int c;
  };
  const int64_t step_tok = gridDim.x / a.items;
  const int step_c = static_cast<int>(gridDim.x % a.items);
  auto next = [&](Item& it) {
    it.tok += step_tok;
    it.c += step_c;
    if (it.c >= a.items) {
      it.c -= a.items;
      it.tok++;
    }
  };
  Item cur{static_cast<int64_t>(blockIdx.x / a.items), static_cast<int>(blockIdx.x % a.items)};
  Item ahead = cur;  // producer (thread 0): the next item to load
  int64_t issued = 0;
  const uint64_t policy = l2_evict_first_policy();
  auto stage = [&](int64_t j) { return stages + (j % kStages) * static_cast<size_t>(a.stage_bytes); };
  auto issue = [&]() {
    const unsigned bar = smem_addr(bars + issued % kStages);
    unsigned dst = smem_addr(stage(issued));
    const int r0 = ahead.c * a.chunk, r1 = min(r0 + a.chunk, rows);
    mbar_arrive_expect_tx(bar, static_cast<unsigned>((r1 - r0) * D * sizeof(T)));
    auto piece = [&](const T* base, int lo, int hi) {  // rows [lo, hi) of one tensor
      if (hi <= lo) return;
      const unsigned bytes = static_cast<unsigned>((hi - lo) * D * sizeof(T));
      bulk_load_hint(dst, base + static_cast<int64_t>(lo) * D, bytes, bar, policy);
      dst += bytes;
    };
    piece(q + ahead.tok * a.q_stride, r0, min(r1, a.hq));
    piece(k + ahead.tok * a.k_stride, max(r0 - a.hq, 0), min(r1 - a.hq, a.hk));
    piece(v + ahead.tok * a.v_stride, max(r0 - a.hq - a.hk, 0), r1 - a.hq - a.hk);
    issued++;
    next(ahead);
  };
  pdl_enter();  // before any global read: the previous kernel may still run
  if (tid == 0)
    for (int j = 0; j < kStages - 1 && ahead.tok < a.tokens; j++) issue();
  const WT* wq = static_cast<const WT*>(a.wq);
  const WT* wk = static_cast<const WT*>(a.wk);
  for (int i = tid; i < 2 * D; i += kFusedThreads)
    wsm[i] = (i < D ? weight_of(wq, i) : weight_of(wk, i - D)) + a.w_add;

  // This thread's pairs of an item's angle table (threads below the pair count).
  const int pairs = GEN ? a.rot_vec * N / 2 : HALF;
  auto position = [&](const Item& it, int i) -> int {
    return a.pos[(GEN && a.mrope ? turns.axis[i] * a.tokens : 0) + it.tok];
  };
  auto angle = [&](float2* t, int i, int p) {
    const unsigned long long prod = static_cast<unsigned long long>(static_cast<long long>(p)) *
                                    turn_sm[i];
    const int hi = static_cast<int>(prod >> 32);  // signed turn fraction * 2^32
    float sn, cn;
    sincospif(static_cast<float>(hi) * 0x1p-31f, &sn, &cn);
    t[i] = make_float2(cn, sn);
  };
  __syncthreads();  // weights, turns and barriers visible
  Item nxt = cur;
  next(nxt);
  int pos_next = 0;
  int64_t slot = -1;
  if (cur.tok < a.tokens) {
    slot = __ldg(a.slots + cur.tok);
    for (int i = tid; i < pairs; i += kFusedThreads) angle(table, i, position(cur, i));
    if (nxt.tok < a.tokens && tid < pairs) pos_next = position(nxt, tid);
  }
  __syncthreads();

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
  float wqa[N], wqb[N], wka[N], wkb[N];
#pragma unroll
  for (int e = 0; e < N; e++) {
    wqa[e] = wsm[va * N + e];
    wqb[e] = wsm[vb * N + e];
    wka[e] = wsm[D + va * N + e];
    wkb[e] = wsm[D + vb * N + e];
  }

  int64_t j = 0;
  for (; cur.tok < a.tokens; j++) {
    unsigned char* st = stage(j);
    int64_t slot_next = -1;
    if (nxt.tok < a.tokens) slot_next = __ldg(a.slots + nxt.tok);
    if (!mbar_wait_bounded(smem_addr(bars + j % kStages), static_cast<unsigned>((j / kStages) & 1),
                           kFusedWaitLimit)) {
      atomicOr(a.status, kStatusBitCacheBulkWait);
      *abort_flag = 1;
    }
    const float2* tb = table + (j & 1) * HALF;
    float2 cs[N];
    if (!GEN || !a.interleaved) {
      if (rotates) {
#pragma unroll
        for (int e = 0; e < N; e++) cs[e] = tb[l * N + e];
      }
    } else {
#pragma unroll
      for (int h = 0; h < N / 2; h++) {
        if (va < a.rot_vec) cs[h] = tb[va * (N / 2) + h];
        if (vb < a.rot_vec) cs[N / 2 + h] = tb[vb * (N / 2) + h];
      }
    }
    const int r0 = cur.c * a.chunk, r1 = min(r0 + a.chunk, rows);
    // The token's place in the cache; a slot outside it keeps nothing.
    const bool kept = slot >= 0 && slot < a.geo.slots;
    int64_t code_off = 0, scale_off = 0;
    if (r1 > a.hq && kept) {
      const int64_t block = a.geo.block_of(slot);
      const int64_t place = slot - block * a.geo.block_size;
      code_off = block * a.geo.code_block_stride + place * a.geo.code_row;
      scale_off = block * a.geo.scale_block_stride + place * a.geo.scale_row;
    }

    // One pass of GW rows.  KIND 0: all Q, 1: all K, 2: all V, 3: any mix, or
    // past the last row (those lanes still join the shuffles).
    auto pass = [&](auto kind, int first) {
      constexpr int KIND = decltype(kind)::value;
      const int row = first + g;
      const bool valid = KIND != 3 || row < r1;
      const bool is_q = KIND == 0 || (KIND == 3 && row < a.hq);
      const bool is_v = KIND == 2 || (KIND == 3 && row >= a.hq + a.hk);
      uint4* r = reinterpret_cast<uint4*>(st + static_cast<size_t>(valid ? row - r0 : 0) * D *
                                                   sizeof(T));
      float xa[N], xb[N];
      Vec<T>::unpack(r[va], xa);
      Vec<T>::unpack(r[vb], xb);
      if (KIND != 2) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < N; e++) {
          ss = fmaf(xa[e], xa[e], ss);
          ss = fmaf(xb[e], xb[e], ss);
        }
        ss = group_sum<L>(ss);
        if (KIND != 3 || !is_v) {
          const float inv = rsqrtf(fmaf(ss, a.inv_d, a.eps));
#pragma unroll
          for (int e = 0; e < N; e++) {
            xa[e] *= inv * (KIND == 0 ? wqa[e] : KIND == 1 ? wka[e] : is_q ? wqa[e] : wka[e]);
            xb[e] *= inv * (KIND == 0 ? wqb[e] : KIND == 1 ? wkb[e] : is_q ? wqb[e] : wkb[e]);
          }
          if (!GEN || (!a.interleaved && rotates)) {
#pragma unroll
            for (int e = 0; e < N; e++) {
              const float na = xa[e], nb = xb[e];
              xa[e] = fmaf(na, cs[e].x, -nb * cs[e].y);
              xb[e] = fmaf(na, cs[e].y, nb * cs[e].x);
            }
          } else if (a.interleaved) {
#pragma unroll
            for (int h = 0; h < N / 2; h++) {
              if (va < a.rot_vec) {
                const float x0 = xa[2 * h], x1 = xa[2 * h + 1];
                xa[2 * h] = fmaf(x0, cs[h].x, -x1 * cs[h].y);
                xa[2 * h + 1] = fmaf(x0, cs[h].y, x1 * cs[h].x);
              }
              if (vb < a.rot_vec) {
                const float x0 = xb[2 * h], x1 = xb[2 * h + 1];
                xb[2 * h] = fmaf(x0, cs[N / 2 + h].x, -x1 * cs[N / 2 + h].y);
                xb[2 * h + 1] = fmaf(x0, cs[N / 2 + h].y, x1 * cs[N / 2 + h].x);
              }
            }
          }
        }
      }
      if (KIND == 0 || (KIND == 3 && is_q && valid)) {
        r[va] = Vec<T>::pack(xa);
        r[vb] = Vec<T>::pack(xb);
      }
      if (KIND == 0) return;
      const int head = row - a.hq - (is_v ? a.hk : 0);
      const CacheSide side = is_v ? a.side[1] : a.side[0];
      const bool write = kept && valid && !is_q;
      if constexpr (!FP4) {
        const float top = clamp_scale(group_max<L>(fmaxf(max_abs(xa), max_abs(xb))));
        if (!write) return;
        const float inv = fp8_inverse(top);
        unsigned char* o = side.codes + code_off + static_cast<int64_t>(head) * D;
        uint32_t ca[N / 4], cb[N / 4];
        fp8_codes(xa, inv, ca);
        fp8_codes(xb, inv, cb);
        if constexpr (N == 8) {
          st_stream8(o + va * N, make_uint2(ca[0], ca[N / 4 - 1]));
          st_stream8(o + vb * N, make_uint2(cb[0], cb[N / 4 - 1]));
        } else {
          st_stream4(o + va * N, ca[0]);
          st_stream4(o + vb * N, cb[0]);
        }
        if (l == 0) reinterpret_cast<float*>(side.scales + scale_off)[head] = fp8_scale(top);
      } else {
        const uint32_t ba = mx_scale_byte(clamp_scale(group_max<W>(max_abs(xa))));
        const uint32_t bb = mx_scale_byte(clamp_scale(group_max<W>(max_abs(xb))));
        if (!write) return;
        unsigned char* o = side.codes + code_off + static_cast<int64_t>(head) * (D / 2);
        unsigned char* s = side.scales + scale_off + static_cast<int64_t>(head) * (D / 32);
        const uint32_t ca = fp4_codes(xa, mx_inverse(ba)), cb = fp4_codes(xb, mx_inverse(bb));
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
    for (int first = r0 + warp * GW; first < r1; first += kFusedWarps * GW) {  // warp-uniform
      const int last = first + GW;
      if (last <= r1 && last <= a.hq)
        pass(std::integral_constant<int, 0>(), first);
      else if (last <= r1 && first >= a.hq && last <= a.hq + a.hk)
        pass(std::integral_constant<int, 1>(), first);
      else if (last <= r1 && first >= a.hq + a.hk)
        pass(std::integral_constant<int, 2>(), first);
      else
        pass(std::integral_constant<int, 3>(), first);
    }
    // the next item's angles, into the other table
    const Item done = cur;
    cur = nxt;
    next(nxt);
    slot = slot_next;
    if (cur.tok < a.tokens) {
      float2* t = table + ((j + 1) & 1) * HALF;
      if (tid < pairs) angle(t, tid, pos_next);
      for (int i = tid + kFusedThreads; i < pairs; i += kFusedThreads) angle(t, i, position(cur, i));
      if (nxt.tok < a.tokens && tid < pairs) pos_next = position(nxt, tid);
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (*abort_flag) break;
    if (tid == 0) {
      if (r0 < a.hq)
        bulk_store_hint(static_cast<T*>(a.q_out) + done.tok * a.q_stride +
                            static_cast<int64_t>(r0) * D,
                        smem_addr(st), static_cast<unsigned>((min(r1, a.hq) - r0) * D * sizeof(T)),
                        policy);
      bulk_commit();  // possibly empty: one group per item
      if (ahead.tok < a.tokens) {
        bulk_wait_read<1>();  // the stage of item j - 1 has been read out
        issue();
      }
    }
  }
  if (tid == 0) {
    bulk_wait<0>();  // every store has landed before the block's shared memory is released
    // After an abandoned wait (at item j), let the loads still in flight
    // finish (bounded); after a normal finish there are none (j == issued).
    for (int64_t m = j; m < issued; m++)
      if (!mbar_wait_bounded(smem_addr(bars + m % kStages),
                             static_cast<unsigned>((m / kStages) & 1), kFusedWaitLimit))
        break;
  }
}

// Resident blocks over the current device for this kernel with `smem` bytes;
// the last answer of each device is kept (a racing thread at worst asks again).
template <typename Kernel>
cudaError_t fused_resident(Kernel kernel, size_t smem, std::atomic<uint64_t>* cache,
                           int64_t* blocks) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  const uint64_t had = cache[device].load(std::memory_order_relaxed);
  if (had >> 32 == smem) {
    *blocks = static_cast<int64_t>(had & 0xFFFFFFFFu);
    return cudaSuccess;
  }
  int sms = 0, per_sm = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024);
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kFusedThreads, smem);
  if (e != cudaSuccess) return e;
  *blocks = static_cast<int64_t>(sms) * (per_sm > 0 ? per_sm : 1);
  cache[device].store(static_cast<uint64_t>(smem) << 32 | static_cast<uint64_t>(*blocks),
                      std::memory_order_relaxed);
  return cudaSuccess;
}

template <typename T, typename WT, int L, bool FP4, bool GEN>
cudaError_t fused_launch(FusedArgs& a, const RopeTurns& turns, cudaStream_t s) {
  constexpr int row_bytes = FusedSmem<T, L>::D * static_cast<int>(sizeof(T));
  const int rows = a.hq + 2 * a.hk;
  const int item_bytes = a.tokens * rows * row_bytes >= 152 * 4 * 2 * int64_t(kItemBytesMany)
                             ? kItemBytesMany
                             : kItemBytesFew;
  a.items = static_cast<int>((static_cast<int64_t>(rows) * row_bytes + item_bytes - 1) / item_bytes);
  a.chunk = (rows + a.items - 1) / a.items;
  // whole passes of the four warps, where that does not outgrow the stage
  constexpr int pass_rows = kFusedWarps * (kWarp / L);
  const int even = (a.chunk + pass_rows - 1) / pass_rows * pass_rows;
  if (a.items > 1 && even * row_bytes <= item_bytes) a.chunk = even;
  a.items = (rows + a.chunk - 1) / a.chunk;
  a.stage_bytes = (static_cast<unsigned>(a.chunk * row_bytes) + 127u) & ~127u;
  const size_t smem = FusedSmem<T, L>::bytes(a.stage_bytes);
  auto kernel = qk_cache_kernel<T, WT, L, FP4, GEN>;
  static std::atomic<uint64_t> cache[64];
  int64_t resident = 0;
  const cudaError_t e = fused_resident(kernel, smem, cache, &resident);
  if (e != cudaSuccess) return e;
  const int64_t total = a.tokens * a.items;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(total < resident ? total : resident)),
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
  cudaError_t e = status_word(&a.status);
  if (e != cudaSuccess) return e;
  const int lanes = static_cast<int>(c.head_dim / (2 * n));
  if (is_bf16)
    return w_is_bf16 ? fused_w<__nv_bfloat16, __nv_bfloat16>(a, c.fp4, lanes, turns, stream)
                     : fused_w<__nv_bfloat16, float>(a, c.fp4, lanes, turns, stream);
  return w_is_bf16 ? fused_w<float, __nv_bfloat16>(a, c.fp4, lanes, turns, stream)
                   : fused_w<float, float>(a, c.fp4, lanes, turns, stream);
}

}  // namespace nr
