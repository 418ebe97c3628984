// Quantised paged K/V cache for sm_103a: writing new tokens, and reading
// sequences back.
//
// Write: a group of L lanes owns one (token, head) row, each lane units of
// eight values, so the row's (FP8) or the 32-element group's (MXFP4) largest
// magnitude is a butterfly over lanes.  Each input byte is read once and each
// code written once; HBM (large calls) or latency (decode) bounds it: [16381,
// 8, 128] bf16 to FP8 in 16.2 us (0.92 of the measured copy rate), 32 tokens in
// 1.6 us.
//
// Read: a block first resolves the slots of a few output rows (a binary search
// for the sequence, a page-table lookup) into shared memory, then streams
// their codes, sixteen a thread, and writes widened rows: [100003, 8, 128] FP8
// to bf16 in 93.1 us (0.98 of the measured copy rate).
#include "quant.cuh"

namespace nr {
namespace {

constexpr int kCacheThreads = 128;
constexpr int kUnit = 8;  // values a lane handles at a time

struct WriteArgs {
  const void* src[2];   // k, v
  int64_t stride[2];    // elements between tokens
  CacheSide side[2];
  CacheGeom geo;
  const int64_t* slots;
  FastDiv heads;
  uint32_t rows;  // tokens * heads
  int units;      // head_dim / 8
};

// Raw words of a unit (8 values), the largest magnitude among them, and the
// values themselves.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  template <bool WIDE>
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = ld_stream(p);
  }
  // Of the packed pairs, sign bits cleared: two values an instruction.
  __device__ __forceinline__ float top() const {
    const uint32_t m = max2(max2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                            max2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    return fmaxf(bf16_lo(m), bf16_hi(m));
  }
  __device__ __forceinline__ void get(float (&f)[kUnit]) const {
    Vec<__nv_bfloat16>::unpack(v, f);
  }
  // The larger of each pair of halves; a NaN counts as nothing.
  __device__ __forceinline__ static uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};
template <>
struct Raw<float> {
  uint4 v, w;
  __device__ __forceinline__ void zero() { v = w = make_uint4(0u, 0u, 0u, 0u); }
  template <bool WIDE>
  __device__ __forceinline__ void load(const float* p) {
    if (WIDE) {
      ld_stream32(p, v, w);
    } else {
      v = ld_stream(p);
      w = ld_stream(p + 4);
    }
  }
  __device__ __forceinline__ float top() const {
    float f[kUnit];
    get(f);
    return max_abs(f);
  }
  __device__ __forceinline__ void get(float (&f)[kUnit]) const {
    float a[4], b[4];
    Vec<float>::unpack(v, a);
    Vec<float>::unpack(w, b);
#pragma unroll
    for (int e = 0; e < 4; e++) f[e] = a[e], f[e + 4] = b[e];
  }
};

// L lanes a row, NV units a lane (head_dim <= 8 * L * NV); lane l has units l,
// l + L, ...  blockIdx.y: 0 K, 1 V.  Few lanes and several units a lane: what a
// row costs once (its slot, its scale's division, the butterfly) is shared by
// more values.  At [16381, 8, 128] bf16 -> fp8: 16 lanes with one unit 33 us.
// WIDE: f32 rows are 32-byte aligned, a unit is one access.
template <typename T, bool FP4, int L, int NV, bool WIDE>
__global__ void __launch_bounds__(kCacheThreads) kv_write_kernel(const WriteArgs a) {
  constexpr int GW = kWarp / L;
  const int warp = threadIdx.x / kWarp, lane32 = threadIdx.x % kWarp;
  const int l = lane32 % L;
  const uint32_t row =
      (blockIdx.x * (kCacheThreads / kWarp) + warp) * static_cast<uint32_t>(GW) + lane32 / L;
  const bool is_v = blockIdx.y != 0;
  const CacheSide side = is_v ? a.side[1] : a.side[0];
  const int dim = a.units * kUnit;

  // Every load before any use; a padded token's row is in bounds, and its
  // values go nowhere.
  Raw<T> x[NV];
  int64_t slot = -1;
  uint32_t head = 0;
#pragma unroll
  for (int j = 0; j < NV; j++) x[j].zero();
  const uint32_t tok = a.heads.quot(row < a.rows ? row : 0);
  pdl_enter();  // before any global read: the previous kernel may still run
  if (row < a.rows) {
    head = row - tok * a.heads.div;
    slot = a.slots[tok];
    const T* p = static_cast<const T*>(is_v ? a.src[1] : a.src[0]) +
                 tok * (is_v ? a.stride[1] : a.stride[0]) + head * dim;
#pragma unroll
    for (int j = 0; j < NV; j++)
      if (l + j * L < a.units) x[j].template load<WIDE>(p + (l + j * L) * kUnit);
  }
  float top[NV], row_top = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; j++) {
    top[j] = x[j].top();
    if (FP4)
      top[j] = group_max<4>(top[j]);  // units 4i .. 4i + 3: one 32-element group
    else
      row_top = fmaxf(row_top, top[j]);
  }
  if (!FP4) row_top = group_max<L>(row_top);
  // slots outside the cache (padding) are skipped
  if (slot < 0 || slot >= a.geo.slots) return;
  const int64_t block = a.geo.block_of(slot);
  const int64_t place = slot - block * a.geo.block_size;
  unsigned char* codes = side.codes + block * a.geo.code_block_stride + place * a.geo.code_row;
  unsigned char* scales = side.scales + block * a.geo.scale_block_stride + place * a.geo.scale_row;
  float f[kUnit];
  if (!FP4) {
    const float am = clamp_scale(row_top), inv = fp8_inverse(am);
    codes += head * dim;
#pragma unroll
    for (int j = 0; j < NV; j++)
      if (l + j * L < a.units) {
        uint32_t c[2];
        x[j].get(f);
        fp8_codes(f, inv, c);
        st_stream8(codes + (l + j * L) * kUnit, make_uint2(c[0], c[1]));
      }
    if (l == 0) reinterpret_cast<float*>(scales)[head] = fp8_scale(am);
  } else {
    codes += head * (dim / 2);
    scales += head * (dim / 32);
#pragma unroll
    for (int j = 0; j < NV; j++)
      if (l + j * L < a.units) {
        const int u = l + j * L;
        const uint32_t byte = mx_scale_byte(clamp_scale(top[j]));
        x[j].get(f);
        st_stream4(codes + u * (kUnit / 2), fp4_codes(f, mx_inverse(byte)));
        if (u % 4 == 0) scales[u / 4] = static_cast<unsigned char>(byte);
      }
  }
}

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

template <typename T, bool FP4, int L, int NV>
cudaError_t write_l(const WriteArgs& a, cudaStream_t s) {
  constexpr unsigned rows = kCacheThreads / L;
  const dim3 grid((a.rows + rows - 1) / rows, 2);
  if constexpr (sizeof(T) == 4) {
    if (aligned32(a.src[0]) && aligned32(a.src[1]) && a.stride[0] % 8 == 0 && a.stride[1] % 8 == 0)
      return launch_pdl(kv_write_kernel<T, FP4, L, NV, true>, grid, dim3(kCacheThreads), 0, s, a);
  }
  return launch_pdl(kv_write_kernel<T, FP4, L, NV, false>, grid, dim3(kCacheThreads), 0, s, a);
}

template <typename T, bool FP4>
cudaError_t write_t(const WriteArgs& a, cudaStream_t s) {
  if (a.units <= 4) return write_l<T, FP4, 4, 1>(a, s);
  if (a.units <= 8) return write_l<T, FP4, 4, 2>(a, s);
  if (a.units <= 12) return write_l<T, FP4, 4, 3>(a, s);
  if (a.units <= 16) return write_l<T, FP4, 4, 4>(a, s);
  if (a.units <= 24) return write_l<T, FP4, 8, 3>(a, s);
  if (a.units <= 32) return write_l<T, FP4, 8, 4>(a, s);
  return write_l<T, FP4, 16, 4>(a, s);
}

// ---------------------------------------------------------------------------
// Read
// ---------------------------------------------------------------------------
constexpr int kReadThreads = 256;
constexpr int kReadMaxRows = 64;   // output rows a block resolves
constexpr int kReadUnit = 16;      // codes a thread widens at a time
constexpr int kReadSeqs = 1024;    // cu_seqlens entries searched in shared memory

struct ReadArgs {
  void* out[2];
  CacheSide side[2];
  CacheGeom geo;
  const int32_t* table;  // [seqs, width]
  const int32_t* cu;     // [seqs + 1]
  int64_t width;
  int64_t blocks;
  int seqs;
  int64_t rows;        // rows of the outputs
  int block_rows;      // output rows of a thread block
  FastDiv row_units;   // heads * head_dim / 16
  FastDiv head_units;  // head_dim / 16
};

// The slot of output row r: -1 for a row of no sequence (left as it is), -2
// for one whose page is missing (read as zeros).
__device__ __forceinline__ int64_t slot_of(const ReadArgs& a, const int32_t* cu, int64_t r) {
  if (r >= a.rows || r < cu[0] || r >= cu[a.seqs]) return -1;
  int lo = 0, hi = a.seqs;  // cu[lo] <= r < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (cu[mid] <= r) lo = mid;
    else hi = mid;
  }
  const int64_t t = r - cu[lo];
  const int64_t page = a.geo.block_of(t);
  if (page >= a.width) return -2;
  const int64_t block = a.table[lo * a.width + page];
  if (block < 0 || block >= a.blocks) return -2;
  return block * a.geo.block_size + (t - page * a.geo.block_size);
}

// 16 values to an output row; WIDE: 32-byte aligned.
template <bool WIDE>
__device__ __forceinline__ void put16(__nv_bfloat16* p, const float (&f)[16]) {
  uint4 v[2];
#pragma unroll
  for (int h = 0; h < 2; h++) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; e++) x[e] = f[8 * h + e];
    v[h] = Vec<__nv_bfloat16>::pack(x);
  }
  if (WIDE) {
    st_stream32(p, v[0], v[1]);
  } else {
    st_stream(p, v[0]);
    st_stream(p + 8, v[1]);
  }
}
template <bool WIDE>
__device__ __forceinline__ void put16(float* p, const float (&f)[16]) {
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const float x[4] = {f[8 * h], f[8 * h + 1], f[8 * h + 2], f[8 * h + 3]};
    const float y[4] = {f[8 * h + 4], f[8 * h + 5], f[8 * h + 6], f[8 * h + 7]};
    if (WIDE) {
      st_stream32(p + 8 * h, Vec<float>::pack(x), Vec<float>::pack(y));
    } else {
      st_stream(p + 8 * h, Vec<float>::pack(x));
      st_stream(p + 8 * h + 4, Vec<float>::pack(y));
    }
  }
}

template <typename T, bool FP4, bool WIDE>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const ReadArgs a) {
  __shared__ int64_t code_at[kReadMaxRows];  // byte offsets, or -1 / -2
  __shared__ int64_t scale_at[kReadMaxRows];
  __shared__ int32_t cu_sm[kReadSeqs + 1];
  pdl_enter();
  // One load a thread instead of a chain of them in the search.
  const bool few = a.seqs <= kReadSeqs;
  if (few) {
    for (int i = threadIdx.x; i <= a.seqs; i += kReadThreads) cu_sm[i] = a.cu[i];
    __syncthreads();
  }
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.block_rows;
  if (threadIdx.x < a.block_rows) {
    const int64_t slot = slot_of(a, few ? cu_sm : a.cu, row0 + threadIdx.x);
    int64_t c = slot, s = slot;
    if (slot >= 0) {
      const int64_t block = a.geo.block_of(slot);
      const int64_t place = slot - block * a.geo.block_size;
      c = block * a.geo.code_block_stride + place * a.geo.code_row;
      s = block * a.geo.scale_block_stride + place * a.geo.scale_row;
    }
    code_at[threadIdx.x] = c;
    scale_at[threadIdx.x] = s;
  }
  __syncthreads();
  const bool is_v = blockIdx.y != 0;
  T* out = static_cast<T*>(is_v ? a.out[1] : a.out[0]) +
           row0 * static_cast<int64_t>(a.row_units.div) * kReadUnit;
  const CacheSide side = is_v ? a.side[1] : a.side[0];
  const uint32_t n = static_cast<uint32_t>(a.block_rows) * a.row_units.div;
  constexpr int U = 4;
  for (uint32_t base = threadIdx.x; base < n; base += U * kReadThreads) {
    uint4 codes[U];
    float scale[U];
    int64_t where[U];
#pragma unroll
    for (int j = 0; j < U; j++) {
      const uint32_t i = base + j * kReadThreads;
      where[j] = -1;
      codes[j] = make_uint4(0u, 0u, 0u, 0u);
      scale[j] = 0.0f;
      if (i >= n) continue;
      const uint32_t r = a.row_units.quot(i), u = i - r * a.row_units.div;
      where[j] = code_at[r];
      if (where[j] < 0) continue;
      if (FP4) {
        const uint2 c = reinterpret_cast<const uint2*>(side.codes + where[j])[u];
        codes[j].x = c.x;
        codes[j].y = c.y;
        const uint32_t byte = side.scales[scale_at[r] + u / 2];
        // 2^(byte - 127); bytes 0 and 255 (2^-127, NaN) as the format has them
        scale[j] = byte == 0 ? 0x1p-127f : __uint_as_float(byte == 255 ? 0x7FC00000u : byte << 23);
      } else {
        codes[j] = ld_stream(reinterpret_cast<const uint4*>(side.codes + where[j]) + u);
        scale[j] =
            reinterpret_cast<const float*>(side.scales + scale_at[r])[a.head_units.quot(u)];
      }
    }
#pragma unroll
    for (int j = 0; j < U; j++) {
      if (where[j] == -1) continue;
      float f[kReadUnit];
      const uint32_t w[4] = {codes[j].x, codes[j].y, codes[j].z, codes[j].w};
#pragma unroll
      for (int h = 0; h < kReadUnit / 2; h++) {
        __half2_raw p;
        if (FP4)
          p = __nv_cvt_fp4x2_to_halfraw2(
              static_cast<__nv_fp4x2_storage_t>(w[h / 4] >> (8 * (h % 4))), __NV_E2M1);
        else
          p = __nv_cvt_fp8x2_to_halfraw2(
              static_cast<__nv_fp8x2_storage_t>(w[h / 2] >> (16 * (h % 2))), __NV_E4M3);
        const float2 v = __half22float2(__half2(p));
        f[2 * h] = v.x * scale[j];
        f[2 * h + 1] = v.y * scale[j];
      }
      put16<WIDE>(out + static_cast<int64_t>(base + j * kReadThreads) * kReadUnit, f);
    }
  }
}

template <typename T, bool FP4>
cudaError_t read_t(ReadArgs& a, cudaStream_t s) {
  // About four units a thread, so that resolving a slot is shared by many.
  int64_t rows = 4 * kReadThreads / static_cast<int64_t>(a.row_units.div);
  rows = rows < 1 ? 1 : rows > kReadMaxRows ? kReadMaxRows : rows;
  a.block_rows = static_cast<int>(rows);
  const dim3 grid(static_cast<unsigned>((a.rows + rows - 1) / rows), 2);
  // rows are multiples of 32 bytes, so the bases decide
  auto kernel = aligned32(a.out[0]) && aligned32(a.out[1]) ? kv_read_kernel<T, FP4, true>
                                                           : kv_read_kernel<T, FP4, false>;
  return launch_pdl(kernel, grid, dim3(kReadThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_kv_write(const KvCacheArgs& c, const void* k, const void* v,
                            const int64_t* slots, int64_t tokens, int64_t k_stride,
                            int64_t v_stride, int is_bf16, cudaStream_t stream) {
  WriteArgs a{{k, v},
              {k_stride, v_stride},
              {{c.k_codes, c.k_scales}, {c.v_codes, c.v_scales}},
              cache_geometry(c),
              slots,
              FastDiv(static_cast<uint32_t>(c.heads)),
              static_cast<uint32_t>(tokens * c.heads),
              static_cast<int>(c.head_dim / kUnit)};
  if (is_bf16)
    return c.fp4 ? write_t<__nv_bfloat16, true>(a, stream)
                 : write_t<__nv_bfloat16, false>(a, stream);
  return c.fp4 ? write_t<float, true>(a, stream) : write_t<float, false>(a, stream);
}

cudaError_t launch_kv_read(const KvCacheArgs& c, void* k_out, void* v_out, const int32_t* table,
                           int64_t width, const int32_t* cu, int64_t seqs, int64_t rows,
                           int is_bf16, cudaStream_t stream) {
  ReadArgs a{{k_out, v_out},
             {{c.k_codes, c.k_scales}, {c.v_codes, c.v_scales}},
             cache_geometry(c),
             table,
             cu,
             width,
             c.blocks,
             static_cast<int>(seqs),
             rows,
             0,
             FastDiv(static_cast<uint32_t>(c.heads * c.head_dim / kReadUnit)),
             FastDiv(static_cast<uint32_t>(c.head_dim / kReadUnit))};
  if (is_bf16)
    return c.fp4 ? read_t<__nv_bfloat16, true>(a, stream) : read_t<__nv_bfloat16, false>(a, stream);
  return c.fp4 ? read_t<float, true>(a, stream) : read_t<float, false>(a, stream);
}

}  // namespace nr
