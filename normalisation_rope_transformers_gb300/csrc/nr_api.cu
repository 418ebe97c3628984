// C ABI of the fused row-normalisation library: argument validation, the
// per-call rotary constants, and status reporting.  Every check runs on the
// host before any launch; a rejected call touches no device memory.
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <nvtx3/nvToolsExt.h>

#include "../../include/nr.h"
#include "nr_internal.h"

namespace {

// One NVTX range per entry-point call, named after the entry point, so that
// profilers (nsys, ncu --nvtx) can attribute kernels to the call that
// launched them.  Without a tool attached the push and pop cost a few
// nanoseconds.
struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
  CallRange(const CallRange&) = delete;
  CallRange& operator=(const CallRange&) = delete;
};

thread_local char g_message[512];

nr_status fail(nr_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_message, sizeof g_message, fmt, ap);
  va_end(ap);
  return s;
}

nr_status ok() {
  g_message[0] = '\0';
  return NR_OK;
}

nr_status from_cuda(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ok();
  return fail(NR_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int elem_size(nr_dtype d) { return d == NR_BF16 ? 2 : 4; }
int vec_elems(nr_dtype d) { return d == NR_BF16 ? 8 : 4; }
bool valid_dtype(int d) { return d == NR_F32 || d == NR_BF16; }

// `count` rows of `span` bytes, `stride` bytes apart, starting at `base`.
struct Region {
  uintptr_t base;
  int64_t stride;
  int64_t span;
  int64_t count;
};

Region dense(const void* p, int64_t bytes) {
  return Region{reinterpret_cast<uintptr_t>(p), bytes, bytes, 1};
}

// Conservative overlap test: false only when the two regions are provably
// disjoint (disjoint address ranges, or equal strides with rows that interleave
// without touching -- e.g. Q and K heads inside one fused QKV row).
bool overlap(const Region& a, const Region& b) {
  if (a.count <= 0 || b.count <= 0 || a.span <= 0 || b.span <= 0) return false;
  const uintptr_t a_end = a.base + static_cast<uintptr_t>((a.count - 1) * a.stride + a.span);
  const uintptr_t b_end = b.base + static_cast<uintptr_t>((b.count - 1) * b.stride + b.span);
  if (a_end <= b.base || b_end <= a.base) return false;
  if (a.stride == b.stride && a.stride >= a.span && a.stride >= b.span) {
    const int64_t s = a.stride;
    const int64_t diff = static_cast<int64_t>(b.base - a.base);  // two's complement
    const int64_t delta = ((diff % s) + s) % s;                   // b's row start inside a's period
    if (a.span <= delta && delta + b.span <= s) return false;
  }
  return true;
}

bool eps_ok(float eps) { return isfinite(eps) && eps >= 0.0f; }

}  // namespace

extern "C" {

int nr_version(void) { return 200; }

const char* nr_last_error_message(void) { return g_message; }

const char* nr_status_string(nr_status s) {
  switch (s) {
    case NR_OK: return "NR_OK";
    case NR_ERR_NULL: return "NR_ERR_NULL";
    case NR_ERR_SHAPE: return "NR_ERR_SHAPE";
    case NR_ERR_DTYPE: return "NR_ERR_DTYPE";
    case NR_ERR_ALIGN: return "NR_ERR_ALIGN";
    case NR_ERR_ALIAS: return "NR_ERR_ALIAS";
    case NR_ERR_UNSUPPORTED: return "NR_ERR_UNSUPPORTED";
    case NR_ERR_CUDA: return "NR_ERR_CUDA";
    case NR_ERR_VALUE: return "NR_ERR_VALUE";
    case NR_ERR_TIMEOUT: return "NR_ERR_TIMEOUT";
  }
  return "NR_ERR_UNKNOWN";
}

nr_status nr_rmsnorm(void* out, const void* x, const void* w, void* residual, int64_t rows,
                     int64_t hidden, nr_dtype dtype, float eps, int gemma, cudaStream_t stream) {
  CallRange range("nr_rmsnorm");
  if (!valid_dtype(dtype)) return fail(NR_ERR_DTYPE, "nr_rmsnorm: unknown dtype %d", (int)dtype);
  if (rows < 0) return fail(NR_ERR_SHAPE, "nr_rmsnorm: rows = %lld < 0", (long long)rows);
  if (hidden <= 0) return fail(NR_ERR_SHAPE, "nr_rmsnorm: hidden = %lld <= 0", (long long)hidden);
  if (!eps_ok(eps)) return fail(NR_ERR_VALUE, "nr_rmsnorm: eps must be finite and >= 0");
  if (gemma != 0 && gemma != 1) return fail(NR_ERR_VALUE, "nr_rmsnorm: gemma must be 0 or 1");
  if (rows == 0) return ok();
  if (!out || !x || !w) return fail(NR_ERR_NULL, "nr_rmsnorm: out, x and w must be non-NULL");
  const int vec = vec_elems(dtype);
  if (hidden % vec != 0)
    return fail(NR_ERR_UNSUPPORTED, "nr_rmsnorm: hidden = %lld is not a multiple of %d",
                (long long)hidden, vec);
  if (rows > INT32_MAX || hidden / vec > INT32_MAX)
    return fail(NR_ERR_SHAPE, "nr_rmsnorm: rows or hidden too large");
  if (!aligned16(out) || !aligned16(x) || !aligned16(w) || (residual && !aligned16(residual)))
    return fail(NR_ERR_ALIGN, "nr_rmsnorm: pointers must be 16-byte aligned");
  const int64_t row_bytes = hidden * elem_size(dtype);
  const Region ro = dense(out, rows * row_bytes), rx = dense(x, rows * row_bytes);
  const Region rw = dense(w, row_bytes);
  if (out != x && overlap(ro, rx))
    return fail(NR_ERR_ALIAS, "nr_rmsnorm: out partially overlaps x (only out == x is allowed)");
  if (overlap(ro, rw)) return fail(NR_ERR_ALIAS, "nr_rmsnorm: out overlaps w");
  if (residual) {
    const Region rr = dense(residual, rows * row_bytes);
    if (overlap(rr, rx) || overlap(rr, ro) || overlap(rr, rw))
      return fail(NR_ERR_ALIAS, "nr_rmsnorm: residual overlaps x, out or w");
  }
  return from_cuda(nr::launch_rmsnorm(out, x, w, residual, rows, hidden, dtype == NR_BF16, eps,
                                      gemma, stream),
                   "nr_rmsnorm launch");
}

nr_status nr_rmsnorm_quant_fp8(void* codes, void* out_bf16, const void* x, const void* w,
                               void* residual, int64_t rows, int64_t hidden, nr_dtype dtype,
                               float eps, int gemma, float scale, cudaStream_t stream) {
  CallRange range("nr_rmsnorm_quant_fp8");
  const char* fn = "nr_rmsnorm_quant_fp8";
  if (!valid_dtype(dtype)) return fail(NR_ERR_DTYPE, "%s: unknown dtype %d", fn, (int)dtype);
  if (rows < 0 || hidden <= 0)
    return fail(NR_ERR_SHAPE, "%s: need rows >= 0 and hidden > 0", fn);
  if (!eps_ok(eps)) return fail(NR_ERR_VALUE, "%s: eps must be finite and >= 0", fn);
  if (gemma != 0 && gemma != 1) return fail(NR_ERR_VALUE, "%s: gemma must be 0 or 1", fn);
  const float inv_scale = 1.0f / scale;
  if (!(isfinite(scale) && scale > 0.0f && isfinite(inv_scale)))
    return fail(NR_ERR_VALUE, "%s: scale must be finite and > 0 with a finite reciprocal", fn);
  if (rows == 0) return ok();
  if (!codes || !x || !w) return fail(NR_ERR_NULL, "%s: codes, x and w must be non-NULL", fn);
  const int vec = vec_elems(dtype);
  if (hidden % vec != 0)
    return fail(NR_ERR_UNSUPPORTED, "%s: hidden = %lld is not a multiple of %d", fn,
                (long long)hidden, vec);
  if (hidden / vec > nr::kQuantMaxVectors)
    return fail(NR_ERR_UNSUPPORTED, "%s: hidden = %lld is above %lld for this dtype", fn,
                (long long)hidden, (long long)(nr::kQuantMaxVectors * vec));
  if (rows > INT32_MAX) return fail(NR_ERR_SHAPE, "%s: rows too large", fn);
  if (!aligned16(codes) || !aligned16(x) || !aligned16(w) || (residual && !aligned16(residual)) ||
      (out_bf16 && !aligned16(out_bf16)))
    return fail(NR_ERR_ALIGN, "%s: pointers must be 16-byte aligned", fn);
  const int64_t row_bytes = hidden * elem_size(dtype);
  const Region rc = dense(codes, rows * hidden), rb = dense(out_bf16, out_bf16 ? rows * hidden * 2 : 0);
  const Region rx = dense(x, rows * row_bytes), rw = dense(w, row_bytes);
  const Region rr = dense(residual, residual ? rows * row_bytes : 0);
  if (overlap(rc, rx) || overlap(rc, rw) || overlap(rc, rr) || overlap(rc, rb) || overlap(rb, rx) ||
      overlap(rb, rw) || overlap(rb, rr))
    return fail(NR_ERR_ALIAS, "%s: an output overlaps an input or the other output", fn);
  if (overlap(rr, rx) || overlap(rr, rw))
    return fail(NR_ERR_ALIAS, "%s: residual overlaps x or w", fn);
  return from_cuda(nr::launch_rmsnorm_quant_fp8(codes, out_bf16, x, w, residual, rows, hidden,
                                                dtype == NR_BF16, eps, gemma, inv_scale, stream),
                   "nr_rmsnorm_quant_fp8 launch");
}

}  // extern "C"

namespace {

// Llama-3 rescale of one rotary frequency: keep short wavelengths, divide long
// ones by `factor`, and blend linearly (in 1/wavelength) between the two bands.
double llama3_rescale(double freq, const nr_rope_config& c) {
  if (!(c.llama3_factor > 0.0)) return freq;
  const double wavelength = 2.0 * M_PI / freq;
  const double short_band = c.llama3_original_max_position / c.llama3_high_freq_factor;
  const double long_band = c.llama3_original_max_position / c.llama3_low_freq_factor;
  if (wavelength < short_band) return freq;
  if (wavelength > long_band) return freq / c.llama3_factor;
  const double blend =
      c.llama3_high_freq_factor == c.llama3_low_freq_factor
          ? 0.0
          : (c.llama3_original_max_position / wavelength - c.llama3_low_freq_factor) /
                (c.llama3_high_freq_factor - c.llama3_low_freq_factor);
  return blend * freq + (1.0 - blend) * freq / c.llama3_factor;
}

// M-RoPE position row (0 = t, 1 = h, 2 = w) of rotary pair i.
unsigned char mrope_row(int64_t i, const nr_rope_config& c) {
  const int32_t* sec = c.mrope_section;
  if (c.mrope_interleaved) {
    const int64_t cycle = i / 3;
    if (i % 3 == 1 && cycle < sec[1]) return 1;
    if (i % 3 == 2 && cycle < sec[2]) return 2;
    return 0;
  }
  if (i < sec[0]) return 0;
  return i < sec[0] + sec[1] ? 1 : 2;
}

// The rotary configuration and eps for a head of head_dim elements in vectors
// of `vec`; the rotary dimension and whether M-RoPE is on.
nr_status check_rope(const char* fn, const nr_rope_config& rope, int64_t head_dim, int vec,
                     float eps, int64_t* rot_out, bool* mrope_out) {
  const int64_t rot = *rot_out = rope.rotary_dim == 0 ? head_dim : rope.rotary_dim;
  if (rot <= 0 || rot > head_dim || rot % 2 != 0)
    return fail(NR_ERR_SHAPE, "%s: rotary_dim %lld must be even and in (0, head_dim]", fn,
                (long long)rot);
  if ((rope.interleaved != 0 && rope.interleaved != 1) ||
      (rope.mrope_interleaved != 0 && rope.mrope_interleaved != 1))
    return fail(NR_ERR_VALUE, "%s: interleaved flags must be 0 or 1", fn);
  if (rot % (rope.interleaved ? vec : 2 * vec) != 0)
    return fail(NR_ERR_UNSUPPORTED, "%s: rotary_dim %lld must be a multiple of %d", fn,
                (long long)rot, rope.interleaved ? vec : 2 * vec);
  if (!eps_ok(eps)) return fail(NR_ERR_VALUE, "%s: eps must be finite and >= 0", fn);
  if (!(isfinite(rope.theta) && rope.theta > 0.0))
    return fail(NR_ERR_VALUE, "%s: theta must be finite and > 0", fn);
  if (!isfinite(rope.llama3_factor) ||
      (rope.llama3_factor > 0.0 &&
       !(rope.llama3_low_freq_factor > 0.0 &&
         rope.llama3_high_freq_factor >= rope.llama3_low_freq_factor &&
         rope.llama3_original_max_position > 0.0 && isfinite(rope.llama3_high_freq_factor) &&
         isfinite(rope.llama3_original_max_position))))
    return fail(NR_ERR_VALUE, "%s: Llama-3 factors must be positive and finite, high >= low", fn);
  const int32_t* sec = rope.mrope_section;
  const bool mrope = *mrope_out = sec[0] != 0 || sec[1] != 0 || sec[2] != 0;
  if (sec[0] < 0 || sec[1] < 0 || sec[2] < 0 ||
      (mrope && static_cast<int64_t>(sec[0]) + sec[1] + sec[2] != rot / 2))
    return fail(NR_ERR_SHAPE, "%s: M-RoPE sections must be >= 0 and sum to rotary_dim / 2", fn);
  return NR_OK;
}

// The rotary constants of a configuration.  They depend on it alone, and a
// program's calls mostly share one, so the last one's stay at hand (per thread):
// 64 powers cost about 2 us of a decode call's host time.
const nr::RopeTurns& rope_turns(const nr_rope_config& rope, int64_t rot, bool mrope) {
  thread_local nr_rope_config had;
  thread_local int64_t had_rot = 0;  // no rotary dimension is 0
  thread_local nr::RopeTurns turns;
  if (had_rot == rot && memcmp(&had, &rope, sizeof rope) == 0) return turns;
  had_rot = 0;
  // turn_i = frac(freq_i / 2pi) * 2^64, freq_i = theta^(-2i/rot) (Llama-3
  // rescaled when asked), in double.  Positions are integers, so
  // pos * freq_i mod 2pi = pos * (freq_i mod 2pi) mod 2pi.
  for (int64_t i = 0; i < nr::kMaxHalfDim; i++) {
    turns.turn[i] = 0;
    turns.axis[i] = 0;
  }
  for (int64_t i = 0; i < rot / 2; i++) {
    const double freq = llama3_rescale(
        pow(rope.theta, -2.0 * static_cast<double>(i) / static_cast<double>(rot)), rope);
    const double turns_per_step = freq / (2.0 * M_PI);
    const double frac = turns_per_step - floor(turns_per_step);
    const double scaled = ldexp(frac, 64);
    turns.turn[i] =
        scaled >= 18446744073709551616.0 ? 0ull : static_cast<unsigned long long>(scaled);
    turns.axis[i] = mrope ? mrope_row(i, rope) : 0;
  }
  memcpy(&had, &rope, sizeof rope);
  had_rot = rot;
  return turns;
}

nr_status qk_norm_rope_impl(const char* fn, void* q_out, void* k_out, const void* q, const void* k,
                            const void* wq, const void* wk, nr_dtype w_dtype,
                            const int32_t* positions, int64_t tokens, int64_t hq, int64_t hk,
                            int64_t head_dim, int64_t q_tok_stride, int64_t k_tok_stride,
                            float eps, int gemma, const nr_rope_config& rope, nr_dtype dtype,
                            cudaStream_t stream) {
  if (!valid_dtype(dtype) || !valid_dtype(w_dtype))
    return fail(NR_ERR_DTYPE, "%s: unknown dtype (%d, weights %d)", fn, (int)dtype, (int)w_dtype);
  if (tokens < 0 || hq < 1 || hk < 0 || head_dim <= 0)
    return fail(NR_ERR_SHAPE, "%s: need tokens >= 0, hq >= 1, hk >= 0, head_dim > 0", fn);
  if (head_dim % 2 != 0) return fail(NR_ERR_SHAPE, "%s: head_dim must be even", fn);
  const int vec = vec_elems(dtype);
  const int64_t lanes = head_dim / (2 * vec);
  if (head_dim % (2 * vec) != 0 || lanes > 32 || (lanes & (lanes - 1)) != 0)
    return fail(NR_ERR_UNSUPPORTED,
                "%s: head_dim %lld not supported for this dtype (bf16: 16..512, f32: 8..256, "
                "powers of two)",
                fn, (long long)head_dim);
  int64_t rot = 0;
  bool mrope = false;
  if (const nr_status s = check_rope(fn, rope, head_dim, vec, eps, &rot, &mrope)) return s;
  if (gemma != 0 && gemma != 1) return fail(NR_ERR_VALUE, "%s: gemma must be 0 or 1", fn);
  if (q_tok_stride < hq * head_dim || (hk > 0 && k_tok_stride < hk * head_dim))
    return fail(NR_ERR_SHAPE, "%s: token stride smaller than heads * head_dim", fn);
  if (tokens > INT32_MAX || hq + hk > 65536)
    return fail(NR_ERR_SHAPE, "%s: tokens or head count too large", fn);
  if (tokens == 0) return ok();
  if (!q_out || !q || !wq || !positions)
    return fail(NR_ERR_NULL, "%s: q_out, q, wq and positions must be non-NULL", fn);
  if (hk > 0 && (!k_out || !k || !wk))
    return fail(NR_ERR_NULL, "%s: k_out, k and wk must be non-NULL when hk > 0", fn);
  const int es = elem_size(dtype);
  if ((q_tok_stride * es) % 16 != 0 || (hk > 0 && (k_tok_stride * es) % 16 != 0))
    return fail(NR_ERR_ALIGN, "%s: token strides must be multiples of 16 bytes", fn);
  if (!aligned16(q_out) || !aligned16(q) || !aligned16(wq) ||
      (hk > 0 && (!aligned16(k_out) || !aligned16(k) || !aligned16(wk))) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u))
    return fail(NR_ERR_ALIGN,
                "%s: q/k/weights must be 16-byte aligned, positions 4-byte aligned", fn);

  const Region rq{reinterpret_cast<uintptr_t>(q), q_tok_stride * es, hq * head_dim * es, tokens};
  const Region rqo{reinterpret_cast<uintptr_t>(q_out), q_tok_stride * es, hq * head_dim * es,
                   tokens};
  const Region rk{reinterpret_cast<uintptr_t>(k), k_tok_stride * es, hk * head_dim * es,
                  hk > 0 ? tokens : 0};
  const Region rko{reinterpret_cast<uintptr_t>(k_out), k_tok_stride * es, hk * head_dim * es,
                   hk > 0 ? tokens : 0};
  const int ws = elem_size(w_dtype);
  const Region rwq = dense(wq, head_dim * ws);
  const Region rwk = dense(wk, hk > 0 ? head_dim * ws : 0);
  const Region rpos = dense(positions, (mrope ? 3 : 1) * tokens * 4);
  if ((q_out != q && overlap(rqo, rq)) || overlap(rqo, rk) || overlap(rqo, rwq) ||
      overlap(rqo, rwk) || overlap(rqo, rpos) || overlap(rqo, rko))
    return fail(NR_ERR_ALIAS, "%s: q_out overlaps an input or k_out", fn);
  if ((k_out != k && overlap(rko, rk)) || overlap(rko, rq) || overlap(rko, rwq) ||
      overlap(rko, rwk) || overlap(rko, rpos))
    return fail(NR_ERR_ALIAS, "%s: k_out overlaps an input", fn);

  const nr::RopeTurns& turns = rope_turns(rope, rot, mrope);
  return from_cuda(nr::launch_qk_norm_rope(q_out, k_out, q, k, wq, wk, w_dtype == NR_BF16,
                                           positions, tokens, hq, hk, head_dim, q_tok_stride,
                                           k_tok_stride, eps, turns, gemma, rot, rope.interleaved,
                                           mrope ? 1 : 0, dtype == NR_BF16, stream),
                   fn);
}

}  // namespace

extern "C" {

nr_status nr_qk_norm_rope(void* q_out, void* k_out, const void* q, const void* k, const void* wq,
                          const void* wk, nr_dtype w_dtype, const int32_t* positions,
                          int64_t tokens, int64_t hq, int64_t hk, int64_t head_dim,
                          int64_t q_tok_stride, int64_t k_tok_stride, float eps, double theta,
                          int gemma, nr_dtype dtype, cudaStream_t stream) {
  CallRange range("nr_qk_norm_rope");
  nr_rope_config rope = {};
  rope.theta = theta;
  return qk_norm_rope_impl("nr_qk_norm_rope", q_out, k_out, q, k, wq, wk, w_dtype, positions,
                           tokens, hq, hk, head_dim, q_tok_stride, k_tok_stride, eps, gemma, rope,
                           dtype, stream);
}

nr_status nr_qk_norm_rope_ex(void* q_out, void* k_out, const void* q, const void* k,
                             const void* wq, const void* wk, nr_dtype w_dtype,
                             const int32_t* positions, int64_t tokens, int64_t hq, int64_t hk,
                             int64_t head_dim, int64_t q_tok_stride, int64_t k_tok_stride,
                             float eps, int gemma, const nr_rope_config* rope, nr_dtype dtype,
                             cudaStream_t stream) {
  CallRange range("nr_qk_norm_rope_ex");
  if (rope == nullptr) return fail(NR_ERR_NULL, "nr_qk_norm_rope_ex: rope config is NULL");
  return qk_norm_rope_impl("nr_qk_norm_rope_ex", q_out, k_out, q, k, wq, wk, w_dtype, positions,
                           tokens, hq, hk, head_dim, q_tok_stride, k_tok_stride, eps, gemma, *rope,
                           dtype, stream);
}

nr_status nr_ln_modulate(void* out, const void* x, const void* shift, const void* scale,
                         int64_t rows, int64_t hidden, int64_t rows_per_sample, float eps,
                         nr_dtype dtype, cudaStream_t stream) {
  CallRange range("nr_ln_modulate");
  if (!valid_dtype(dtype)) return fail(NR_ERR_DTYPE, "nr_ln_modulate: unknown dtype %d", (int)dtype);
  if (rows < 0 || hidden <= 0 || rows_per_sample < 1)
    return fail(NR_ERR_SHAPE, "nr_ln_modulate: need rows >= 0, hidden > 0, rows_per_sample >= 1");
  if (!eps_ok(eps)) return fail(NR_ERR_VALUE, "nr_ln_modulate: eps must be finite and >= 0");
  if (rows == 0) return ok();
  if (!out || !x || !shift || !scale)
    return fail(NR_ERR_NULL, "nr_ln_modulate: out, x, shift and scale must be non-NULL");
  const int vec = vec_elems(dtype);
  if (hidden % vec != 0)
    return fail(NR_ERR_UNSUPPORTED, "nr_ln_modulate: hidden = %lld is not a multiple of %d",
                (long long)hidden, vec);
  if (rows > INT32_MAX || hidden / vec > INT32_MAX)
    return fail(NR_ERR_SHAPE, "nr_ln_modulate: rows or hidden too large");
  if (!aligned16(out) || !aligned16(x) || !aligned16(shift) || !aligned16(scale))
    return fail(NR_ERR_ALIGN, "nr_ln_modulate: pointers must be 16-byte aligned");
  const int64_t row_bytes = hidden * elem_size(dtype);
  const int64_t samples = (rows + rows_per_sample - 1) / rows_per_sample;
  const Region ro = dense(out, rows * row_bytes), rx = dense(x, rows * row_bytes);
  if (out != x && overlap(ro, rx))
    return fail(NR_ERR_ALIAS, "nr_ln_modulate: out partially overlaps x (only out == x is allowed)");
  if (overlap(ro, dense(shift, samples * row_bytes)) || overlap(ro, dense(scale, samples * row_bytes)))
    return fail(NR_ERR_ALIAS, "nr_ln_modulate: out overlaps shift or scale");
  return from_cuda(nr::launch_ln_modulate(out, x, shift, scale, rows, hidden, rows_per_sample,
                                          dtype == NR_BF16, eps, stream),
                   "nr_ln_modulate launch");
}

nr_status nr_gated_residual_ln_modulate(void* out, void* residual, const void* y,
                                        const void* gate, const void* shift, const void* scale,
                                        int64_t rows, int64_t hidden, int64_t rows_per_sample,
                                        float eps, nr_dtype dtype, cudaStream_t stream) {
  CallRange range("nr_gated_residual_ln_modulate");
  const char* fn = "nr_gated_residual_ln_modulate";
  if (!valid_dtype(dtype)) return fail(NR_ERR_DTYPE, "%s: unknown dtype %d", fn, (int)dtype);
  if (rows < 0 || hidden <= 0 || rows_per_sample < 1)
    return fail(NR_ERR_SHAPE, "%s: need rows >= 0, hidden > 0, rows_per_sample >= 1", fn);
  if (!eps_ok(eps)) return fail(NR_ERR_VALUE, "%s: eps must be finite and >= 0", fn);
  if (rows == 0) return ok();
  if (!out || !residual || !y || !gate || !shift || !scale)
    return fail(NR_ERR_NULL, "%s: every pointer must be non-NULL", fn);
  const int vec = vec_elems(dtype);
  if (hidden % vec != 0)
    return fail(NR_ERR_UNSUPPORTED, "%s: hidden = %lld is not a multiple of %d", fn,
                (long long)hidden, vec);
  if (hidden / vec > nr::kGatedMaxVectors)
    return fail(NR_ERR_UNSUPPORTED, "%s: hidden = %lld is above %lld for this dtype", fn,
                (long long)hidden, (long long)(nr::kGatedMaxVectors * vec));
  if (rows > INT32_MAX) return fail(NR_ERR_SHAPE, "%s: rows too large", fn);
  if (!aligned16(out) || !aligned16(residual) || !aligned16(y) || !aligned16(gate) ||
      !aligned16(shift) || !aligned16(scale))
    return fail(NR_ERR_ALIGN, "%s: pointers must be 16-byte aligned", fn);
  const int64_t row_bytes = hidden * elem_size(dtype);
  const int64_t samples = (rows + rows_per_sample - 1) / rows_per_sample;
  const Region ro = dense(out, rows * row_bytes), rr = dense(residual, rows * row_bytes);
  const Region ins[] = {dense(y, rows * row_bytes), dense(gate, samples * row_bytes),
                        dense(shift, samples * row_bytes), dense(scale, samples * row_bytes)};
  if (overlap(ro, rr)) return fail(NR_ERR_ALIAS, "%s: out overlaps residual", fn);
  for (const Region& in : ins)
    if (overlap(ro, in) || overlap(rr, in))
      return fail(NR_ERR_ALIAS, "%s: out or residual overlaps an input", fn);
  return from_cuda(nr::launch_gated_ln_modulate(out, residual, y, gate, shift, scale, rows, hidden,
                                                rows_per_sample, dtype == NR_BF16, eps, stream),
                   "nr_gated_residual_ln_modulate launch");
}

}  // extern "C"

namespace {

nr_status act_and_mul(const char* fn, int gelu, void* out, const void* x, int64_t rows,
                      int64_t inter, nr_dtype dtype, cudaStream_t stream) {
  if (!valid_dtype(dtype)) return fail(NR_ERR_DTYPE, "%s: unknown dtype %d", fn, (int)dtype);
  if (rows < 0 || inter <= 0) return fail(NR_ERR_SHAPE, "%s: need rows >= 0 and inter > 0", fn);
  if (rows == 0) return ok();
  if (!out || !x) return fail(NR_ERR_NULL, "%s: out and x must be non-NULL", fn);
  const int vec = vec_elems(dtype);
  if (inter % vec != 0)
    return fail(NR_ERR_UNSUPPORTED, "%s: inter = %lld is not a multiple of %d", fn,
                (long long)inter, vec);
  if (inter / vec > INT32_MAX / 2) return fail(NR_ERR_SHAPE, "%s: inter too large", fn);
  if (!aligned16(out) || !aligned16(x))
    return fail(NR_ERR_ALIGN, "%s: pointers must be 16-byte aligned", fn);
  const int64_t es = elem_size(dtype);
  if (overlap(dense(out, rows * inter * es), dense(x, rows * 2 * inter * es)))
    return fail(NR_ERR_ALIAS, "%s: out overlaps x", fn);
  const cudaError_t e = gelu ? nr::launch_gelu_and_mul(out, x, rows, inter, dtype == NR_BF16, stream)
                             : nr::launch_silu_and_mul(out, x, rows, inter, dtype == NR_BF16, stream);
  return from_cuda(e, fn);
}

}  // namespace

namespace {

// The cache's sizes, strides and pointers (`need_pointers` false: a call that
// touches nothing).  On success `args` is what the launchers take.
nr_status check_cache(const char* fn, const nr_kv_cache* c, bool need_pointers,
                      nr::KvCacheArgs* args) {
  if (c == nullptr) return fail(NR_ERR_NULL, "%s: the cache is NULL", fn);
  if (c->format != NR_CACHE_FP8 && c->format != NR_CACHE_MXFP4)
    return fail(NR_ERR_DTYPE, "%s: unknown cache format %d", fn, (int)c->format);
  const bool fp4 = c->format == NR_CACHE_MXFP4;
  if (c->blocks < 1 || c->block_size < 1 || c->heads < 1 || c->head_dim < 1)
    return fail(NR_ERR_SHAPE, "%s: blocks, block_size, heads and head_dim must be >= 1", fn);
  if (c->head_dim > 512 || c->head_dim % (fp4 ? 32 : 16) != 0)
    return fail(NR_ERR_UNSUPPORTED, "%s: head_dim %lld must be a multiple of %d, at most 512", fn,
                (long long)c->head_dim, fp4 ? 32 : 16);
  if (c->heads > (int64_t(1) << 24) / c->head_dim || c->blocks > INT32_MAX ||
      c->block_size > INT32_MAX)
    return fail(NR_ERR_SHAPE, "%s: heads, blocks or block_size too large", fn);
  const int64_t code_bytes = c->block_size * c->heads * (fp4 ? c->head_dim / 2 : c->head_dim);
  const int64_t scale_bytes = c->block_size * c->heads * (fp4 ? c->head_dim / 32 : 4);
  if (c->code_block_stride < code_bytes || c->scale_block_stride < scale_bytes)
    return fail(NR_ERR_SHAPE, "%s: a block stride is smaller than a block", fn);
  if (c->code_block_stride > INT64_MAX / 2 / c->blocks ||
      c->scale_block_stride > INT64_MAX / 2 / c->blocks)
    return fail(NR_ERR_SHAPE, "%s: a block stride is too large", fn);
  if (c->code_block_stride % 16 != 0 || (!fp4 && c->scale_block_stride % 4 != 0))
    return fail(NR_ERR_ALIGN, "%s: block strides must be multiples of 16 (codes) and 4 (f32 scales)",
                fn);
  if (need_pointers) {
    if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales)
      return fail(NR_ERR_NULL, "%s: the cache's pointers must be non-NULL", fn);
    if (!aligned16(c->k_codes) || !aligned16(c->v_codes) ||
        (!fp4 && ((reinterpret_cast<uintptr_t>(c->k_scales) |
                   reinterpret_cast<uintptr_t>(c->v_scales)) & 3u)))
      return fail(NR_ERR_ALIGN, "%s: codes must be 16-byte aligned, f32 scales 4-byte", fn);
  }
  *args = nr::KvCacheArgs{static_cast<unsigned char*>(c->k_codes),
                          static_cast<unsigned char*>(c->v_codes),
                          static_cast<unsigned char*>(c->k_scales),
                          static_cast<unsigned char*>(c->v_scales),
                          c->blocks,
                          c->block_size,
                          c->heads,
                          c->head_dim,
                          c->code_block_stride,
                          c->scale_block_stride,
                          fp4};
  return NR_OK;
}

// The cache's four parts: K codes, V codes, K scales, V scales.
struct CacheRegions {
  Region part[4];
  explicit CacheRegions(const nr_kv_cache& c) {
    const bool fp4 = c.format == NR_CACHE_MXFP4;
    const int64_t codes = c.block_size * c.heads * (fp4 ? c.head_dim / 2 : c.head_dim);
    const int64_t scales = c.block_size * c.heads * (fp4 ? c.head_dim / 32 : 4);
    auto region = [&](const void* p, int64_t stride, int64_t span) {
      return Region{reinterpret_cast<uintptr_t>(p), stride, span, c.blocks};
    };
    part[0] = region(c.k_codes, c.code_block_stride, codes);
    part[1] = region(c.v_codes, c.code_block_stride, codes);
    part[2] = region(c.k_scales, c.scale_block_stride, scales);
    part[3] = region(c.v_scales, c.scale_block_stride, scales);
  }
  bool overlaps(const Region& r) const {
    for (const Region& p : part)
      if (overlap(p, r)) return true;
    return false;
  }
  bool overlaps_itself() const {
    for (int i = 0; i < 4; i++)
      for (int j = 0; j < i; j++)
        if (overlap(part[i], part[j])) return true;
    return false;
  }
};

bool misaligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

}  // namespace

extern "C" {

nr_status nr_kv_cache_write(const nr_kv_cache* cache, const void* k, const void* v,
                            const int64_t* slots, int64_t tokens, int64_t k_tok_stride,
                            int64_t v_tok_stride, nr_dtype dtype, cudaStream_t stream) {
  CallRange range("nr_kv_cache_write");
  const char* fn = "nr_kv_cache_write";
  if (!valid_dtype(dtype)) return fail(NR_ERR_DTYPE, "%s: unknown dtype %d", fn, (int)dtype);
  if (tokens < 0) return fail(NR_ERR_SHAPE, "%s: tokens = %lld < 0", fn, (long long)tokens);
  nr::KvCacheArgs args;
  if (const nr_status s = check_cache(fn, cache, tokens > 0, &args)) return s;
  const int64_t row = cache->heads * cache->head_dim;
  if (k_tok_stride < row || v_tok_stride < row)
    return fail(NR_ERR_SHAPE, "%s: token stride smaller than heads * head_dim", fn);
  if (tokens > INT32_MAX / cache->heads)
    return fail(NR_ERR_SHAPE, "%s: tokens * heads too large", fn);
  if (tokens == 0) return ok();
  if (!k || !v || !slots) return fail(NR_ERR_NULL, "%s: k, v and slots must be non-NULL", fn);
  const int es = elem_size(dtype);
  if ((k_tok_stride * es) % 16 != 0 || (v_tok_stride * es) % 16 != 0)
    return fail(NR_ERR_ALIGN, "%s: token strides must be multiples of 16 bytes", fn);
  if (!aligned16(k) || !aligned16(v) || misaligned(slots, 8))
    return fail(NR_ERR_ALIGN, "%s: k and v must be 16-byte aligned, slots 8-byte", fn);
  const CacheRegions held(*cache);
  if (held.overlaps_itself())
    return fail(NR_ERR_ALIAS, "%s: parts of the cache overlap", fn);
  if (held.overlaps(Region{reinterpret_cast<uintptr_t>(k), k_tok_stride * es, row * es, tokens}) ||
      held.overlaps(Region{reinterpret_cast<uintptr_t>(v), v_tok_stride * es, row * es, tokens}) ||
      held.overlaps(dense(slots, tokens * 8)))
    return fail(NR_ERR_ALIAS, "%s: the cache overlaps an input", fn);
  return from_cuda(nr::launch_kv_write(args, k, v, slots, tokens, k_tok_stride, v_tok_stride,
                                       dtype == NR_BF16, stream),
                   "nr_kv_cache_write launch");
}

nr_status nr_qk_norm_rope_cache(const nr_kv_cache* cache, void* q_out, const void* q,
                                const void* k, const void* v, const void* wq, const void* wk,
                                nr_dtype w_dtype, const int32_t* positions, const int64_t* slots,
                                int64_t tokens, int64_t hq, int64_t q_tok_stride,
                                int64_t k_tok_stride, int64_t v_tok_stride, float eps, int gemma,
                                const nr_rope_config* rope, nr_dtype dtype, cudaStream_t stream) {
  CallRange range("nr_qk_norm_rope_cache");
  const char* fn = "nr_qk_norm_rope_cache";
  if (!valid_dtype(dtype) || !valid_dtype(w_dtype))
    return fail(NR_ERR_DTYPE, "%s: unknown dtype (%d, weights %d)", fn, (int)dtype, (int)w_dtype);
  if (rope == nullptr) return fail(NR_ERR_NULL, "%s: rope config is NULL", fn);
  if (tokens < 0 || hq < 1) return fail(NR_ERR_SHAPE, "%s: need tokens >= 0 and hq >= 1", fn);
  nr::KvCacheArgs args;
  if (const nr_status s = check_cache(fn, cache, tokens > 0, &args)) return s;
  const int vec = vec_elems(dtype);
  const int64_t dim = cache->head_dim, lanes = dim / (2 * vec);
  if (dim % (2 * vec) != 0 || lanes < 4 || lanes > 32 || (lanes & (lanes - 1)) != 0)
    return fail(NR_ERR_UNSUPPORTED,
                "%s: head_dim %lld not supported for this dtype (bf16: 64..512, f32: 32..256, "
                "powers of two)",
                fn, (long long)dim);
  int64_t rot = 0;
  bool mrope = false;
  if (const nr_status s = check_rope(fn, *rope, dim, vec, eps, &rot, &mrope)) return s;
  if (args.fp4 && (dim % 64 != 0 || (!rope->interleaved && rot % 64 != 0)))
    return fail(NR_ERR_UNSUPPORTED,
                "%s: MXFP4 needs head_dim %lld and (rotate-half) rotary_dim %lld in multiples of 64",
                fn, (long long)dim, (long long)rot);
  if (gemma != 0 && gemma != 1) return fail(NR_ERR_VALUE, "%s: gemma must be 0 or 1", fn);
  const int64_t hk = cache->heads;
  if (q_tok_stride < hq * dim || k_tok_stride < hk * dim || v_tok_stride < hk * dim)
    return fail(NR_ERR_SHAPE, "%s: token stride smaller than heads * head_dim", fn);
  if (tokens > INT32_MAX || hq + 2 * hk > 65536)
    return fail(NR_ERR_SHAPE, "%s: tokens or head count too large", fn);
  if (tokens == 0) return ok();
  if (!q_out || !q || !k || !v || !wq || !wk || !positions || !slots)
    return fail(NR_ERR_NULL, "%s: every pointer must be non-NULL", fn);
  const int es = elem_size(dtype);
  if ((q_tok_stride * es) % 16 != 0 || (k_tok_stride * es) % 16 != 0 ||
      (v_tok_stride * es) % 16 != 0)
    return fail(NR_ERR_ALIGN, "%s: token strides must be multiples of 16 bytes", fn);
  if (!aligned16(q_out) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(wq) ||
      !aligned16(wk) || misaligned(positions, 4) || misaligned(slots, 8))
    return fail(NR_ERR_ALIGN,
                "%s: q/k/v/weights must be 16-byte aligned, positions 4-byte, slots 8-byte", fn);
  const int ws = elem_size(w_dtype);
  const Region rqo{reinterpret_cast<uintptr_t>(q_out), q_tok_stride * es, hq * dim * es, tokens};
  const Region rq{reinterpret_cast<uintptr_t>(q), q_tok_stride * es, hq * dim * es, tokens};
  const Region ins[] = {
      Region{reinterpret_cast<uintptr_t>(k), k_tok_stride * es, hk * dim * es, tokens},
      Region{reinterpret_cast<uintptr_t>(v), v_tok_stride * es, hk * dim * es, tokens},
      dense(wq, dim * ws), dense(wk, dim * ws), dense(positions, (mrope ? 3 : 1) * tokens * 4),
      dense(slots, tokens * 8)};
  const CacheRegions held(*cache);
  if (held.overlaps_itself()) return fail(NR_ERR_ALIAS, "%s: parts of the cache overlap", fn);
  if ((q_out != q && overlap(rqo, rq)) || held.overlaps(rqo) || held.overlaps(rq))
    return fail(NR_ERR_ALIAS, "%s: q_out overlaps q or the cache", fn);
  for (const Region& in : ins)
    if (overlap(rqo, in) || held.overlaps(in))
      return fail(NR_ERR_ALIAS, "%s: q_out or the cache overlaps an input", fn);
  const nr::RopeTurns& turns = rope_turns(*rope, rot, mrope);
  return from_cuda(nr::launch_qk_norm_rope_cache(args, q_out, q, k, v, wq, wk, w_dtype == NR_BF16,
                                                 positions, slots, tokens, hq, q_tok_stride,
                                                 k_tok_stride, v_tok_stride, eps, turns, gemma,
                                                 rot, rope->interleaved, mrope ? 1 : 0,
                                                 dtype == NR_BF16, stream),
                   "nr_qk_norm_rope_cache launch");
}

nr_status nr_kv_cache_read(void* k_out, void* v_out, const nr_kv_cache* cache,
                           const int32_t* block_table, int64_t table_width,
                           const int32_t* cu_seqlens, int64_t seqs, int64_t rows, nr_dtype dtype,
                           cudaStream_t stream) {
  CallRange range("nr_kv_cache_read");
  const char* fn = "nr_kv_cache_read";
  if (!valid_dtype(dtype)) return fail(NR_ERR_DTYPE, "%s: unknown dtype %d", fn, (int)dtype);
  if (rows < 0 || seqs < 0 || table_width < 0)
    return fail(NR_ERR_SHAPE, "%s: need rows, seqs and table_width >= 0", fn);
  if (rows > INT32_MAX || seqs >= INT32_MAX || table_width > INT32_MAX)
    return fail(NR_ERR_SHAPE, "%s: rows, seqs or table_width too large", fn);
  const bool empty = rows == 0 || seqs == 0;
  nr::KvCacheArgs args;
  if (const nr_status s = check_cache(fn, cache, !empty, &args)) return s;
  if (empty) return ok();
  if (!k_out || !v_out || !cu_seqlens || (!block_table && table_width > 0))
    return fail(NR_ERR_NULL, "%s: k_out, v_out, block_table and cu_seqlens must be non-NULL", fn);
  if (!aligned16(k_out) || !aligned16(v_out) || misaligned(block_table, 4) ||
      misaligned(cu_seqlens, 4))
    return fail(NR_ERR_ALIGN, "%s: outputs must be 16-byte aligned, the tables 4-byte", fn);
  const int64_t bytes = rows * cache->heads * cache->head_dim * elem_size(dtype);
  const Region rk = dense(k_out, bytes), rv = dense(v_out, bytes);
  const Region table = dense(block_table, seqs * table_width * 4);
  const Region cu = dense(cu_seqlens, (seqs + 1) * 4);
  const CacheRegions held(*cache);
  if (overlap(rk, rv) || held.overlaps(rk) || held.overlaps(rv) || overlap(rk, table) ||
      overlap(rv, table) || overlap(rk, cu) || overlap(rv, cu))
    return fail(NR_ERR_ALIAS, "%s: an output overlaps the other, the cache or a table", fn);
  return from_cuda(nr::launch_kv_read(args, k_out, v_out, block_table, table_width, cu_seqlens,
                                      seqs, rows, dtype == NR_BF16, stream),
                   "nr_kv_cache_read launch");
}

}  // extern "C"

namespace {

// Sizes, and the workspace bytes that they need.
nr_status check_group_norm_sizes(const char* fn, int64_t samples, int64_t space, int64_t channels,
                                 int64_t groups, int backward, nr_dtype dtype, int64_t* need) {
  if (!valid_dtype(dtype)) return fail(NR_ERR_DTYPE, "%s: unknown dtype %d", fn, (int)dtype);
  if (samples < 0 || space < 0 || channels <= 0 || groups <= 0)
    return fail(NR_ERR_SHAPE, "%s: need samples, space >= 0 and channels, groups > 0", fn);
  if (channels % groups != 0)
    return fail(NR_ERR_SHAPE, "%s: %lld channels do not divide into %lld groups", fn,
                (long long)channels, (long long)groups);
  const int vec = vec_elems(dtype);
  if (channels % vec != 0)
    return fail(NR_ERR_UNSUPPORTED, "%s: channels = %lld is not a multiple of %d", fn,
                (long long)channels, vec);
  if (channels > 65536)
    return fail(NR_ERR_UNSUPPORTED, "%s: channels = %lld is above 65536", fn, (long long)channels);
  if (samples > INT32_MAX || space > INT64_MAX / 16 / channels ||
      (samples > 0 && space * channels > INT64_MAX / 16 / samples))
    return fail(NR_ERR_SHAPE, "%s: samples, space or channels too large", fn);
  *need = 0;
  if (samples > 0 && space > 0) {
    int64_t blocks = 0;
    *need = nr::group_norm_workspace(samples, space, channels, groups, backward,
                                     dtype == NR_BF16, &blocks);
    if (blocks > INT32_MAX)
      return fail(NR_ERR_SHAPE, "%s: too many samples for one launch", fn);
  }
  return NR_OK;
}

// What both directions share.
nr_status check_group_norm(const char* fn, const nr::GroupNormArgs& a, nr_dtype w_dtype,
                           nr_activation act, int64_t need, int64_t workspace_bytes) {
  if (!valid_dtype(w_dtype))
    return fail(NR_ERR_DTYPE, "%s: unknown weight dtype %d", fn, (int)w_dtype);
  if (act != NR_ACT_NONE && act != NR_ACT_SILU)
    return fail(NR_ERR_VALUE, "%s: unknown activation %d", fn, (int)act);
  if (a.samples == 0 || a.space == 0) return NR_OK;
  if (!a.out || !a.x || !a.mean || !a.rstd || (need > 0 && !a.workspace))
    return fail(NR_ERR_NULL, "%s: the tensors, mean, rstd and workspace must be non-NULL", fn);
  if ((a.w == nullptr) != (a.b == nullptr))
    return fail(NR_ERR_NULL, "%s: w and b are given together or not at all", fn);
  if (!aligned16(a.out) || !aligned16(a.x) || !aligned16(a.w) || !aligned16(a.b) ||
      !aligned16(a.workspace) || misaligned(a.mean, 4) || misaligned(a.rstd, 4))
    return fail(NR_ERR_ALIGN, "%s: pointers must be 16-byte aligned (mean and rstd 4-byte)", fn);
  if (workspace_bytes < need)
    return fail(NR_ERR_SHAPE, "%s: the workspace has %lld bytes, %lld are needed", fn,
                (long long)workspace_bytes, (long long)need);
  return NR_OK;
}

bool any_overlap(const Region* all, int n, const Region& one) {
  for (int i = 0; i < n; i++)
    if (overlap(all[i], one)) return true;
  return false;
}

}  // namespace

extern "C" {

nr_status nr_group_norm_workspace(int64_t samples, int64_t space, int64_t channels,
                                  int64_t groups, int backward, nr_dtype dtype, int64_t* bytes) {
  const char* fn = "nr_group_norm_workspace";
  if (backward != 0 && backward != 1)
    return fail(NR_ERR_VALUE, "%s: backward must be 0 or 1", fn);
  int64_t need = 0;
  if (const nr_status s =
          check_group_norm_sizes(fn, samples, space, channels, groups, backward, dtype, &need))
    return s;
  if (bytes == nullptr) return fail(NR_ERR_NULL, "%s: bytes must be non-NULL", fn);
  *bytes = need;
  return ok();
}

nr_status nr_group_norm(void* out, float* mean, float* rstd, const void* x, const void* w,
                        const void* b, nr_dtype w_dtype, int64_t samples, int64_t space,
                        int64_t channels, int64_t groups, float eps, nr_activation act,
                        nr_dtype dtype, void* workspace, int64_t workspace_bytes,
                        cudaStream_t stream) {
  CallRange range("nr_group_norm");
  const char* fn = "nr_group_norm";
  int64_t need = 0;
  if (const nr_status s =
          check_group_norm_sizes(fn, samples, space, channels, groups, 0, dtype, &need))
    return s;
  if (!eps_ok(eps)) return fail(NR_ERR_VALUE, "%s: eps must be finite and >= 0", fn);
  nr::GroupNormArgs a = {};
  a.out = out;
  a.mean = mean;
  a.rstd = rstd;
  a.x = x;
  a.w = w;
  a.b = b;
  a.w_is_bf16 = w_dtype == NR_BF16;
  a.samples = samples;
  a.space = space;
  a.channels = channels;
  a.groups = groups;
  a.eps = eps;
  a.silu = act == NR_ACT_SILU;
  a.workspace = workspace;
  if (const nr_status s = check_group_norm(fn, a, w_dtype, act, need, workspace_bytes)) return s;
  if (samples == 0 || space == 0) return ok();
  const int64_t bytes = samples * space * channels * elem_size(dtype);
  const int64_t wb = channels * elem_size(w_dtype), stats = samples * groups * 4;
  const Region ro = dense(out, bytes), rx = dense(x, bytes);
  const Region rm = dense(mean, stats), rr = dense(rstd, stats);
  const Region ws = dense(workspace, workspace ? workspace_bytes : 0);
  const Region ins[] = {rx, dense(w, w ? wb : 0), dense(b, b ? wb : 0)};
  if ((out != x && overlap(ro, rx)) || any_overlap(ins + 1, 2, ro) || any_overlap(ins, 3, rm) ||
      any_overlap(ins, 3, rr) || any_overlap(ins, 3, ws) || overlap(ro, rm) || overlap(ro, rr) ||
      overlap(ro, ws) || overlap(rm, rr) || overlap(rm, ws) || overlap(rr, ws))
    return fail(NR_ERR_ALIAS, "%s: an output or the workspace overlaps another tensor", fn);
  return from_cuda(nr::launch_group_norm(a, dtype == NR_BF16, stream), "nr_group_norm launch");
}

nr_status nr_group_norm_backward(void* dx, void* dw, void* db, const void* dy, const void* x,
                                 const float* mean, const float* rstd, const void* w,
                                 const void* b, nr_dtype w_dtype, int64_t samples, int64_t space,
                                 int64_t channels, int64_t groups, nr_activation act,
                                 nr_dtype dtype, void* workspace, int64_t workspace_bytes,
                                 cudaStream_t stream) {
  CallRange range("nr_group_norm_backward");
  const char* fn = "nr_group_norm_backward";
  int64_t need = 0;
  if (const nr_status s =
          check_group_norm_sizes(fn, samples, space, channels, groups, 1, dtype, &need))
    return s;
  nr::GroupNormArgs a = {};
  a.out = dx;
  a.dw = dw;
  a.db = db;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dy = dy;
  a.x = x;
  a.w = w;
  a.b = b;
  a.w_is_bf16 = w_dtype == NR_BF16;
  a.samples = samples;
  a.space = space;
  a.channels = channels;
  a.groups = groups;
  a.silu = act == NR_ACT_SILU;
  a.workspace = workspace;
  if (const nr_status s = check_group_norm(fn, a, w_dtype, act, need, workspace_bytes)) return s;
  if (samples == 0 || space == 0) return ok();
  if (!dy) return fail(NR_ERR_NULL, "%s: dy must be non-NULL", fn);
  if ((dw != nullptr) != (w != nullptr) || (db != nullptr) != (w != nullptr))
    return fail(NR_ERR_NULL, "%s: dw and db are given exactly when w and b are", fn);
  if (!aligned16(dy) || !aligned16(dw) || !aligned16(db))
    return fail(NR_ERR_ALIGN, "%s: pointers must be 16-byte aligned", fn);
  const int64_t bytes = samples * space * channels * elem_size(dtype);
  const int64_t wb = channels * elem_size(w_dtype), stats = samples * groups * 4;
  const Region ro = dense(dx, bytes), rw = dense(dw, dw ? wb : 0), rb = dense(db, db ? wb : 0);
  const Region ws = dense(workspace, workspace ? workspace_bytes : 0);
  const Region ins[] = {dense(dy, bytes),        dense(x, bytes),          dense(mean, stats),
                        dense(rstd, stats),      dense(w, w ? wb : 0),     dense(b, b ? wb : 0)};
  if ((dx != dy && overlap(ro, ins[0])) || (dx != x && overlap(ro, ins[1])) ||
      any_overlap(ins + 2, 4, ro) || any_overlap(ins, 6, rw) || any_overlap(ins, 6, rb) ||
      any_overlap(ins, 6, ws) || overlap(ro, rw) || overlap(ro, rb) || overlap(ro, ws) ||
      overlap(rw, rb) || overlap(rw, ws) || overlap(rb, ws))
    return fail(NR_ERR_ALIAS, "%s: an output or the workspace overlaps another tensor", fn);
  return from_cuda(nr::launch_group_norm_backward(a, dtype == NR_BF16, stream),
                   "nr_group_norm_backward launch");
}

}  // extern "C"

extern "C" {

nr_status nr_device_status(cudaStream_t stream) {
  CallRange range("nr_device_status");
  unsigned bits = 0;
  const cudaError_t e = nr::take_device_status(stream, &bits);
  if (e != cudaSuccess) return from_cuda(e, "nr_device_status");
  if (bits & nr::kStatusBitQkBulkWait)
    return fail(NR_ERR_TIMEOUT, "nr_device_status: a bounded wait for a bulk copy ran out in the "
                                "Q/K norm + RoPE kernel (status bits 0x%x)", bits);
  if (bits != 0)
    return fail(NR_ERR_TIMEOUT, "nr_device_status: the wait probe's wait ran out (status bits "
                                "0x%x)", bits);
  return ok();
}

nr_status nr_test_wait_probe(int64_t limit_cycles, cudaStream_t stream) {
  CallRange range("nr_test_wait_probe");
  if (limit_cycles < 1 || limit_cycles > (int64_t(1) << 32))
    return fail(NR_ERR_VALUE, "nr_test_wait_probe: limit_cycles must be in [1, 2^32]");
  return from_cuda(nr::launch_wait_probe(limit_cycles, stream), "nr_test_wait_probe");
}

nr_status nr_silu_and_mul(void* out, const void* x, int64_t rows, int64_t inter, nr_dtype dtype,
                          cudaStream_t stream) {
  CallRange range("nr_silu_and_mul");
  return act_and_mul("nr_silu_and_mul", 0, out, x, rows, inter, dtype, stream);
}

nr_status nr_gelu_and_mul(void* out, const void* x, int64_t rows, int64_t inter, nr_dtype dtype,
                          cudaStream_t stream) {
  CallRange range("nr_gelu_and_mul");
  return act_and_mul("nr_gelu_and_mul", 1, out, x, rows, inter, dtype, stream);
}

}  // extern "C"
