"""Fused row-normalisation kernels for GB300 (sm_103a): Python binding.

Thin ctypes binding over the C ABI in ``include/nr.h`` (``libnormrope.so``).
Each function marshals torch CUDA tensors into device pointers, sizes and the
current CUDA stream, calls the entry point of the same name, and raises on a
non-OK status.  Every step of the computation runs in the library's kernels;
there is no CPU or PyTorch fallback.  Importing fails loudly when the library
has not been built (``python normalisation_rope_transformers_gb300/build.py``
or ``__graft_entry__.build()``).

    rmsnorm(x, w, residual=None, eps=1e-6, gemma=False, out=None)
    rmsnorm_quant_fp8(x, w, scale, residual=None, eps=1e-6, gemma=False, out_bf16=False)
    qk_norm_rope(q, k, wq, wk, positions, eps=1e-6, theta=10000.0, gemma=False,
                 q_out=None, k_out=None)
    qk_norm_rope_ex(q, k, wq, wk, positions, ..., rotary_dim=None, interleaved=False,
                    llama3=None, mrope_sections=None, mrope_interleaved=False)
    ln_modulate(x, shift, scale, eps=1e-6, rows_per_sample=None, out=None)
    silu_and_mul(x, out=None)
    gelu_and_mul(x, out=None)
    gated_residual_ln_modulate(residual, y, gate, shift, scale, eps=1e-6,
                               rows_per_sample=None, out=None)
    kv_cache_write(k, v, slots, k_cache, v_cache, k_scale, v_scale)
    kv_cache_read(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, rows=None,
                  dtype=None, k_out=None, v_out=None)
    qk_norm_rope_cache(q, k, v, wq, wk, positions, slots, k_cache, v_cache, k_scale, v_scale,
                       ..., q_out=None)
    group_norm(x, groups, w=None, b=None, eps=1e-5, activation=None, out=None, stats=False)
    group_norm_backward(dy, x, mean, rstd, w=None, b=None, activation=None, dx=None)
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnormrope.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("%s is missing: build the CUDA library first "
                      "(python normalisation_rope_transformers_gb300/build.py)" % LIB_PATH)

lib = ctypes.CDLL(LIB_PATH)

_vp, _i64, _f32, _f64, _int = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                                ctypes.c_int)
lib.nr_rmsnorm.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _int, _f32, _int, _vp]
lib.nr_rmsnorm.restype = _int
lib.nr_rmsnorm_quant_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _int, _f32, _int, _f32,
                                     _vp]
lib.nr_rmsnorm_quant_fp8.restype = _int
lib.nr_qk_norm_rope.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _int, _vp, _i64, _i64, _i64, _i64,
                                _i64, _i64, _f32, _f64, _int, _int, _vp]
lib.nr_qk_norm_rope.restype = _int


class RopeConfig(ctypes.Structure):
    """Mirror of nr_rope_config (include/nr.h)."""
    _fields_ = [("rotary_dim", ctypes.c_int64), ("interleaved", ctypes.c_int32),
                ("mrope_interleaved", ctypes.c_int32), ("theta", ctypes.c_double),
                ("llama3_factor", ctypes.c_double), ("llama3_low_freq_factor", ctypes.c_double),
                ("llama3_high_freq_factor", ctypes.c_double),
                ("llama3_original_max_position", ctypes.c_double),
                ("mrope_section", ctypes.c_int32 * 3)]


lib.nr_qk_norm_rope_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _int, _vp, _i64, _i64, _i64,
                                   _i64, _i64, _i64, _f32, _int, ctypes.POINTER(RopeConfig), _int,
                                   _vp]
lib.nr_qk_norm_rope_ex.restype = _int
lib.nr_ln_modulate.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _f32, _int, _vp]
lib.nr_ln_modulate.restype = _int
lib.nr_gated_residual_ln_modulate.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                                              _f32, _int, _vp]
lib.nr_gated_residual_ln_modulate.restype = _int
lib.nr_silu_and_mul.argtypes = [_vp, _vp, _i64, _i64, _int, _vp]
lib.nr_silu_and_mul.restype = _int
lib.nr_gelu_and_mul.argtypes = [_vp, _vp, _i64, _i64, _int, _vp]
lib.nr_gelu_and_mul.restype = _int


class KvCache(ctypes.Structure):
    """Mirror of nr_kv_cache (include/nr.h)."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("blocks", ctypes.c_int64), ("block_size", ctypes.c_int64),
                ("heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("code_block_stride", ctypes.c_int64), ("scale_block_stride", ctypes.c_int64),
                ("format", ctypes.c_int)]


lib.nr_kv_cache_write.argtypes = [ctypes.POINTER(KvCache), _vp, _vp, _vp, _i64, _i64, _i64, _int,
                                  _vp]
lib.nr_kv_cache_write.restype = _int
lib.nr_qk_norm_rope_cache.argtypes = [ctypes.POINTER(KvCache), _vp, _vp, _vp, _vp, _vp, _vp, _int,
                                      _vp, _vp, _i64, _i64, _i64, _i64, _i64, _f32, _int,
                                      ctypes.POINTER(RopeConfig), _int, _vp]
lib.nr_qk_norm_rope_cache.restype = _int
lib.nr_kv_cache_read.argtypes = [_vp, _vp, ctypes.POINTER(KvCache), _vp, _i64, _vp, _i64, _i64,
                                 _int, _vp]
lib.nr_kv_cache_read.restype = _int
lib.nr_group_norm.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _int, _i64, _i64, _i64, _i64, _f32,
                              _int, _int, _vp, _i64, _vp]
lib.nr_group_norm.restype = _int
lib.nr_group_norm_backward.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _i64,
                                       _i64, _i64, _i64, _int, _int, _vp, _i64, _vp]
lib.nr_group_norm_backward.restype = _int
lib.nr_group_norm_workspace.argtypes = [_i64, _i64, _i64, _i64, _int, _int,
                                        ctypes.POINTER(_i64)]
lib.nr_group_norm_workspace.restype = _int
lib.nr_device_status.argtypes = [_vp]
lib.nr_device_status.restype = _int
lib.nr_test_wait_probe.argtypes = [_i64, _vp]
lib.nr_test_wait_probe.restype = _int
lib.nr_status_string.argtypes = [_int]
lib.nr_status_string.restype = ctypes.c_char_p
lib.nr_last_error_message.argtypes = []
lib.nr_last_error_message.restype = ctypes.c_char_p
lib.nr_version.argtypes = []
lib.nr_version.restype = _int

NR_F32 = 0
NR_BF16 = 1
NR_CACHE_FP8 = 0
NR_CACHE_MXFP4 = 1
NR_ACT_NONE = 0
NR_ACT_SILU = 1
ENTRY_POINTS = ("nr_rmsnorm", "nr_rmsnorm_quant_fp8", "nr_qk_norm_rope", "nr_qk_norm_rope_ex", "nr_ln_modulate",
                "nr_silu_and_mul", "nr_gelu_and_mul", "nr_gated_residual_ln_modulate",
                "nr_kv_cache_write", "nr_qk_norm_rope_cache", "nr_kv_cache_read",
                "nr_group_norm", "nr_group_norm_backward", "nr_group_norm_workspace",
                "nr_device_status", "nr_test_wait_probe",
                "nr_status_string", "nr_last_error_message", "nr_version")


class NrError(RuntimeError):
    """A non-OK nr_status from the library."""

    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (lib.nr_status_string(status).decode(), message))
        self.status = status


def _check(status: int):
    if status != 0:
        raise NrError(status, lib.nr_last_error_message().decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return NR_BF16
    if t.dtype == torch.float32:
        return NR_F32
    raise TypeError("tensors are bfloat16 or float32, got %s" % t.dtype)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _cuda(*ts):
    """Every tensor on one CUDA device (checked after the shapes, so that a
    shape error is reported as such whatever the device)."""
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must be on a CUDA device")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("tensors must all be on one CUDA device (%s and %s)" % (dev, t.device))


def _expect(t, name, dtype, shape, contiguous=True):
    """Raise unless `t` is a tensor of `dtype` and `shape` (and contiguous).
    The C ABI sees only pointers, so a short or mistyped operand would be read
    or written past its end; this is where the sizes are checked."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if contiguous and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _rows_2d(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError("%s must be a contiguous [rows, hidden] tensor" % name)
    _dtype_code(t)


def _heads_3d(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dim() != 3 or t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise ValueError("%s must be [tokens, heads, head_dim] with contiguous heads" % name)
    _dtype_code(t)


def _samples(t, name, dtype, rows, hidden, rows_per_sample):
    """A modulation operand: [hidden] (one sample) or [samples, hidden], with
    at least one sample per started group of rows_per_sample rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() not in (1, 2) or t.shape[-1] != hidden or not t.is_contiguous():
        raise ValueError("%s must be a contiguous [samples, %d] tensor, got %s"
                         % (name, hidden, tuple(t.shape)))
    need = -(-rows // rows_per_sample) if rows > 0 else 0
    have = 1 if t.dim() == 1 else t.shape[0]
    if have < need:
        raise ValueError("%s has %d sample rows; %d rows at %d rows per sample need %d"
                         % (name, have, rows, rows_per_sample, need))


def _rows_per_sample(rows_per_sample, rows):
    if rows_per_sample is None:
        return max(rows, 1)
    rps = int(rows_per_sample)
    if rps < 1:
        raise ValueError("rows_per_sample must be >= 1")
    return rps


def rmsnorm(x, w, residual=None, eps=1e-6, gemma=False, out=None):
    """RMSNorm of each row of x [rows, hidden]; with `residual`, first
    residual <- round(x + residual) in place.  Returns out."""
    _rows_2d(x, "x")
    _expect(w, "w", x.dtype, (x.shape[1],))
    if residual is not None:
        _expect(residual, "residual", x.dtype, x.shape)
    if out is not None:
        _expect(out, "out", x.dtype, x.shape)
    _cuda(x, w, residual, out)
    if out is None:
        out = torch.empty_like(x)
    _check(lib.nr_rmsnorm(_ptr(out), _ptr(x), _ptr(w), _ptr(residual), x.shape[0], x.shape[1],
                          _dtype_code(x), float(eps), int(bool(gemma)), _stream(x)))
    return out


def rmsnorm_quant_fp8(x, w, scale, residual=None, eps=1e-6, gemma=False, codes=None,
                      out_bf16=False):
    """RMSNorm of x [rows, hidden] (with the optional residual add), rounded to
    bf16, then e4m3 codes of that value * (1/scale).  Returns codes (uint8),
    or (codes, the bf16 values) when out_bf16 is True (or a tensor to fill)."""
    _rows_2d(x, "x")
    _expect(w, "w", x.dtype, (x.shape[1],))
    if residual is not None:
        _expect(residual, "residual", x.dtype, x.shape)
    if codes is not None:
        _expect(codes, "codes", torch.uint8, x.shape)
    nb = None
    if out_bf16 is not True and out_bf16 is not False and out_bf16 is not None:
        nb = out_bf16
        _expect(nb, "out_bf16", torch.bfloat16, x.shape)
    _cuda(x, w, residual, codes, nb)
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if out_bf16 is True:
        nb = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    _check(lib.nr_rmsnorm_quant_fp8(_ptr(codes), _ptr(nb), _ptr(x), _ptr(w), _ptr(residual),
                                    x.shape[0], x.shape[1], _dtype_code(x), float(eps),
                                    int(bool(gemma)), float(scale), _stream(x)))
    return codes if nb is None else (codes, nb)


def _check_qk(q, k, wq, wk, q_out, k_out):
    """q, k [tokens, heads, head_dim] of one dtype and token count; wq, wk
    [head_dim] of one dtype; outputs with the shapes, dtype and strides of
    their inputs."""
    _heads_3d(q, "q")
    _heads_3d(k, "k")
    if k.dtype != q.dtype:
        raise TypeError("q and k share one dtype")
    if k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
        raise ValueError("q %s and k %s must have the same tokens and head_dim"
                         % (tuple(q.shape), tuple(k.shape)))
    if not isinstance(wq, torch.Tensor) or wq.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("wq must be a float32 or bfloat16 tensor")
    _expect(wq, "wq", wq.dtype, (q.shape[2],))
    if wk is not None or k.shape[1] > 0:  # wk may be None when k has no heads
        _expect(wk, "wk", wq.dtype, (q.shape[2],))
    for o, i, name in ((q_out, q, "q_out"), (k_out, k, "k_out")):
        if o is None:
            continue
        _expect(o, name, i.dtype, i.shape, contiguous=False)
        if o.stride() != i.stride():
            raise ValueError("%s must have the strides of its input" % name)


def qk_norm_rope(q, k, wq, wk, positions, eps=1e-6, theta=10000.0, gemma=False, q_out=None,
                 k_out=None):
    """Per-head RMSNorm + NeoX RoPE of q [tokens, hq, D] and k [tokens, hk, D].
    q and k may be token-strided views (last two axes contiguous); outputs share
    their strides (q_out=q / k_out=k for in place).  Returns (q_out, k_out)."""
    _check_qk(q, k, wq, wk, q_out, k_out)
    _expect(positions, "positions", torch.int32, (q.shape[0],))
    _cuda(q, k, wq, wk, positions, q_out, k_out)
    if q_out is None:
        q_out = torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device)
    if k_out is None:
        k_out = torch.empty_strided(k.shape, k.stride(), dtype=k.dtype, device=k.device)
    _check(lib.nr_qk_norm_rope(_ptr(q_out), _ptr(k_out), _ptr(q), _ptr(k), _ptr(wq), _ptr(wk),
                               _dtype_code(wq), _ptr(positions), q.shape[0], q.shape[1],
                               k.shape[1], q.shape[2], q.stride(0), k.stride(0), float(eps),
                               float(theta), int(bool(gemma)), _dtype_code(q), _stream(q)))
    return q_out, k_out


def qk_norm_rope_ex(q, k, wq, wk, positions, eps=1e-6, gemma=False, rotary_dim=None,
                    interleaved=False, theta=10000.0, llama3=None, mrope_sections=None,
                    mrope_interleaved=False, q_out=None, k_out=None):
    """qk_norm_rope with the RoPE variants: rotary_dim (default head_dim), GPT-J
    interleaved pairs, Llama-3 rescale (llama3 = (factor, low_freq_factor,
    high_freq_factor, original_max_position)) and M-RoPE (positions [3, tokens],
    mrope_sections = (t, h, w)).  Returns (q_out, k_out)."""
    _check_qk(q, k, wq, wk, q_out, k_out)
    _expect(positions, "positions", torch.int32,
            (3, q.shape[0]) if mrope_sections is not None else (q.shape[0],))
    _cuda(q, k, wq, wk, positions, q_out, k_out)
    if q_out is None:
        q_out = torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device)
    if k_out is None:
        k_out = torch.empty_strided(k.shape, k.stride(), dtype=k.dtype, device=k.device)
    cfg = _rope_config(rotary_dim, interleaved, theta, llama3, mrope_sections, mrope_interleaved)
    _check(lib.nr_qk_norm_rope_ex(_ptr(q_out), _ptr(k_out), _ptr(q), _ptr(k), _ptr(wq), _ptr(wk),
                                  _dtype_code(wq), _ptr(positions), q.shape[0], q.shape[1],
                                  k.shape[1], q.shape[2], q.stride(0), k.stride(0), float(eps),
                                  int(bool(gemma)), ctypes.byref(cfg), _dtype_code(q), _stream(q)))
    return q_out, k_out


def _rope_config(rotary_dim, interleaved, theta, llama3, mrope_sections, mrope_interleaved):
    cfg = RopeConfig()
    cfg.rotary_dim = 0 if rotary_dim is None else int(rotary_dim)
    cfg.interleaved = int(bool(interleaved))
    cfg.mrope_interleaved = int(bool(mrope_interleaved))
    cfg.theta = float(theta)
    if llama3 is not None:
        (cfg.llama3_factor, cfg.llama3_low_freq_factor, cfg.llama3_high_freq_factor,
         cfg.llama3_original_max_position) = (float(v) for v in llama3)
    if mrope_sections is not None:
        for i, v in enumerate(mrope_sections):
            cfg.mrope_section[i] = int(v)
    return cfg


# Checked argument layouts of the calls below.  What the checks look at (types,
# shapes, strides and devices, no addresses and no values) is the key, with the
# options as plain numbers: an option may be a 0-d tensor, which counts with the
# value that it has at the call.  A layout that passed once costs one look-up;
# what they found is the entry.
_checked = {}
_CHECKED_MOST = 4096


def _layout(*ts):
    return tuple([None if t is None else (t.dtype, t.shape, t.stride(), t.get_device())
                  for t in ts])


def _remember(key, entry):
    if key is not None:
        if len(_checked) >= _CHECKED_MOST:
            _checked.clear()
        _checked[key] = entry
    return entry


def _known(*key_and_tensors):
    """(key, entry or None) of a call; no key for what is not a tensor (the
    checks then say so)."""
    name, options, ts = key_and_tensors
    try:
        key = (name, options, _layout(*ts))
        return key, _checked.get(key)
    except (AttributeError, TypeError, RuntimeError):
        return None, None


def _stream_of(device):
    return torch.cuda.current_stream(device).cuda_stream


# The same number by a private name, without making a Stream object each call,
# where torch has it; builds without CUDA do not.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)


def _launch(device, fn, *args):
    """fn(*args, the device's current stream) with `device` the current one: the
    library launches on the current device, and a default stream does not say
    which device it is of."""
    if device == torch.cuda.current_device():
        _check(fn(*args, _raw_stream(device)))
    else:
        with torch.cuda.device(device):
            _check(fn(*args, _raw_stream(device)))


def _block_strided(t, name):
    """The stride between blocks of a cache tensor whose blocks are contiguous."""
    inner = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != inner:
            raise ValueError("%s must be contiguous inside a block" % name)
        inner *= size
    if t.shape[0] > 1 and t.stride(0) < inner:
        raise ValueError("the blocks of %s overlap" % name)
    return t.stride(0) if t.shape[0] > 1 else inner


def _cache_layout(k_cache, v_cache, k_scale, v_scale):
    """The fields of KvCache behind its pointers, for four tensors: codes [blocks, block_size, heads, width] uint8
    and scales float32 [blocks, block_size, heads] (fp8, width = head_dim) or
    uint8 [blocks, block_size, heads, head_dim / 32] (mxfp4, width = head_dim / 2)."""
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache"), (k_scale, "k_scale"),
                    (v_scale, "v_scale")):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch tensor" % name)
    if k_cache.dtype != torch.uint8 or k_cache.dim() != 4:
        raise TypeError("k_cache must be uint8 codes [blocks, block_size, heads, width]")
    blocks, page, heads, width = k_cache.shape
    if k_scale.dtype == torch.float32:
        fmt, dim, scales = NR_CACHE_FP8, width, (blocks, page, heads)
    elif k_scale.dtype == torch.uint8:
        fmt, dim, scales = NR_CACHE_MXFP4, 2 * width, (blocks, page, heads, width // 16)
    else:
        raise TypeError("k_scale must be float32 (fp8) or uint8 (mxfp4), got %s" % k_scale.dtype)
    _expect(v_cache, "v_cache", torch.uint8, k_cache.shape, contiguous=False)
    _expect(k_scale, "k_scale", k_scale.dtype, scales, contiguous=False)
    _expect(v_scale, "v_scale", k_scale.dtype, scales, contiguous=False)
    code = _block_strided(k_cache, "k_cache")
    scale = _block_strided(k_scale, "k_scale")
    if _block_strided(v_cache, "v_cache") != code or _block_strided(v_scale, "v_scale") != scale:
        raise ValueError("the K and V parts of the cache must have the same block strides")
    return blocks, page, heads, dim, code, scale * k_scale.element_size(), fmt


def _kv_cache(layout, k_cache, v_cache, k_scale, v_scale):
    return KvCache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                   *layout)


def _check_kv(k, v, slots, heads, dim):
    _heads_3d(k, "k")
    _heads_3d(v, "v")
    if v.dtype != k.dtype:
        raise TypeError("k and v share one dtype")
    shape = (k.shape[0], heads, dim)
    for t, name in ((k, "k"), (v, "v")):
        if tuple(t.shape) != shape:
            raise ValueError("%s must be [tokens, %d, %d] for this cache, got %s"
                             % (name, heads, dim, tuple(t.shape)))
    _expect(slots, "slots", torch.int64, (k.shape[0],))


def _tok_stride(t):
    """Elements between tokens (a single token's stride says nothing)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def kv_cache_write(k, v, slots, k_cache, v_cache, k_scale, v_scale):
    """Quantises k and v [tokens, heads, head_dim] into the places `slots`
    (int64, block * block_size + place; outside the cache: padding, skipped) of
    a paged cache: uint8 codes [blocks, block_size, heads, head_dim] with
    float32 scales [blocks, block_size, heads] (fp8), or codes of width
    head_dim / 2 with uint8 scales [blocks, block_size, heads, head_dim / 32]
    (mxfp4).  k and v may be token-strided, the cache's parts block-strided."""
    key, known = _known("write", None, (k, v, slots, k_cache, v_cache, k_scale, v_scale))
    if known is None:
        layout = _cache_layout(k_cache, v_cache, k_scale, v_scale)
        _check_kv(k, v, slots, layout[2], layout[3])
        _cuda(k, v, slots, k_cache, v_cache, k_scale, v_scale)
        known = _remember(key, (layout, (k.shape[0], _tok_stride(k), _tok_stride(v),
                                         _dtype_code(k)), k.get_device()))
    layout, sizes, device = known
    _launch(device, lib.nr_kv_cache_write, _kv_cache(layout, k_cache, v_cache, k_scale, v_scale),
            k.data_ptr(), v.data_ptr(), slots.data_ptr(), *sizes)


def qk_norm_rope_cache(q, k, v, wq, wk, positions, slots, k_cache, v_cache, k_scale, v_scale,
                       eps=1e-6, gemma=False, rotary_dim=None, interleaved=False, theta=10000.0,
                       llama3=None, mrope_sections=None, mrope_interleaved=False, q_out=None):
    """qk_norm_rope_ex with K (quantised from its f32 value) and V written into
    the cache as kv_cache_write does.  Returns q_out."""
    eps, theta, gemma = float(eps), float(theta), bool(gemma)
    interleaved, mrope_interleaved = bool(interleaved), bool(mrope_interleaved)
    if rotary_dim is not None:
        rotary_dim = int(rotary_dim)
    if llama3 is not None:
        llama3 = tuple([float(v) for v in llama3])
    if mrope_sections is not None:
        mrope_sections = tuple([int(v) for v in mrope_sections])
    options = (eps, gemma, rotary_dim, interleaved, theta, llama3, mrope_sections,
               mrope_interleaved)
    key, known = _known("fused", options, (q, k, v, wq, wk, positions, slots, k_cache, v_cache,
                                           k_scale, v_scale, q_out))
    if known is None:
        layout = _cache_layout(k_cache, v_cache, k_scale, v_scale)
        _check_kv(k, v, slots, layout[2], layout[3])
        _check_qk(q, k, wq, wk, q_out, None)
        _expect(positions, "positions", torch.int32,
                (3, q.shape[0]) if mrope_sections is not None else (q.shape[0],))
        _cuda(q, k, v, wq, wk, positions, slots, k_cache, v_cache, k_scale, v_scale, q_out)
        cfg = _rope_config(rotary_dim, interleaved, theta, llama3, mrope_sections,
                           mrope_interleaved)
        known = _remember(key, (layout, _dtype_code(wq),
                                (q.shape[0], q.shape[1], _tok_stride(q), _tok_stride(k),
                                 _tok_stride(v), eps, int(gemma), cfg,
                                 _dtype_code(q)), q.get_device()))
    layout, wcode, sizes, device = known
    if q_out is None:
        q_out = torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device)
    _launch(device, lib.nr_qk_norm_rope_cache,
            _kv_cache(layout, k_cache, v_cache, k_scale, v_scale), q_out.data_ptr(), q.data_ptr(),
            k.data_ptr(), v.data_ptr(), wq.data_ptr(), wk.data_ptr(), wcode, positions.data_ptr(),
            slots.data_ptr(), *sizes)
    return q_out


def kv_cache_read(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, rows=None,
                  dtype=None, k_out=None, v_out=None):
    """Reads sequences back from the cache: row cu_seqlens[s] + t of k and v
    [rows, heads, head_dim] is token t of sequence s, found through
    block_table [seqs, n] int32; cu_seqlens is [seqs + 1] int32.  Give `rows`
    (at least cu_seqlens[-1], which is not read on the host) or outputs to fill;
    `dtype` is float32 or bfloat16 (the outputs', else bfloat16).  Rows behind
    the last sequence are left as they were (in outputs made here: anything).
    Returns (k, v)."""
    if rows is not None:
        rows = int(rows)
    key, known = _known("read", (rows, dtype), (k_cache, v_cache, k_scale, v_scale, block_table,
                                                cu_seqlens, k_out, v_out))
    if known is None:
        layout = _cache_layout(k_cache, v_cache, k_scale, v_scale)
        if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
            raise ValueError("block_table must be a [seqs, blocks] tensor")
        _expect(block_table, "block_table", torch.int32, block_table.shape)
        _expect(cu_seqlens, "cu_seqlens", torch.int32, (block_table.shape[0] + 1,))
        for t in (k_out, v_out):
            if isinstance(t, torch.Tensor):
                rows = t.shape[0] if rows is None and t.dim() == 3 else rows
                dtype = t.dtype if dtype is None else dtype
        dtype = torch.bfloat16 if dtype is None else dtype
        if rows is None:
            raise ValueError("kv_cache_read needs rows or outputs [rows, heads, head_dim]")
        if rows < 0:
            raise ValueError("rows must be >= 0")
        if dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("dtype must be bfloat16 or float32, got %s" % dtype)
        shape = (rows, layout[2], layout[3])
        for t, name in ((k_out, "k_out"), (v_out, "v_out")):
            if t is not None:
                _expect(t, name, dtype, shape)
        _cuda(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, k_out, v_out)
        known = _remember(key, (layout, shape, dtype, k_cache.device, block_table.shape[1],
                                (block_table.shape[0], shape[0],
                                 NR_BF16 if dtype == torch.bfloat16 else NR_F32)))
    layout, shape, dtype, device, width, sizes = known
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=dtype, device=device)
    _launch(device.index, lib.nr_kv_cache_read, k_out.data_ptr(), v_out.data_ptr(),
            _kv_cache(layout, k_cache, v_cache, k_scale, v_scale), block_table.data_ptr(), width,
            cu_seqlens.data_ptr(), *sizes)
    return k_out, v_out


def _activation(name):
    if name is None or name == "none":
        return NR_ACT_NONE
    if name == "silu":
        return NR_ACT_SILU
    raise ValueError("activation must be None or 'silu', got %r" % (name,))


def _group_norm_workspace(samples, space, channels, groups, backward, code):
    n = ctypes.c_int64()
    _check(lib.nr_group_norm_workspace(samples, space, channels, groups, backward, code,
                                       ctypes.byref(n)))
    return n.value


def _check_norm(x, w, b):
    """x [samples, ..., channels] and its affine parameters; (samples, space,
    channels, dtype code of the parameters)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch tensor")
    if x.dim() < 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous [samples, ..., channels] tensor")
    code = _dtype_code(x)
    samples, channels = x.shape[0], x.shape[-1]
    if (w is None) != (b is None):
        raise ValueError("w and b are given together or not at all")
    if w is not None:
        if not isinstance(w, torch.Tensor) or w.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("w must be a float32 or bfloat16 tensor")
        _expect(w, "w", w.dtype, (channels,))
        _expect(b, "b", w.dtype, (channels,))
        code = _dtype_code(w)
    space = 1
    for n in x.shape[1:-1]:
        space *= n
    return samples, space, channels, code


def group_norm(x, groups, w=None, b=None, eps=1e-5, activation=None, out=None, stats=False):
    """Group norm of x [samples, ..., channels] (contiguous, any number of axes
    between; a torch channels_last [N, C, H, W] is x.permute(0, 2, 3, 1)) with w and b [channels] (float32 or bfloat16; both or
    neither), then `activation` (None or "silu").  Returns out, or (out, mean,
    rstd) with stats=True: the [samples, groups] float32 statistics that
    group_norm_backward takes.  No autograd graph is recorded: the gradient is
    a call of its own."""
    groups, eps, act = int(groups), float(eps), _activation(activation)
    key, known = _known("norm", (groups, eps, act), (x, w, b, out))
    if known is None:
        samples, space, channels, wcode = _check_norm(x, w, b)
        if groups < 1 or channels % groups:
            raise ValueError("%d channels do not divide into %d groups" % (channels, groups))
        if out is not None:
            _expect(out, "out", x.dtype, x.shape)
        _cuda(x, w, b, out)
        code = _dtype_code(x)
        known = _remember(key, (wcode, (samples, space, channels, groups, eps, act, code),
                                _group_norm_workspace(samples, space, channels, groups, 0, code),
                                x.device))
    wcode, sizes, need, device = known
    if out is None:
        out = torch.empty_like(x)
    shape = (sizes[0], sizes[3])
    # with no elements nothing is written
    held = torch.empty if sizes[1] else torch.zeros
    mean = held(shape, dtype=torch.float32, device=device)
    rstd = held(shape, dtype=torch.float32, device=device)
    workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _launch(device.index, lib.nr_group_norm, out.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
            x.data_ptr(), None if w is None else w.data_ptr(), None if b is None else b.data_ptr(),
            wcode, *sizes, None if workspace is None else workspace.data_ptr(), need)
    return (out, mean, rstd) if stats else out


def group_norm_backward(dy, x, mean, rstd, w=None, b=None, activation=None, dx=None):
    """The gradient of group_norm: dy and x [samples, ..., channels], the mean
    and rstd that it returned, the same w, b and activation.  Returns (dx, dw,
    db); dw and db have w's dtype (None without w).  dx may be dy or x."""
    act = _activation(activation)
    key, known = _known("norm back", act, (dy, x, mean, rstd, w, b, dx))
    if known is None:
        samples, space, channels, wcode = _check_norm(x, w, b)
        _expect(dy, "dy", x.dtype, x.shape)
        if not isinstance(mean, torch.Tensor) or mean.dim() != 2:
            raise ValueError("mean must be a [samples, groups] tensor")
        groups = mean.shape[1]
        _expect(mean, "mean", torch.float32, (samples, groups))
        _expect(rstd, "rstd", torch.float32, (samples, groups))
        if groups < 1 or channels % groups:
            raise ValueError("%d channels do not divide into %d groups" % (channels, groups))
        if dx is not None:
            _expect(dx, "dx", x.dtype, x.shape)
        _cuda(x, dy, mean, rstd, w, b, dx)
        code = _dtype_code(x)
        known = _remember(key, (wcode, (samples, space, channels, groups, act, code),
                                _group_norm_workspace(samples, space, channels, groups, 1, code),
                                x.device))
    wcode, sizes, need, device = known
    if dx is None:
        dx = torch.empty_like(x)
    dw = db = pw = pb = pdw = pdb = None
    if w is not None:
        held = torch.empty_like if sizes[0] and sizes[1] else torch.zeros_like
        dw, db = held(w), held(b)
        pw, pb, pdw, pdb = w.data_ptr(), b.data_ptr(), dw.data_ptr(), db.data_ptr()
    workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _launch(device.index, lib.nr_group_norm_backward, dx.data_ptr(), pdw, pdb, dy.data_ptr(),
            x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), pw, pb, wcode, *sizes,
            None if workspace is None else workspace.data_ptr(), need)
    return dx, dw, db


def ln_modulate(x, shift, scale, eps=1e-6, rows_per_sample=None, out=None):
    """LayerNorm (no affine) of x [rows, hidden] then * (1 + scale) + shift,
    with shift/scale [samples, hidden] (row r uses sample r // rows_per_sample).
    Returns out."""
    _rows_2d(x, "x")
    rows_per_sample = _rows_per_sample(rows_per_sample, x.shape[0])
    for t, name in ((shift, "shift"), (scale, "scale")):
        _samples(t, name, x.dtype, x.shape[0], x.shape[1], rows_per_sample)
    if out is not None:
        _expect(out, "out", x.dtype, x.shape)
    _cuda(x, shift, scale, out)
    if out is None:
        out = torch.empty_like(x)
    _check(lib.nr_ln_modulate(_ptr(out), _ptr(x), _ptr(shift), _ptr(scale), x.shape[0],
                              x.shape[1], int(rows_per_sample), float(eps), _dtype_code(x),
                              _stream(x)))
    return out


def gated_residual_ln_modulate(residual, y, gate, shift, scale, eps=1e-6, rows_per_sample=None,
                               out=None):
    """residual <- round(residual + gate * y) in place, then LayerNorm (no affine)
    of it * (1 + scale) + shift.  gate/shift/scale are [samples, hidden]; row r
    uses sample r // rows_per_sample.  Returns out."""
    _rows_2d(residual, "residual")
    _expect(y, "y", residual.dtype, residual.shape)
    rows, hidden = residual.shape
    rows_per_sample = _rows_per_sample(rows_per_sample, rows)
    for t, name in ((gate, "gate"), (shift, "shift"), (scale, "scale")):
        _samples(t, name, residual.dtype, rows, hidden, rows_per_sample)
    if out is not None:
        _expect(out, "out", residual.dtype, residual.shape)
    _cuda(residual, y, gate, shift, scale, out)
    if out is None:
        out = torch.empty_like(residual)
    _check(lib.nr_gated_residual_ln_modulate(
        _ptr(out), _ptr(residual), _ptr(y), _ptr(gate), _ptr(shift), _ptr(scale),
        residual.shape[0], residual.shape[1], int(rows_per_sample), float(eps),
        _dtype_code(residual), _stream(residual)))
    return out


def _act_and_mul(fn, x, out):
    _rows_2d(x, "x")
    if x.shape[1] % 2:
        raise ValueError("x must be a contiguous [rows, 2*inter] tensor")
    inter = x.shape[1] // 2
    if out is not None:
        _expect(out, "out", x.dtype, (x.shape[0], inter))
    _cuda(x, out)
    if out is None:
        out = torch.empty((x.shape[0], inter), dtype=x.dtype, device=x.device)
    _check(fn(_ptr(out), _ptr(x), x.shape[0], inter, _dtype_code(x), _stream(x)))
    return out


def device_status(device=None):
    """Wait for the current stream of `device` and raise NrError
    (NR_ERR_TIMEOUT) if a kernel gave up a bounded wait since the last check."""
    _check(lib.nr_device_status(torch.cuda.current_stream(device).cuda_stream))


def wait_probe(limit_cycles=100000, device=None):
    """Launch the library's wait probe: one wait that nothing completes, given
    up after `limit_cycles` SM clock cycles (the next device_status() raises)."""
    _check(lib.nr_test_wait_probe(int(limit_cycles), torch.cuda.current_stream(device).cuda_stream))


def silu_and_mul(x, out=None):
    """silu(x[:, :I]) * x[:, I:] for x [rows, 2I].  Returns out [rows, I]."""
    return _act_and_mul(lib.nr_silu_and_mul, x, out)


def gelu_and_mul(x, out=None):
    """gelu_tanh(x[:, :I]) * x[:, I:] for x [rows, 2I].  Returns out [rows, I]."""
    return _act_and_mul(lib.nr_gelu_and_mul, x, out)


__all__ = ["rmsnorm", "rmsnorm_quant_fp8", "qk_norm_rope", "qk_norm_rope_ex", "RopeConfig", "ln_modulate",
           "silu_and_mul", "gelu_and_mul", "device_status", "wait_probe",
           "gated_residual_ln_modulate", "kv_cache_write", "kv_cache_read", "qk_norm_rope_cache",
           "group_norm", "group_norm_backward", "KvCache", "NrError", "lib",
           "LIB_PATH", "ENTRY_POINTS", "NR_F32", "NR_BF16", "NR_CACHE_FP8", "NR_CACHE_MXFP4",
           "NR_ACT_NONE", "NR_ACT_SILU"]
