"""The cache and group-norm entry points on the CPU: every refusal of the C ABI
and of the binding comes before a launch, and the reference that the GPU tests
use agrees with the formats' definitions."""
import ctypes

import numpy as np
import pytest
import torch

from tests import cache_ref as ref
from tests.test_abi_host import (ALIAS, ALIGN, DTYPE, F32, BF16, NULL, OK, SHAPE, UNSUP, VALUE, A,
                                 MB, RopeConfig)


class KvCache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("blocks", ctypes.c_int64), ("block_size", ctypes.c_int64),
                ("heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("code_block_stride", ctypes.c_int64), ("scale_block_stride", ctypes.c_int64),
                ("format", ctypes.c_int)]


@pytest.fixture(scope="module")
def lib(lib_path):
    import normalisation_rope_transformers_gb300 as nrt
    return nrt.lib


@pytest.fixture(scope="module")
def nrt(lib_path):
    import normalisation_rope_transformers_gb300 as nrt
    return nrt


def cache(fmt=0, heads=2, dim=64, blocks=4, page=16, **kw):
    """A cache at fake addresses, 16 MB apart."""
    width, per = (dim, 4) if fmt == 0 else (dim // 2, dim // 32)
    c = KvCache(A, A + 16 * MB, A + 32 * MB, A + 48 * MB, blocks, page, heads, dim,
                page * heads * width, page * heads * per, fmt)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


# device-like addresses of the other operands
K, V, SLOTS, Q, QO, W, POS, OUT, TABLE, CU = (A + (64 + 16 * i) * MB for i in range(10))


def cast(c, nrt):
    return None if c is None else ctypes.cast(ctypes.byref(c), ctypes.POINTER(nrt.KvCache))


def write(nrt, c, k=K, v=V, slots=SLOTS, tokens=3, ks=None, vs=None, dtype=BF16):
    row = 128 if c is None else c.heads * c.head_dim
    return nrt.lib.nr_kv_cache_write(cast(c, nrt), k, v, slots, tokens, row if ks is None else ks,
                                     row if vs is None else vs, dtype, None)


CACHE_ERRORS = [
    (dict(format=7), DTYPE), (dict(blocks=0), SHAPE), (dict(block_size=0), SHAPE),
    (dict(heads=0), SHAPE), (dict(head_dim=0), SHAPE), (dict(head_dim=24), UNSUP),
    (dict(head_dim=528), UNSUP), (dict(heads=1 << 20), SHAPE), (dict(blocks=1 << 40), SHAPE),
    (dict(code_block_stride=64), SHAPE), (dict(scale_block_stride=4), SHAPE),
    (dict(code_block_stride=16 * 128 + 8), ALIGN), (dict(scale_block_stride=16 * 8 + 2), ALIGN),
    (dict(code_block_stride=1 << 62), SHAPE), (dict(k_codes=None), NULL), (dict(v_scales=None), NULL),
    (dict(v_codes=A + 16 * MB + 8), ALIGN), (dict(k_scales=A + 32 * MB + 2), ALIGN),
    (dict(v_codes=A), ALIAS), (dict(k_scales=A + 64), ALIAS), (dict(v_scales=A + 32 * MB), ALIAS),
]


@pytest.mark.parametrize("kw,want", CACHE_ERRORS)
def test_bad_caches_are_refused(nrt, kw, want):
    assert write(nrt, cache(**kw)) == want, nrt.lib.nr_last_error_message()


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE), (dict(dtype=5), DTYPE),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(ks=127), SHAPE),
    (dict(vs=132), ALIGN), (dict(k=K + 8), ALIGN), (dict(slots=SLOTS + 4), ALIGN),
    (dict(k=A + 64), ALIAS), (dict(slots=A + 32 * MB), ALIAS), (dict(tokens=0, k=None), OK),
])
def test_bad_writes_are_refused(nrt, kw, want):
    assert write(nrt, cache(), **kw) == want, nrt.lib.nr_last_error_message()


def test_null_cache_and_mxfp4_head_dim(nrt):
    assert write(nrt, None) == NULL
    assert write(nrt, cache(fmt=1, dim=48)) == UNSUP
    assert write(nrt, cache(fmt=1, dim=96), tokens=0) == OK


def fused(nrt, c, rope=None, q=Q, qo=QO, tokens=3, hq=4, wq=W, pos=POS, dtype=BF16, eps=1e-6,
          gemma=0, qs=None, slots=SLOTS):
    rope = RopeConfig(theta=1e4) if rope is None else rope
    row = c.heads * c.head_dim
    return nrt.lib.nr_qk_norm_rope_cache(
        cast(c, nrt), qo, q, K, V, wq, W, F32, pos, slots, tokens, hq,
        hq * c.head_dim if qs is None else qs, row, row, eps, gemma,
        ctypes.cast(ctypes.byref(rope), ctypes.POINTER(nrt.RopeConfig)) if rope else None, dtype,
        None)


@pytest.mark.parametrize("kw,want", [
    (dict(c=cache(dim=96)), UNSUP), (dict(c=cache(dim=48)), UNSUP),
    (dict(c=cache(dim=512), dtype=F32), UNSUP), (dict(c=cache(dim=32)), UNSUP),
    (dict(c=cache(fmt=1, dim=32), dtype=F32), UNSUP),
    (dict(c=cache(fmt=1, dim=128), rope=RopeConfig(theta=1e4, rotary_dim=32)), UNSUP),
    (dict(c=cache(), rope=RopeConfig(theta=0.0)), VALUE),
    (dict(c=cache(), rope=RopeConfig(theta=1e4, rotary_dim=80)), SHAPE),
    (dict(c=cache(), rope=RopeConfig(theta=1e4, rotary_dim=24)), UNSUP),
    (dict(c=cache(), eps=-1.0), VALUE), (dict(c=cache(), gemma=2), VALUE),
    (dict(c=cache(), hq=0), SHAPE), (dict(c=cache(), qs=100), SHAPE),
    (dict(c=cache(), qs=260), ALIGN), (dict(c=cache(), q=None), NULL),
    (dict(c=cache(), pos=None), NULL), (dict(c=cache(), pos=POS + 2), ALIGN),
    (dict(c=cache(), qo=Q + 16), ALIAS), (dict(c=cache(), qo=K), ALIAS),
    (dict(c=cache(), qo=A + 64), ALIAS), (dict(c=cache(), slots=QO), ALIAS),
    (dict(c=cache(), tokens=0, q=None), OK),
])
def test_bad_preambles_are_refused(nrt, kw, want):
    kw = dict(kw)
    assert fused(nrt, kw.pop("c"), **kw) == want, nrt.lib.nr_last_error_message()


def test_a_null_rope_config_is_refused(nrt):
    c = cache()
    assert nrt.lib.nr_qk_norm_rope_cache(cast(c, nrt), QO, Q, K, V, W, W, F32, POS, SLOTS, 3, 2, 128,
                                         128, 128, 1e-6, 0, None, BF16, None) == NULL


def read(nrt, c, ko=OUT, vo=OUT + 16 * MB, table=TABLE + 64 * MB, width=2, cu=CU + 64 * MB, seqs=2,
         rows=20, dtype=BF16):
    return nrt.lib.nr_kv_cache_read(ko, vo, cast(c, nrt), table, width, cu, seqs, rows, dtype, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), SHAPE), (dict(seqs=-1), SHAPE), (dict(width=-1), SHAPE),
    (dict(rows=1 << 31), SHAPE), (dict(dtype=9), DTYPE), (dict(ko=None), NULL),
    (dict(cu=None), NULL), (dict(table=None), NULL), (dict(ko=OUT + 8), ALIGN),
    (dict(cu=CU + 2), ALIGN), (dict(vo=OUT + 64), ALIAS), (dict(ko=A), ALIAS),
    (dict(table=OUT), ALIAS), (dict(rows=0, ko=None), OK), (dict(seqs=0, ko=None), OK),
])
def test_bad_reads_are_refused(nrt, kw, want):
    assert read(nrt, cache(), **kw) == want, nrt.lib.nr_last_error_message()


def gn(nrt, out=OUT, mean=Q, rstd=QO, x=K, w=V, b=W, wd=F32, n=2, s=100, c=64, g=8, eps=1e-5, act=0,
       dtype=BF16, ws=POS, wsb=1 << 20):
    return nrt.lib.nr_group_norm(out, mean, rstd, x, w, b, wd, n, s, c, g, eps, act, dtype, ws, wsb,
                                 None)


BIG = dict(n=1, s=1 << 16, c=64, g=8)  # beyond the one-launch kernel: needs a workspace


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), DTYPE), (dict(wd=3), DTYPE), (dict(n=-1), SHAPE), (dict(s=-1), SHAPE),
    (dict(c=0), SHAPE), (dict(g=0), SHAPE), (dict(g=7), SHAPE), (dict(c=60, g=6), UNSUP),
    (dict(c=65544, g=1), UNSUP), (dict(s=1 << 60), SHAPE), (dict(n=1 << 31), SHAPE),
    (dict(eps=-1.0), VALUE), (dict(eps=float("nan")), VALUE), (dict(act=2), VALUE),
    (dict(out=None), NULL), (dict(mean=None), NULL), (dict(w=None), NULL), (dict(b=None), NULL),
    (dict(ws=None, **BIG), NULL), (dict(wsb=64, **BIG), SHAPE), (dict(out=OUT + 8), ALIGN),
    (dict(rstd=QO + 2), ALIGN), (dict(out=K + 16), ALIAS), (dict(out=V), ALIAS),
    (dict(mean=QO), ALIAS), (dict(mean=K), ALIAS), (dict(ws=K, **BIG), ALIAS),
    (dict(n=0, out=None), OK), (dict(s=0, out=None), OK),
])
def test_bad_group_norms_are_refused(nrt, kw, want):
    assert gn(nrt, **kw) == want, nrt.lib.nr_last_error_message()


def gnb(nrt, dx=OUT, dw=TABLE, db=CU, dy=SLOTS, x=K, mean=Q, rstd=QO, w=V, b=W, wd=F32, n=2, s=100,
        c=64, g=8, act=0, dtype=BF16, ws=POS, wsb=1 << 20):
    return nrt.lib.nr_group_norm_backward(dx, dw, db, dy, x, mean, rstd, w, b, wd, n, s, c, g, act,
                                          dtype, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), NULL), (dict(dw=None), NULL), (dict(db=None), NULL),
    (dict(w=None, b=None), NULL), (dict(ws=None), NULL), (dict(wsb=8), SHAPE),
    (dict(dw=TABLE + 4), ALIGN), (dict(dx=K + 16), ALIAS), (dict(dw=K), ALIAS),
    (dict(db=TABLE), ALIAS), (dict(ws=OUT), ALIAS), (dict(act=-1), VALUE), (dict(n=0, dy=None), OK),
])
def test_bad_group_norm_gradients_are_refused(nrt, kw, want):
    assert gnb(nrt, **kw) == want, nrt.lib.nr_last_error_message()


def test_workspace_query(nrt):
    n = ctypes.c_int64(-1)
    q = nrt.lib.nr_group_norm_workspace
    assert q(2, 100, 64, 8, 0, BF16, ctypes.byref(n)) == OK and n.value == 0
    assert q(1, 1 << 16, 64, 8, 0, BF16, ctypes.byref(n)) == OK and n.value > 0
    assert q(0, 100, 64, 8, 1, BF16, ctypes.byref(n)) == OK and n.value == 0
    assert q(2, 100, 64, 8, 1, F32, ctypes.byref(n)) == OK and n.value > 0
    assert q(2, 100, 64, 8, 2, F32, ctypes.byref(n)) == VALUE
    assert q(2, 100, 64, 8, 0, F32, None) == NULL
    assert q(2, 100, 64, 7, 0, F32, ctypes.byref(n)) == SHAPE


# ---------------------------------------------------------------------------
# the binding's own checks (host tensors: a call that passes them stops at the
# device check)
# ---------------------------------------------------------------------------
bf = torch.bfloat16


def parts(fmt="fp8", blocks=3, page=4, heads=2, dim=64):
    if fmt == "fp8":
        c, s = (blocks, page, heads, dim), torch.zeros(blocks, page, heads)
    else:
        c = (blocks, page, heads, dim // 2)
        s = torch.zeros(blocks, page, heads, dim // 32, dtype=torch.uint8)
    return [torch.zeros(c, dtype=torch.uint8), torch.zeros(c, dtype=torch.uint8), s, s.clone()]


def kv(t=5, heads=2, dim=64, dtype=bf):
    return torch.zeros(t, heads, dim, dtype=dtype)


def slots(t=5):
    return torch.zeros(t, dtype=torch.int64)


def swapped(i, t):
    p = parts()
    p[i] = t
    return p


I32 = torch.int32
BAD = {
    "v dtype": lambda b: b.kv_cache_write(kv(), kv(dtype=torch.float32), slots(), *parts()),
    "k heads": lambda b: b.kv_cache_write(kv(heads=3), kv(heads=3), slots(), *parts()),
    "v tokens": lambda b: b.kv_cache_write(kv(), kv(t=4), slots(), *parts()),
    "k head_dim": lambda b: b.kv_cache_write(kv(dim=32), kv(dim=32), slots(), *parts()),
    "half k": lambda b: b.kv_cache_write(kv(dtype=torch.float16), kv(dtype=torch.float16), slots(),
                                         *parts()),
    "int32 slots": lambda b: b.kv_cache_write(kv(), kv(), slots().int(), *parts()),
    "short slots": lambda b: b.kv_cache_write(kv(), kv(), slots(4), *parts()),
    "strided slots": lambda b: b.kv_cache_write(kv(), kv(), slots(10)[::2], *parts()),
    "strided heads": lambda b: b.kv_cache_write(torch.zeros(5, 64, 2, dtype=bf).transpose(1, 2), kv(),
                                                slots(), *parts()),
    "codes dtype": lambda b: b.kv_cache_write(kv(), kv(), slots(),
                                              *swapped(0, torch.zeros(3, 4, 2, 64))),
    "v codes shape": lambda b: b.kv_cache_write(
        kv(), kv(), slots(), *swapped(1, torch.zeros(2, 4, 2, 64, dtype=torch.uint8))),
    "scale dtype": lambda b: b.kv_cache_write(
        kv(), kv(), slots(), *swapped(2, torch.zeros(3, 4, 2, dtype=torch.float16))),
    "scale shape": lambda b: b.kv_cache_write(kv(), kv(), slots(), *swapped(3, torch.zeros(3, 4, 1))),
    "mixed scales": lambda b: b.kv_cache_write(
        kv(), kv(), slots(), *swapped(3, torch.zeros(3, 4, 2, dtype=torch.uint8))),
    "block not contiguous": lambda b: b.kv_cache_write(
        kv(), kv(), slots(), *swapped(0, torch.zeros(3, 2, 4, 64, dtype=torch.uint8).transpose(1, 2))),
    "different block strides": lambda b: b.kv_cache_write(
        kv(), kv(), slots(), *swapped(0, torch.zeros(3, 2, 4, 2, 64, dtype=torch.uint8)[:, 0])),
    "not a tensor": lambda b: b.kv_cache_write(kv(), kv(), None, *parts()),
    "no cache": lambda b: b.kv_cache_write(kv(), kv(), slots(), None, *parts()[1:]),
    "fused q dim": lambda b: b.qk_norm_rope_cache(kv(dim=32), kv(), kv(), torch.ones(64),
                                                  torch.ones(64), slots().int(), slots(), *parts()),
    "fused positions": lambda b: b.qk_norm_rope_cache(kv(), kv(), kv(), torch.ones(64),
                                                      torch.ones(64), slots(), slots(), *parts()),
    "fused wk": lambda b: b.qk_norm_rope_cache(kv(), kv(), kv(), torch.ones(64), torch.ones(32),
                                               slots().int(), slots(), *parts()),
    "fused v": lambda b: b.qk_norm_rope_cache(kv(), kv(), kv(t=4), torch.ones(64), torch.ones(64),
                                              slots().int(), slots(), *parts()),
    "fused q_out": lambda b: b.qk_norm_rope_cache(kv(), kv(), kv(), torch.ones(64), torch.ones(64),
                                                  slots().int(), slots(), *parts(), q_out=kv(t=4)),
    "read table": lambda b: b.kv_cache_read(*parts(), torch.zeros(2, 2), torch.zeros(3, dtype=I32), 4),
    "read table 1d": lambda b: b.kv_cache_read(*parts(), torch.zeros(2, dtype=I32),
                                               torch.zeros(3, dtype=I32), 4),
    "read cu": lambda b: b.kv_cache_read(*parts(), torch.zeros(2, 2, dtype=I32),
                                         torch.zeros(2, dtype=I32), 4),
    "read no rows": lambda b: b.kv_cache_read(*parts(), torch.zeros(2, 2, dtype=I32),
                                              torch.zeros(3, dtype=I32)),
    "read rows < 0": lambda b: b.kv_cache_read(*parts(), torch.zeros(2, 2, dtype=I32),
                                               torch.zeros(3, dtype=I32), -1),
    "read dtype": lambda b: b.kv_cache_read(*parts(), torch.zeros(2, 2, dtype=I32),
                                            torch.zeros(3, dtype=I32), 4, dtype=torch.float16),
    "read k_out": lambda b: b.kv_cache_read(*parts(), torch.zeros(2, 2, dtype=I32),
                                            torch.zeros(3, dtype=I32), 4, k_out=kv(t=3)),
    "norm groups": lambda b: b.group_norm(torch.zeros(2, 5, 64, dtype=bf), 7),
    "norm no groups": lambda b: b.group_norm(torch.zeros(2, 5, 64, dtype=bf), 0),
    "norm 1d": lambda b: b.group_norm(torch.zeros(64, dtype=bf), 8),
    "norm strided": lambda b: b.group_norm(torch.zeros(2, 64, 5, dtype=bf).transpose(1, 2), 8),
    "norm half": lambda b: b.group_norm(torch.zeros(2, 5, 64, dtype=torch.float16), 8),
    "norm w alone": lambda b: b.group_norm(torch.zeros(2, 5, 64), 8, torch.ones(64)),
    "norm w length": lambda b: b.group_norm(torch.zeros(2, 5, 64), 8, torch.ones(32), torch.ones(32)),
    "norm b dtype": lambda b: b.group_norm(torch.zeros(2, 5, 64), 8, torch.ones(64),
                                           torch.ones(64, dtype=bf)),
    "norm activation": lambda b: b.group_norm(torch.zeros(2, 5, 64), 8, activation="relu"),
    "norm out": lambda b: b.group_norm(torch.zeros(2, 5, 64), 8, out=torch.zeros(2, 5, 32)),
    "grad dy": lambda b: b.group_norm_backward(torch.zeros(2, 4, 64), torch.zeros(2, 5, 64),
                                               torch.zeros(2, 8), torch.zeros(2, 8)),
    "grad mean": lambda b: b.group_norm_backward(torch.zeros(2, 5, 64), torch.zeros(2, 5, 64),
                                                 torch.zeros(3, 8), torch.zeros(2, 8)),
    "grad groups": lambda b: b.group_norm_backward(torch.zeros(2, 5, 64), torch.zeros(2, 5, 64),
                                                   torch.zeros(2, 7), torch.zeros(2, 7)),
    "grad rstd dtype": lambda b: b.group_norm_backward(
        torch.zeros(2, 5, 64), torch.zeros(2, 5, 64), torch.zeros(2, 8),
        torch.zeros(2, 8, dtype=bf)),
}


@pytest.mark.parametrize("case", sorted(BAD))
def test_mismatched_operands_are_refused(nrt, case):
    with pytest.raises((ValueError, TypeError)) as err:
        BAD[case](nrt)
    assert "CUDA" not in str(err.value), str(err.value)


def test_well_formed_operands_reach_the_device_check(nrt):
    table, cu = torch.zeros(2, 2, dtype=I32), torch.zeros(3, dtype=I32)
    both = torch.zeros(3, 2, 4, 2, 64, dtype=torch.uint8)
    scales = torch.zeros(3, 2, 4, 2)
    calls = [
        lambda: nrt.kv_cache_write(kv(), kv(), slots(), *parts()),
        lambda: nrt.kv_cache_write(kv(), kv(), slots(), *parts("mxfp4")),
        lambda: nrt.kv_cache_write(kv(), kv(), slots(), both[:, 0], both[:, 1], scales[:, 0],
                                   scales[:, 1]),
        lambda: nrt.kv_cache_read(*parts(), table, cu, 7, dtype=torch.float32),
        lambda: nrt.kv_cache_read(*parts(), table, cu, k_out=kv()),
        lambda: nrt.qk_norm_rope_cache(kv(heads=4), kv(), kv(), torch.ones(64), torch.ones(64),
                                       slots().int(), slots(), *parts()),
        lambda: nrt.group_norm(torch.zeros(2, 3, 5, 64, dtype=bf), 8, torch.ones(64), torch.ones(64)),
        lambda: nrt.group_norm_backward(torch.zeros(2, 5, 64), torch.zeros(2, 5, 64),
                                        torch.zeros(2, 8), torch.zeros(2, 8), activation="silu"),
    ]
    for call in calls:
        for _ in range(2):  # a refused layout is not remembered as a good one
            with pytest.raises(ValueError, match="CUDA"):
                call()


# ---------------------------------------------------------------------------
# the reference
# ---------------------------------------------------------------------------
def test_reference_grids():
    assert ref.E4M3[-1] == 448 and ref.E4M3[1] == 2.0 ** -9 and len(ref.E4M3) == 127
    t = torch.from_numpy(np.arange(127, dtype=np.uint8)).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.E4M3)
    mid = (ref.E2M1[1:] + ref.E2M1[:-1]) / 2
    assert np.array_equal(ref.nearest(mid, ref.E2M1), [0, 2, 2, 4, 4, 6, 6])  # ties to even


def test_reference_agrees_with_torchs_e4m3():
    x = torch.randn(4000, generator=torch.Generator().manual_seed(1)) * 200
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = ref.nearest(x.abs().numpy(), ref.E4M3) | np.where(np.signbit(x.numpy()), 0x80, 0)
    assert np.array_equal(got.astype(np.uint8), want)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_reference_holds_within_half_a_step(fmt):
    """|held - x| is at most half a step of the element's grid: 2^-4 relative (fp8,
    normal) or 2^-10 of the scale below it, with three f32 roundings on the way;
    e2m1 steps are at most 2 wide, and 1/2 below 2."""
    x = np.random.default_rng(3).standard_normal((50, 96)).astype(np.float32)
    x[3] = 0
    x[4] *= np.float32(1e-36)
    codes, scales = ref.quant(x, fmt)
    got = ref.held(codes, scales)
    err = np.abs(got - x)
    u = 2.0 ** -24
    if fmt == "fp8":
        s = scales[:, None].astype(np.float64)
        assert np.all(err <= (2.0 ** -4 + 4 * u) * np.abs(x) + 2.0 ** -10 * s * (1 + 4 * u))
        assert np.all(got[3] == 0)
    else:
        f = np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, -1)
        step = np.where(np.abs(x) <= 2 * f, 0.25, np.where(np.abs(x) <= 4 * f, 0.5, 1.0)) * f
        assert np.all(err <= step)
        assert np.all(np.abs(x) <= 6 * f)
