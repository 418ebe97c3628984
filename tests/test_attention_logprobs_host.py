"""The attention, 8-bit norm and log-probability entry points on the CPU: every refusal of the C
ABI and of the binding comes before a launch; options count with their value at each call; the
reference of attention agrees with a direct computation."""
import ctypes

import numpy as np
import pytest
import torch

from tests import attention_ref as aref
from tests import cache_ref
from tests.test_abi_host import (A, ALIAS, ALIGN, BF16, DTYPE, F32, MB, NULL, OK, SHAPE, UNSUP,
                                 VALUE)
from tests.test_kv_cache_host import CACHE_ERRORS, cache, cast

bf, I32 = torch.bfloat16, torch.int32
# device-like addresses, 16 MB apart, behind the cache's four
(OUT, LSE, Q, TABLE, LENS, CU, TREE, WS, X, W, RES, CODES, SCALES, LOGITS, TOKENS, F0, F1, F2, F3,
 DL) = (A + (64 + 16 * i) * MB for i in range(20))


@pytest.fixture(scope="module")
def nrt(lib_path):
    import normalisation_rope_transformers_gb300 as nrt
    return nrt


def attend(nrt, c, out=OUT, lse=LSE, q=Q, table=TABLE, width=4, lens=LENS, cu=CU, seqs=2, tokens=3,
           hq=4, qs=None, tree=None, words=0, scale=0.1, dtype=BF16, ws=WS, wsb=1 << 30):
    qs = hq * c.head_dim if qs is None else qs
    return nrt.lib.nr_cache_attention(out, lse, q, cast(c, nrt), table, width, lens, cu, seqs,
                                      tokens, hq, qs, tree, words, scale, dtype, ws, wsb, None)


@pytest.mark.parametrize("kw,want", CACHE_ERRORS[:17])
def test_bad_caches_are_refused(nrt, kw, want):
    assert attend(nrt, cache(**kw), qs=1 << 20) == want, nrt.lib.nr_last_error_message()


@pytest.mark.parametrize("kw,want", [
    (dict(seqs=-1), SHAPE), (dict(tokens=-1), SHAPE), (dict(width=-1), SHAPE), (dict(words=-1), SHAPE),
    (dict(hq=0), SHAPE), (dict(hq=3), SHAPE), (dict(hq=1 << 20), SHAPE), (dict(dtype=7), DTYPE),
    (dict(tokens=1 << 30), SHAPE), (dict(seqs=1 << 31), SHAPE), (dict(width=1 << 31), SHAPE),
    (dict(qs=255), SHAPE), (dict(qs=260), ALIGN), (dict(qs=1 << 62), SHAPE), (dict(cu=None), SHAPE),
    (dict(tree=TREE), NULL), (dict(words=1), NULL), (dict(scale=float("inf")), VALUE),
    (dict(scale=float("nan")), VALUE), (dict(out=None), NULL), (dict(q=None), NULL),
    (dict(lens=None), NULL), (dict(table=None), NULL), (dict(ws=None), NULL), (dict(wsb=1000), SHAPE),
    (dict(out=OUT + 8), ALIGN), (dict(q=Q + 8), ALIGN), (dict(lse=LSE + 2), ALIGN),
    (dict(cu=CU + 2), ALIGN), (dict(tree=TREE + 1, words=1), ALIGN), (dict(ws=WS + 8), ALIGN),
    (dict(out=Q), ALIAS), (dict(lse=OUT + 64), ALIAS), (dict(out=A), ALIAS), (dict(ws=A), ALIAS),
    (dict(lse=LENS), ALIAS), (dict(out=TREE, tree=TREE + 16, words=1), ALIAS), (dict(ws=OUT), ALIAS),
    (dict(tokens=0, out=None), OK), (dict(seqs=0, tokens=0, cu=None, q=None), OK),
])
def test_bad_attention_is_refused(nrt, kw, want):
    assert attend(nrt, cache(), **kw) == want, nrt.lib.nr_last_error_message()


@pytest.mark.parametrize("dim", [16, 32, 96, 192, 512])
def test_other_head_sizes_are_refused(nrt, dim):
    assert attend(nrt, cache(dim=dim)) == UNSUP
    n = ctypes.c_int64(-1)
    assert nrt.lib.nr_cache_attention_workspace(dim, ctypes.byref(n)) == UNSUP


def test_attention_workspace_query(nrt):
    n = ctypes.c_int64(-1)
    for dim in (64, 128, 256):
        assert nrt.lib.nr_cache_attention_workspace(dim, ctypes.byref(n)) == OK and n.value > 0
        c = cache(dim=dim)
        assert attend(nrt, c, wsb=n.value - 1) == SHAPE
    assert nrt.lib.nr_cache_attention_workspace(64, None) == NULL


def quant(nrt, codes=CODES, scales=SCALES, x=X, w=W, res=RES, rows=3, hidden=256, dtype=BF16, eps=1e-6,
          gemma=0, layout=0):
    return nrt.lib.nr_rmsnorm_quant(codes, scales, x, w, res, rows, hidden, dtype, eps, gemma, layout,
                                    None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=4), DTYPE), (dict(layout=3), VALUE), (dict(rows=-1), SHAPE), (dict(hidden=0), SHAPE),
    (dict(eps=-1.0), VALUE), (dict(eps=float("nan")), VALUE), (dict(gemma=2), VALUE),
    (dict(hidden=252), UNSUP), (dict(hidden=264, layout=1), UNSUP), (dict(hidden=272, layout=2), UNSUP),
    (dict(hidden=32776), UNSUP), (dict(hidden=16388, dtype=F32), UNSUP), (dict(rows=1 << 31), SHAPE),
    (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(x=None), NULL), (dict(w=None), NULL),
    (dict(x=X + 8), ALIGN), (dict(codes=CODES + 8), ALIGN), (dict(scales=SCALES + 2), ALIGN),
    (dict(res=RES + 4), ALIGN), (dict(codes=X), ALIAS), (dict(scales=CODES + 16), ALIAS),
    (dict(scales=RES), ALIAS), (dict(res=X), ALIAS), (dict(res=W), ALIAS), (dict(rows=0, x=None), OK),
])
def test_bad_norms_are_refused(nrt, kw, want):
    assert quant(nrt, **kw) == want, nrt.lib.nr_last_error_message()


def score(nrt, lp=F0, ent=F1, lse=F2, tlp=F3, tids=DL, logits=LOGITS, tokens=TOKENS, rows=3, vocab=100,
          stride=100, top=4, inv_t=1.0, dtype=BF16):
    return nrt.lib.nr_token_logprobs(lp, ent, lse, tlp, tids, logits, tokens, rows, vocab, stride, top,
                                     inv_t, dtype, None)


LOGIT_ERRORS = [
    (dict(dtype=4), DTYPE), (dict(rows=-1), SHAPE), (dict(vocab=0), SHAPE), (dict(stride=99), SHAPE),
    (dict(vocab=1 << 31, stride=1 << 31), SHAPE), (dict(rows=1 << 30), SHAPE),
    (dict(stride=1 << 61), SHAPE), (dict(inv_t=0.0), VALUE), (dict(inv_t=-1.0), VALUE),
    (dict(inv_t=float("inf")), VALUE), (dict(inv_t=float("nan")), VALUE), (dict(logits=None), NULL),
    (dict(tokens=None), NULL), (dict(lse=None), NULL), (dict(logits=LOGITS + 1), ALIGN),
    (dict(tokens=TOKENS + 4), ALIGN), (dict(lse=F2 + 2), ALIGN), (dict(rows=0, logits=None), OK),
]


@pytest.mark.parametrize("kw,want", LOGIT_ERRORS + [
    (dict(top=-1), SHAPE), (dict(top=33), SHAPE), (dict(top=9, vocab=8), SHAPE), (dict(lp=None), NULL),
    (dict(ent=None), NULL), (dict(tlp=None), NULL), (dict(tids=None), NULL), (dict(tids=DL + 4), ALIGN),
    (dict(lp=LOGITS), ALIAS), (dict(ent=F0), ALIAS), (dict(tids=TOKENS), ALIAS), (dict(tlp=DL + 8), ALIAS),
])
def test_bad_scores_are_refused(nrt, kw, want):
    assert score(nrt, **kw) == want, nrt.lib.nr_last_error_message()


def grad(nrt, dl=DL, dlp=F0, dent=F1, logits=LOGITS, tokens=TOKENS, lse=F2, ent=F3, rows=3, vocab=100,
         stride=100, ds=100, inv_t=1.0, dtype=BF16):
    return nrt.lib.nr_token_logprobs_backward(dl, dlp, dent, logits, tokens, lse, ent, rows, vocab,
                                              stride, ds, inv_t, dtype, None)


@pytest.mark.parametrize("kw,want", LOGIT_ERRORS + [
    (dict(ds=99), SHAPE), (dict(dl=None), NULL), (dict(ent=None), NULL), (dict(dl=DL + 1), ALIGN),
    (dict(dl=LOGITS + 2), ALIAS), (dict(dl=LOGITS, ds=104), ALIAS), (dict(dl=F0), ALIAS),
    (dict(dl=TOKENS), ALIAS), (dict(dent=F1 + 1), ALIGN),
])
def test_bad_gradients_are_refused(nrt, kw, want):
    assert grad(nrt, **kw) == want, nrt.lib.nr_last_error_message()


# ---------------------------------------------------------------------------
# the binding's own checks (host tensors: a call that passes them stops at the device check)
# ---------------------------------------------------------------------------
def parts(blocks=3, page=4, heads=2, dim=64):
    c = [torch.zeros(blocks, page, heads, dim, dtype=torch.uint8) for _ in range(2)]
    return c + [torch.zeros(blocks, page, heads) for _ in range(2)]


def i32(*shape):
    return torch.zeros(*shape, dtype=I32)


def q(tokens=3, heads=4, dim=64, dtype=bf):
    return torch.zeros(tokens, heads, dim, dtype=dtype)


REFUSED = {
    "q of another head size": lambda b: b.cache_attention(q(dim=128), *parts(), i32(3, 2), i32(3)),
    "q heads": lambda b: b.cache_attention(q(heads=3), *parts(), i32(3, 2), i32(3)),
    "q dtype": lambda b: b.cache_attention(q(dtype=torch.float16), *parts(), i32(3, 2), i32(3)),
    "q layout": lambda b: b.cache_attention(q(3, 64, 4).transpose(1, 2), *parts(), i32(3, 2), i32(3)),
    "tokens without cu_q": lambda b: b.cache_attention(q(), *parts(), i32(2, 2), i32(2)),
    "table axes": lambda b: b.cache_attention(q(), *parts(), i32(3), i32(3)),
    "table dtype": lambda b: b.cache_attention(q(), *parts(), i32(3, 2).long(), i32(3)),
    "lens": lambda b: b.cache_attention(q(), *parts(), i32(3, 2), i32(4)),
    "cu_q": lambda b: b.cache_attention(q(), *parts(), i32(2, 2), i32(2), cu_q=i32(2)),
    "tree rows": lambda b: b.cache_attention(q(), *parts(), i32(2, 2), i32(2), cu_q=i32(3), tree=i32(2, 1)),
    "tree words": lambda b: b.cache_attention(q(), *parts(), i32(2, 2), i32(2), cu_q=i32(3), tree=i32(3, 0)),
    "tree dtype": lambda b: b.cache_attention(q(), *parts(), i32(2, 2), i32(2), cu_q=i32(3),
                                              tree=i32(3, 1).long()),
    "out": lambda b: b.cache_attention(q(), *parts(), i32(3, 2), i32(3), out=q().float()),
    "norm w": lambda b: b.rmsnorm_quant(torch.zeros(2, 64, dtype=bf), torch.zeros(64)),
    "norm group": lambda b: b.rmsnorm_quant(torch.zeros(2, 64, dtype=bf), torch.zeros(64, dtype=bf),
                                            scales="group"),
    "norm layout": lambda b: b.rmsnorm_quant(torch.zeros(2, 64, dtype=bf), torch.zeros(64, dtype=bf),
                                             scales="column"),
    "norm scales_out": lambda b: b.rmsnorm_quant(torch.zeros(2, 64, dtype=bf), torch.zeros(64, dtype=bf),
                                                 scales_out=torch.zeros(2, 1)),
    "norm codes": lambda b: b.rmsnorm_quant(torch.zeros(2, 64, dtype=bf), torch.zeros(64, dtype=bf),
                                            codes=torch.zeros(2, 64)),
    "tokens dtype": lambda b: b.token_logprobs(torch.zeros(2, 9), i32(2)),
    "tokens rows": lambda b: b.token_logprobs(torch.zeros(2, 9), torch.zeros(3, dtype=torch.int64)),
    "top": lambda b: b.token_logprobs(torch.zeros(2, 9), torch.zeros(2, dtype=torch.int64), top=10),
    "logits layout": lambda b: b.token_logprobs(torch.zeros(9, 2).T, torch.zeros(2, dtype=torch.int64)),
    "logits rows": lambda b: b.token_logprobs(torch.zeros(9).expand(2, 9),
                                              torch.zeros(2, dtype=torch.int64)),
    "temperature": lambda b: b.token_logprobs(torch.zeros(2, 9), torch.zeros(2, dtype=torch.int64),
                                              temperature=0),
    "entropy": lambda b: b.token_logprobs_backward(None, torch.zeros(2), torch.zeros(2, 9),
                                                   torch.zeros(2, dtype=torch.int64), torch.zeros(2)),
    "dlogits": lambda b: b.token_logprobs_backward(None, None, torch.zeros(2, 9),
                                                   torch.zeros(2, dtype=torch.int64), torch.zeros(2),
                                                   dlogits=torch.zeros(2, 8)),
}


@pytest.mark.parametrize("name", sorted(REFUSED))
def test_mismatched_operands_are_refused(nrt, name):
    with pytest.raises((TypeError, ValueError)) as e:
        REFUSED[name](nrt)
    assert "CUDA" not in str(e.value), "refused for its device alone"


def test_host_tensors_are_refused(nrt):
    w = torch.zeros(64, dtype=bf)
    t = torch.zeros(2, dtype=torch.int64)
    for call in (lambda: nrt.cache_attention(q(), *parts(), i32(3, 2), i32(3)),
                 lambda: nrt.rmsnorm_quant(torch.zeros(2, 64, dtype=bf), w),
                 lambda: nrt.token_logprobs(torch.zeros(2, 9), t),
                 lambda: nrt.token_logprobs_backward(None, None, torch.zeros(2, 9), t, torch.zeros(2))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.fixture
def recorded(nrt, monkeypatch):
    """The binding with its device check off; the arguments of each launch."""
    calls = []
    monkeypatch.setattr(nrt, "_cuda", lambda *ts: None)
    monkeypatch.setattr(nrt, "_launch", lambda device, fn, *args: calls.append(args))
    monkeypatch.setattr(nrt, "_checked", {})
    return calls


def test_options_changed_in_place(nrt, recorded):
    scale, t, eps = torch.tensor(0.5), torch.tensor(2.0), torch.tensor(0.25)
    top = torch.tensor(3)
    ids = torch.zeros(2, dtype=torch.int64)
    for v in (0.5, 0.125, 0.5):
        scale.fill_(v)
        nrt.cache_attention(q(), *parts(), i32(3, 2), i32(3), scale=scale)
        assert recorded[-1][-4] == v
        t.fill_(v)
        nrt.token_logprobs(torch.zeros(2, 9), ids, top=top, temperature=t)
        assert recorded[-1][-2] == 1 / v
        eps.fill_(v)
        nrt.rmsnorm_quant(torch.zeros(2, 64, dtype=bf), torch.zeros(64, dtype=bf), eps=eps)
        assert v in recorded[-1]
    top.fill_(4)
    assert nrt.token_logprobs(torch.zeros(2, 9), ids, top=top).top_ids.shape == (2, 4)

    def kept(entry):
        for v in entry:
            yield from kept(v) if isinstance(v, tuple) else (v,)

    assert not any(isinstance(v, torch.Tensor) for key in nrt._checked for v in kept(key))


def test_the_default_scale(nrt, recorded):
    nrt.cache_attention(q(dim=64), *parts(), i32(3, 2), i32(3))
    assert recorded[-1][-4] == 0.125


def test_reference_against_a_direct_computation():
    rng = np.random.default_rng(0)
    p = aref.make_cache(rng, 4, 8, 2, 64, "fp8")
    table = np.array([[2, 0, 3]], np.int32)
    x = rng.standard_normal((3, 4, 64)).astype(np.float32)
    tree = np.array([[1], [3], [5]], np.int32)
    out, lse, tol, _ = aref.attention(x, p, table, [20], [0, 3], tree, 0.125, True)
    k, v = (torch.from_numpy(cache_ref.held(p[i], p[2 + i]).reshape(32, 2, 64)) for i in range(2))
    at = torch.tensor([16 + i for i in range(8)] + list(range(8)) + [24 + i for i in range(4)])
    mask = torch.zeros(3, 20)
    mask[:, 17:] = torch.tensor([[0.0, 1, 1], [0, 0, 1], [0, 1, 0]]) * -1e30
    for h in range(4):
        s = torch.from_numpy(x[:, h]).double() @ k[at, h // 2].T * 0.125 + mask.double()
        want = torch.softmax(s, 1) @ v[at, h // 2]
        assert np.allclose(out[:, h], want.numpy(), rtol=1e-12, atol=1e-14)
        assert np.allclose(lse[:, h], torch.logsumexp(s, 1).numpy(), rtol=1e-12)
    assert (tol > 0).all() and (tol < 1e-4).all()
