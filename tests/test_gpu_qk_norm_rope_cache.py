"""The attention preamble that writes the cache, on the GPU.

q_out: the rule of qk_norm_rope (1 bf16 ulp or the cancellation allowance, K =
32).  V: bit for bit what the plain reference quantises.  K is quantised from
an f32 value whose distance from the oracle's exact y is at most e = 32 * 2^-24 *
mag (the same allowance), so
  scale  fp8: |448 scale - max |y|| <= max e, and one rounding of the quotient;
  held   within half a step of the element's grid of y, plus e: fp8 steps are 2^-3
         of the value (2^-9 scales below 2^-6 scales), so half a step is 2^-4 |y| or
         2^-10 scale; e2m1 steps are 1/2, 1, 2 scales wide up to 2, 4, 6 scales.
A group whose largest value lies within e of a border between two mxfp4 scales may
take either."""
import numpy as np
import pytest
import torch

import oracle
import synth
from tests import cache_ref as ref
from tests.gpu_util import dev, host_bits
from tests.parity import check_bf16, check_f32
from tests.test_gpu_kv_cache import bf, f32, flat, make_cache

pytestmark = pytest.mark.gpu
K_ROPE, U = 32, 2.0 ** -24


def check_k(codes, scales, y, mag, fmt):
    e = K_ROPE * U * mag
    got = ref.held(codes, scales)
    if fmt == "fp8":
        top = np.abs(y).max(-1)
        s = scales.astype(np.float64)
        assert np.all(np.abs(448 * s - top) <= e.max(-1) + U * 448 * s), "scale"
        half = np.maximum(2.0 ** -4 * (np.abs(y) + e), 2.0 ** -10 * s[..., None])
    else:
        g = np.abs(y).reshape(*y.shape[:-1], -1, 32).max(-1)
        ge = e.reshape(*y.shape[:-1], -1, 32).max(-1)
        s = 2.0 ** (scales.astype(np.float64) - 127)
        assert np.all(g - ge <= 6 * s) and np.all(g + ge > 3 * s), "scale"
        f = np.repeat(s, 32, -1)
        half = np.where(np.abs(y) - e <= 2 * f, 0.25, np.where(np.abs(y) - e <= 4 * f, 0.5, 1.0)) * f
        half = np.where(np.abs(y) + e > 2 * f, np.maximum(half, 0.5 * f), half)
        half = np.where(np.abs(y) + e > 4 * f, f, half)
    # one f32 rounding of the product with the reciprocal, and its own two
    assert np.all(np.abs(got - y) <= half + e + 4 * U * np.abs(y)), "held"


def run(nr, tokens, hq, hk, D, fmt="fp8", dtype=bf, wdtype=torch.float32, page=16, seed=0, pos=None,
        fused_rows=False, interleaved_blocks=False, inplace=False, pad=True, **kw):
    q, k, wq, wk, p = synth.qk_inputs(tokens, hq, hk, D, seed, dtype, wdtype, pos_start=3)
    v = synth.tensor(seed, 77, (tokens, hk, D), dtype)
    if pos is not None:
        p = pos
    blocks = -(-tokens // page) + 2
    parts = make_cache(fmt, blocks, page, hk, D, seed, interleaved_blocks)
    before = [flat(x) for x in parts]
    slots = torch.randperm(blocks * page, generator=torch.Generator().manual_seed(seed))[:tokens]
    if pad and tokens > 2:
        slots[2] = -1
    qd, kd, vd = dev(q), dev(k), dev(v)
    if fused_rows:
        row = torch.cat([qd, kd, vd], 1)
        qd, kd, vd = row[:, :hq], row[:, hq:hq + hk], row[:, hq + hk:]
    q_out = nr.qk_norm_rope_cache(qd, kd, vd, dev(wq), dev(wk), dev(p), dev(slots), *parts,
                                  q_out=qd if inplace else None, **kw)
    torch.cuda.synchronize()
    r = oracle.qk_norm_rope_ex(host_bits(q), host_bits(k), host_bits(wq), host_bits(wk), p.numpy(),
                               want_y=True, **kw)
    got = host_bits(q_out.contiguous())
    if dtype == bf:
        check_bf16(got, r[0], r[2], r[4], k_cancel=K_ROPE, what="q")
    else:
        check_f32(got, r[2], rel=1e-5, mag=r[4], k_cancel=K_ROPE, what="q")
    keep = [i for i in range(tokens) if slots[i] >= 0]
    at = slots[keep].numpy()
    y = np.asarray(r[3]).reshape(tokens, hk, D)[keep]
    mag = np.asarray(r[5]).reshape(tokens, hk, D)[keep]
    check_k(flat(parts[0])[at], flat(parts[2])[at], y, mag, fmt)
    want = ref.quant(f32(v)[keep], fmt)
    for part, old, w in ((parts[1], before[1], want[0]), (parts[3], before[3], want[1])):
        old = old.copy()
        old[at] = w
        assert np.array_equal(flat(part).view(np.uint8), old.view(np.uint8)), "V"
    other = np.setdiff1d(np.arange(blocks * page), at)
    for part, old in ((parts[0], before[0]), (parts[2], before[2])):
        assert np.array_equal(flat(part)[other].view(np.uint8), old[other].view(np.uint8))


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("tokens,hq,hk,D", [(1, 1, 1, 64), (1, 32, 8, 128), (5, 3, 1, 256),
                                            (33, 8, 2, 128), (70, 5, 5, 512), (300, 24, 24, 128),
                                            (7, 64, 8, 64)])
def test_bf16(nr, fmt, tokens, hq, hk, D):
    run(nr, tokens, hq, hk, D, fmt, seed=tokens + D)


@pytest.mark.parametrize("fmt,D", [("fp8", 32), ("fp8", 64), ("fp8", 128), ("fp8", 256),
                                   ("mxfp4", 64), ("mxfp4", 128), ("mxfp4", 256)])
def test_f32(nr, fmt, D):
    run(nr, 21, 6, 2, D, fmt, dtype=torch.float32, seed=D)


@pytest.mark.parametrize("tokens", [2431, 9800])
def test_many_tokens(nr, tokens):
    """Items of part of a token, and whole tokens over several rounds of the warps."""
    run(nr, tokens, 5, 2, 64, "fp8", page=64, seed=4)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_views_of_a_fused_row_in_place(nr, fmt):
    run(nr, 40, 4, 2, 128, fmt, fused_rows=True, interleaved_blocks=True, inplace=True, page=8)


@pytest.mark.parametrize("kw", [dict(gemma=True), dict(eps=0.0), dict(theta=5e5),
                                dict(rotary_dim=64), dict(rotary_dim=64, interleaved=True),
                                dict(interleaved=True),
                                dict(theta=5e5, llama3=(8.0, 1.0, 4.0, 8192.0))])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_variants(nr, fmt, kw):
    run(nr, 31, 4, 2, 128, fmt, seed=9, **kw)


@pytest.mark.parametrize("rot", [16, 32, 96])
def test_partial_rotary_fp8(nr, rot):
    run(nr, 19, 3, 2, 128, "fp8", seed=rot, rotary_dim=rot)


@pytest.mark.parametrize("kw", [dict(rotary_dim=64), dict(rotary_dim=64, interleaved=True),
                                dict(rotary_dim=8, interleaved=True), dict(rotary_dim=24)])
def test_f32_variants(nr, kw):
    run(nr, 17, 3, 2, 128, "fp8", dtype=torch.float32, wdtype=bf, seed=6, **kw)


def test_mrope_4bit_f32_sections_from_an_iterator(nr):
    pos = torch.from_numpy(np.random.default_rng(7).integers(0, 8192, (3, 9)).astype(np.int32))
    run(nr, 9, 6, 2, 128, "mxfp4", dtype=torch.float32, pos=pos, seed=8,
        mrope_sections=(16, 24, 24), theta=1e6)
    q, k, wq, wk, _ = (dev(t) for t in synth.qk_inputs(9, 4, 2, 128, 3, bf, torch.float32))
    v, slots = torch.randn(9, 2, 128, device="cuda").to(bf), torch.arange(9, device="cuda")
    a, b = make_cache("fp8", 2, 8, 2, 128), make_cache("fp8", 2, 8, 2, 128)
    qa = nr.qk_norm_rope_cache(q, k, v, wq, wk, dev(pos), slots, *a, mrope_sections=(16, 24, 24))
    qb = nr.qk_norm_rope_cache(q, k, v, wq, wk, dev(pos), slots, *b,
                               mrope_sections=iter((16, 24, 24)))
    assert torch.equal(qa, qb) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_alternating_configurations(nr):
    """Calls that take turns with different rotary constants, as two models in one
    process would."""
    q, k, wq, wk, p = (dev(t) for t in synth.qk_inputs(20, 4, 2, 128, 3, bf, torch.float32,
                                                       pos_start=900))
    v, slots = torch.randn(20, 2, 128, device="cuda").to(bf), torch.arange(20, device="cuda")
    kws = [dict(), dict(theta=5e5), dict(rotary_dim=64), dict(theta=5e5,
                                                              llama3=(8.0, 1.0, 4.0, 8192.0))]
    first = []
    for _ in range(2):
        for i, kw in enumerate(kws):
            out = nr.qk_norm_rope_cache(q, k, v, wq, wk, p, slots,
                                        *make_cache("fp8", 3, 8, 2, 128), **kw)
            plain = nr.qk_norm_rope_ex(q, k, wq, wk, p, **kw)[0]
            # the two kernels' f32 roundings differ by far less than a bf16 step
            assert (out.float() - plain.float()).abs().max() <= 2.0 ** -7 * plain.float().abs().max()
            if len(first) < len(kws):
                first.append(out)
            assert torch.equal(out, first[i])


def test_host_threads_on_streams_of_their_own(nr):
    """Four host threads, each with its stream, cache and rotary configuration."""
    import threading

    kws = [dict(), dict(theta=5e5), dict(rotary_dim=64), dict(interleaved=True)]
    q, k, wq, wk, p = (dev(t) for t in synth.qk_inputs(40, 4, 2, 128, 3, bf, torch.float32))
    v, slots = torch.randn(40, 2, 128, device="cuda").to(bf), torch.arange(40, device="cuda")
    x = torch.randn(1, 30000, 64, device="cuda").to(bf)
    caches = [make_cache("fp8", 5, 8, 2, 128) for _ in kws]

    def call(kw, parts):
        out = nr.qk_norm_rope_cache(q, k, v, wq, wk, p, slots, *parts, **kw)
        y, mean, rstd = nr.group_norm(x, 8, activation="silu", stats=True)
        dx = nr.group_norm_backward(x, x, mean, rstd, activation="silu")[0]
        return out, y, dx, parts[0].clone(), parts[2].clone()

    want = [call(kw, parts) for kw, parts in zip(kws, caches)]
    torch.cuda.synchronize()
    got, errors = [None] * len(kws), []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    got[i] = call(kws[i], caches[i])
            s.synchronize()
        except Exception as e:  # reported below, in the test's thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(kws))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))


def test_bf16_weights_and_far_positions(nr):
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 131072, 7, 99999999], dtype=torch.int32)
    run(nr, 8, 4, 2, 128, wdtype=bf, pos=pos, seed=2)


@pytest.mark.parametrize("interleaved", [False, True])
def test_mrope(nr, interleaved):
    rng = np.random.default_rng(7)
    pos = torch.from_numpy(rng.integers(0, 8192, (3, 33)).astype(np.int32))
    run(nr, 33, 6, 2, 128, pos=pos, seed=8, mrope_sections=(16, 24, 24),
        mrope_interleaved=interleaved, theta=1e6)


def test_no_tokens(nr):
    parts = make_cache("fp8", 2, 4, 2, 64)
    before = [flat(p) for p in parts]
    q = torch.empty(0, 4, 64, dtype=bf, device="cuda")
    kv = torch.empty(0, 2, 64, dtype=bf, device="cuda")
    w = torch.ones(64, device="cuda")
    out = nr.qk_norm_rope_cache(q, kv, kv, w, w, torch.empty(0, dtype=torch.int32, device="cuda"),
                                torch.empty(0, dtype=torch.int64, device="cuda"), *parts)
    assert out.shape == (0, 4, 64)
    assert all(np.array_equal(flat(p), b) for p, b in zip(parts, before))


def test_padding_may_hold_anything(nr):
    """NaN in a padded token's k and v reaches nothing; its q is still written."""
    T = 6
    q, k, wq, wk, p = (dev(t) for t in synth.qk_inputs(T, 4, 2, 128, 3, bf, torch.float32))
    v = torch.randn(T, 2, 128, device="cuda").to(bf)
    slots = torch.tensor([3, -1, 5, 1 << 40, 0, -9], device="cuda")
    a, b = make_cache("fp8", 2, 4, 2, 128), make_cache("fp8", 2, 4, 2, 128)
    qa = nr.qk_norm_rope_cache(q, k, v, wq, wk, p, slots, *a)
    k[[1, 3, 5]] = float("nan")
    v[[1, 3, 5]] = float("nan")
    qb = nr.qk_norm_rope_cache(q, k, v, wq, wk, p, slots, *b)
    assert torch.equal(qa, qb)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_and_replayed(nr):
    T = 50
    q, k, wq, wk, p = (dev(t) for t in synth.qk_inputs(T, 8, 2, 128, 3, bf, torch.float32))
    v = torch.randn(T, 2, 128, device="cuda").to(bf)
    slots = torch.arange(T, device="cuda")
    parts = make_cache("mxfp4", 4, 16, 2, 128)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = nr.qk_norm_rope_cache(q, k, v, wq, wk, p, slots, *parts)
    for i in range(2):
        k.copy_(torch.randn(T, 2, 128))
        p.add_(T)
        slots.copy_(torch.arange(T) if i == 0 else torch.arange(T).flip(0))
        graph.replay()
        other = make_cache("mxfp4", 4, 16, 2, 128)
        want = nr.qk_norm_rope_cache(q, k, v, wq, wk, p, slots, *other)
        assert torch.equal(out, want)
        assert all(torch.equal(x.view(64, -1)[:T], y.view(64, -1)[:T])
                   for x, y in zip(parts, other))


def test_a_clip_in_two_chunks_through_norm_preamble_cache_and_attention(nr):
    """As a causal video model runs them: group norm + SiLU of a frame's
    features, the preamble of its tokens into the cache, the cache of all frames
    so far read back, attention over it.  Against the same in 64 bits without a
    cache: K and V are held within half an e4m3 step (2^-4 of each value, and
    2^-10 of the row's 448th below it), so a score moves by at most d_s =
    sum_j |q_j| dk_j / sqrt(D) and the output by at most
    (e^(2 max d_s) - 1) max |v| + max dv, with bf16 roundings (2^-8) of the reads,
    of q and of the inputs' products on top."""
    g = torch.Generator().manual_seed(11)
    space, chan, heads, D, frames = 48, 128, 2, 64, 2
    w_norm, b_norm = torch.ones(chan, device="cuda"), torch.zeros(chan, device="cuda")
    proj = (torch.randn(chan, 3 * heads * D, generator=g) / chan ** 0.5).to(bf).cuda()
    wq = wk = torch.ones(D, device="cuda")
    parts = make_cache("fp8", 8, 16, heads, D)
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    keys, values = [], []
    for f in range(frames):
        x = torch.randn(1, 6, 8, chan, generator=g).to(bf).cuda()
        h = nr.group_norm(x, 8, w_norm, b_norm, activation="silu")
        qkv = (h.view(space, chan) @ proj).view(space, 3 * heads, D)
        q, k, v = qkv[:, :heads], qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
        at = torch.arange(f * space, (f + 1) * space, device="cuda")
        qr = nr.qk_norm_rope_cache(q, k, v, wq, wk, at.to(torch.int32), at, *parts)
        n = (f + 1) * space
        kc, vc = nr.kv_cache_read(*parts, table,
                                  torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
        # the same in 64 bits, from the bf16 projections and without a cache
        plain = nr.qk_norm_rope(q.float().contiguous(), k.float().contiguous(), wq, wk,
                                at.to(torch.int32))
        q64 = plain[0].double()
        keys.append(plain[1].double())
        values.append(v.double())
        k64, v64 = torch.cat(keys), torch.cat(values)

        def attend(q, k, v):
            p = torch.softmax(torch.einsum("qhd,khd->hqk", q, k) / D ** 0.5, -1)
            return torch.einsum("hqk,khd->qhd", p, v)

        def off(t):  # how far a held and read-back value may be
            top = t.abs().amax(-1, keepdim=True)
            return torch.maximum(2.0 ** -4 * t.abs(), 2.0 ** -10 * top / 448) + 2.0 ** -8 * t.abs() * 1.07

        assert torch.all((kc.double() - k64).abs() <= off(k64) + 1e-4)
        assert torch.all((vc.double() - v64).abs() <= off(v64) + 1e-6)
        ds = torch.einsum("qhd,khd->hqk", q64.abs(), off(k64) + 1e-4) / D ** 0.5
        ds = ds + torch.einsum("qhd,khd->hqk", 2.0 ** -8 * q64.abs() + 1e-4,
                               k64.abs() + off(k64)) / D ** 0.5
        bound = (torch.exp(2 * ds.max()) - 1) * v64.abs().max() + off(v64).max() + 1e-6
        err = (attend(qr.double(), kc.double(), vc.double()) - attend(q64, k64, v64)).abs().max()
        assert err <= bound, (err, bound)
