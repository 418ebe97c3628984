"""Log probabilities of given tokens, entropy, alternatives and their gradient against 64 bits.

Tolerances count f32 roundings, u = 2^-24.  With t = (x - m) / T the exponent of a term: x - m is
rounded, multiplied by a rounded 1 / T times log2(e) (3 u |t| together), and its exponential is
within 2^-22; the terms are positive and summed in at most `steps` steps.  So ln l is within
2^-22 + (3 mean|t| + steps) u, the mean by the terms' weights; the rest adds a few u of the sizes
that are added."""
import pytest
import torch

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def reference(x, tokens, temperature):
    """(logprob, entropy, lse, z) and the mean of |z - max| by weight, in 64 bits."""
    z = x.double() / temperature
    m = z.amax(1, keepdim=True)
    none = m[:, 0] == -float("inf")
    # z - m first: next to the lowest bf16 or f32 value, 64 bits step by 2^75, and lse is m
    d = torch.where(none[:, None], -float("inf"), z - m)
    ln_l = torch.where(none, 0.0, d.exp().sum(1).log())
    lse, logp = m[:, 0] + ln_l, d - ln_l[:, None]
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(1)
    inside = (tokens >= 0) & (tokens < x.shape[1])
    lp = torch.where(inside, logp.gather(1, tokens.clamp(0, x.shape[1] - 1)[:, None])[:, 0], 0.0)
    by_weight = torch.where(p > 0, p * -d, 0.0).sum(1)
    return lp, entropy, lse, logp, z, by_weight


def close(got, want, tol, what):
    got = got.double()
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    off = torch.where(same, 0.0, (got - want).abs())
    assert (off <= tol).all(), "%s: off by %g, allowed %g" % (what, (off - tol).max() + 0, tol.max())


def check(r, x, tokens, top, temperature):
    lp, entropy, lse, logp, z, d = reference(x, tokens, temperature)
    steps = x.shape[1] / 512 + 64
    base = 2.0 ** -22 + (3 * d + steps) * U
    big = z.amax(1).abs()
    big = torch.where(torch.isfinite(big), big, 0.0)
    ln_l = torch.where(torch.isfinite(lse), (lse - z.amax(1)).abs(), 0.0)
    reach = torch.where(torch.isfinite(lp), lp.abs(), 0.0)
    close(r.lse, lse, base + 4 * U * (big + ln_l), "lse")
    # z_token - m and ln l cancel at most to the logprob
    close(r.logprob, lp, base + 4 * U * (reach + 2 * ln_l), "logprob")
    close(r.entropy, entropy, 2 * base + (2.0 ** -21 + 2 * steps * U) * d + 8 * U * ln_l, "entropy")
    if top:
        order = x.float().sort(dim=1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(r.top_ids, order)
        want = logp.gather(1, order)
        reach = torch.where(torch.isfinite(want), want.abs(), 0.0)
        close(r.top_logprob, want, (base + 8 * U * ln_l)[:, None] + 4 * U * reach, "top_logprob")
    else:
        assert r.top_ids is None and r.top_logprob is None


def logits(seed, rows, vocab, dtype, width=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g, device="cuda") * width
    tokens = torch.randint(-2, vocab + 2, (rows,), generator=g, device="cuda")
    return x.to(dtype), tokens


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 33, 256, 1000, 1023, 8192, 8200, 32003, 131072, 151551])
def test_vocabularies(nr, vocab, dtype):
    for rows, top in ((1, min(vocab, 20)), (3, 0), (37, min(vocab, 5))):
        x, tokens = logits(vocab + rows, rows, vocab, dtype)
        check(nr.token_logprobs(x, tokens, top=top), x, tokens, top, 1.0)


@pytest.mark.parametrize("rows", [1, 2, 19, 20, 75, 76, 151, 153, 400])
def test_rows(nr, rows):
    x, tokens = logits(rows, rows, 20011, bf)
    check(nr.token_logprobs(x, tokens, top=32), x, tokens, 32, 1.0)


@pytest.mark.parametrize("temperature", [0.01, 0.6, 1.0, 7.0])
@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
def test_temperatures(nr, temperature, dtype):
    x, tokens = logits(5, 6, 5000, dtype)
    check(nr.token_logprobs(x, tokens, top=3, temperature=temperature), x, tokens, 3, temperature)


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
def test_ties_take_the_lowest_index(nr, dtype):
    """All equal, few different values, zeros of both signs, and rising and falling rows (every
    element a candidate)."""
    rows = torch.stack([torch.full((40000,), 2.5), torch.arange(40000) % 3 - 1.0,
                        torch.where(torch.arange(40000) % 2 == 0, 0.0, -0.0),
                        torch.linspace(-9, 9, 40000), torch.linspace(9, -9, 40000),
                        torch.where(torch.arange(40000) == 39999, 1.0, 0.0)]).to(dtype).cuda()
    tokens = torch.arange(6, device="cuda")
    for top in (1, 7, 32):
        check(nr.token_logprobs(rows, tokens, top=top), rows, tokens, top, 1.0)
    many = rows.repeat(60, 1)
    tokens = tokens.repeat(60)
    check(nr.token_logprobs(many, tokens, top=32), many, tokens, 32, 1.0)


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
def test_masked_logits(nr, dtype):
    """-inf and the type's lowest value: some, all but one, all, and both in one row."""
    low = torch.finfo(dtype).min
    x, _ = logits(6, 8, 30001, dtype)
    x[0, 5:] = -float("inf")
    x[1] = -float("inf")
    x[1, 30000] = 3
    x[2] = -float("inf")
    x[3] = low
    x[4, ::2] = low
    x[5] = -float("inf")
    x[5, 100:200] = low
    x[6, :29990] = -float("inf")
    tokens = torch.tensor([2, 30000, 7, 9, 3, 150, 0, -1], device="cuda")
    for rows in (x, x.repeat(40, 1)):
        t = tokens.repeat(rows.shape[0] // 8)
        check(nr.token_logprobs(rows, t, top=10), rows, t, 10, 1.0)


def test_rows_without_probabilities(nr):
    """A NaN or +inf anywhere: NaN, and ids inside [-1, vocab); the other rows are right."""
    for vocab in (9, 30001):
        x, tokens = logits(7, 6, vocab, f32)
        tokens = tokens.clamp(0, vocab - 1)
        x[0, 0] = x[2, vocab - 1] = float("nan")
        x[4] = float("nan")
        x[5, 3] = float("inf")
        r = nr.token_logprobs(x, tokens, top=3)
        for i in (0, 2, 4, 5):
            assert torch.isnan(r.lse[i]) and torch.isnan(r.logprob[i]) and torch.isnan(r.entropy[i])
            assert torch.isnan(r.top_logprob[i]).all()
        assert ((r.top_ids >= -1) & (r.top_ids < vocab)).all()
        keep = [1, 3]
        check(type(r)(*[v[keep] for v in r]), x[keep], tokens[keep], 3, 1.0)


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("offset", [0, 1, 3, 5])
def test_strided_rows_at_any_address(nr, dtype, offset):
    buf, tokens = logits(8, 5, 5003 + 64, dtype)
    x = buf[:, offset:offset + 5003]
    tokens = tokens.clamp(max=5010)
    r = nr.token_logprobs(x, tokens, top=4)
    check(r, x, tokens, 4, 1.0)
    dlp, dent = torch.randn(5, device="cuda"), torch.randn(5, device="cuda")
    back = dict(lse=r.lse, entropy=r.entropy)
    grad = nr.token_logprobs_backward(dlp, dent, x, tokens, **back)
    assert grad.is_contiguous()
    check_grad(grad, dlp, dent, x, tokens, r, 1.0)
    # into a strided tensor, and in place
    out = torch.full_like(buf, 3.0)
    got = nr.token_logprobs_backward(dlp, dent, x, tokens, dlogits=out[:, 2:5005], **back)
    assert torch.equal(got, grad)
    assert (out[:, :2] == 3).all() and (out[:, 5005:] == 3).all()
    held = buf.clone()
    got = nr.token_logprobs_backward(dlp, dent, x, tokens, dlogits=x, **back)
    assert torch.equal(got, grad) and torch.equal(buf[:, :offset], held[:, :offset])
    assert torch.equal(buf[:, offset + 5003:], held[:, offset + 5003:])


def grad_reference(dlp, dent, x, tokens, lse, entropy, temperature):
    """The formula in 64 bits, and its tolerance: z - lse has a rounding of its own and that of
    1 / T, its exponential 2 u |.| and 2^-22; three products and a sum follow."""
    z = x.double() / temperature
    logp = z - lse.double()[:, None]
    p = logp.exp()
    none = lse == -float("inf")
    p[none] = 0
    logp = torch.where(torch.isfinite(logp), logp, 0.0)
    inside = (tokens >= 0) & (tokens < x.shape[1]) & ~none
    g = torch.zeros_like(lse) if dlp is None else torch.where(inside, dlp, 0.0)
    h = torch.zeros_like(lse) if dent is None else torch.where(none, 0.0, dent)
    g, h = g.double()[:, None], h.double()[:, None]
    ent = 0.0 if dent is None else entropy.double()[:, None]
    d = -p * (g + h * (logp + ent))
    at = torch.where(inside, tokens, 0)
    one = torch.zeros_like(d).scatter_(1, at[:, None], inside.double()[:, None])
    d = d + one * g
    size = p * (g.abs() + h.abs() * (logp.abs() + abs(ent)))
    lp_err = U * (torch.where(torch.isfinite(z), z.abs(), 0.0) + 2 * logp.abs())
    tol = size * (2 * lp_err + 4 * U * logp.abs() + 2.0 ** -22 + 8 * U) + p * h.abs() * lp_err + one * g.abs() * 4 * U
    return d / temperature, tol / temperature


def check_grad(got, dlp, dent, x, tokens, r, temperature):
    want, tol = grad_reference(dlp, dent, x, tokens, r.lse, r.entropy, temperature)
    half = torch.finfo(x.dtype).eps / 2
    tol = tol + half * want.abs() * 1.01 + torch.finfo(x.dtype).tiny
    off = (got.double() - want).abs()
    assert (off <= tol).all(), "off by %g" % (off - tol).max()


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 7), (2, 8), (5, 4097), (33, 8192), (70, 32003)])
@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_gradient(nr, rows, vocab, dtype, temperature):
    x, tokens = logits(rows, rows, vocab, dtype)
    r = nr.token_logprobs(x, tokens, temperature=temperature)
    dlp, dent = torch.randn(rows, device="cuda"), torch.randn(rows, device="cuda")
    for g, h in ((dlp, dent), (dlp, None), (None, dent), (None, None)):
        got = nr.token_logprobs_backward(g, h, x, tokens, r.lse, r.entropy if h is not None else None,
                                         temperature=temperature)
        check_grad(got, g, h, x, tokens, r, temperature)


def test_gradient_of_masked_and_padded_rows(nr):
    x, _ = logits(9, 5, 1001, f32)
    x[0, 10:900] = -float("inf")
    x[1] = -float("inf")
    x[2] = torch.finfo(f32).min
    tokens = torch.tensor([3, 3, 3, -1, 1001], device="cuda")
    r = nr.token_logprobs(x, tokens)
    dlp, dent = torch.randn(5, device="cuda"), torch.randn(5, device="cuda")
    got = nr.token_logprobs_backward(dlp, dent, x, tokens, r.lse, r.entropy)
    assert (got[0, 10:900] == 0).all() and (got[1] == 0).all()
    # lse of the third row is the lowest value itself: its log probabilities are gone in f32
    keep = [0, 1, 3, 4]
    r = type(r)(*[None if v is None else v[keep] for v in r])
    check_grad(got[keep], dlp[keep], dent[keep], x[keep], tokens[keep], r, 1.0)
    got = nr.token_logprobs_backward(dlp, None, x, tokens, nr.token_logprobs(x, tokens).lse)
    assert (got[3:] == 0).all()  # padding has no log probability


def test_gradient_against_differences(nr):
    """Of the 64-bit definition, h = 1e-4: its own error is below h^2 times the third
    derivative, here below 1e-8."""
    x, _ = logits(10, 3, 50, f32)
    tokens = torch.tensor([4, 0, 49], device="cuda")
    dlp, dent = torch.randn(3, device="cuda"), torch.randn(3, device="cuda")
    r = nr.token_logprobs(x, tokens, temperature=0.8)
    got = nr.token_logprobs_backward(dlp, dent, x, tokens, r.lse, r.entropy, temperature=0.8)

    def loss(v):
        lp, ent, _, _, _, _ = reference(v, tokens, 0.8)
        return dlp.double() * lp + dent.double() * ent

    for j in range(50):
        e = torch.zeros(50, dtype=torch.float64, device="cuda")
        e[j] = 1e-4
        d = (loss(x.double() + e) - loss(x.double() - e)) / 2e-4
        assert ((got[:, j].double() - d).abs() < 2e-6).all()


def test_same_bits_each_time_and_in_a_graph(nr):
    x, tokens = logits(11, 9, 70001, bf)
    want = nr.token_logprobs(x, tokens, top=20)
    for _ in range(3):
        for a, b in zip(nr.token_logprobs(x, tokens, top=20), want):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = nr.token_logprobs(x, tokens, top=20)
        d = nr.token_logprobs_backward(want.lse, None, x, tokens, r.lse)
    y, _ = logits(12, 9, 70001, bf)
    x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    check(r, x, tokens, 20, 1.0)
    check_grad(d, want.lse, None, x, tokens, r, 1.0)


def test_offsets_past_32_bits(nr):
    rows, vocab = 17000, 262144
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    x = torch.zeros(rows, vocab, dtype=bf, device="cuda")
    assert x.numel() > 1 << 32
    y, _ = logits(13, 2, vocab, bf)
    x[0], x[-1] = y[0], y[1]
    tokens = torch.full((rows,), 5, device="cuda")
    ends = [0, rows - 1]
    r = nr.token_logprobs(x, tokens, top=5)
    check(type(r)(*[v[ends] for v in r]), y, tokens[ends], 5, 1.0)
    dlp = torch.ones(rows, device="cuda")
    want = nr.token_logprobs_backward(dlp[ends], None, y, tokens[ends], r.lse[ends])
    got = nr.token_logprobs_backward(dlp, None, x, tokens, r.lse, dlogits=x)
    assert torch.equal(got[ends], want)


def test_no_rows(nr):
    r = nr.token_logprobs(torch.zeros(0, 50, device="cuda"),
                          torch.zeros(0, dtype=torch.int64, device="cuda"), top=3)
    assert r.logprob.shape == (0,) and r.top_ids.shape == (0, 3)
