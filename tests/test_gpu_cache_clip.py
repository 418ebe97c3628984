"""Two chunks of a clip through norm, preamble, cache and attention, each piece held
to its own bound: the queries against the rotated ones in 64 bits, and attention over
the K and V that were read back against attention of the exact queries over the same K
and V, where nothing but the queries' bf16 rounding is left.

q: the f32 norm and rotation are off by at most 2^-18 of the pair's size (32 U as the
preamble's other tests allow, and the 64-bit reference by nothing), and bf16 rounds by
2^-8.  Attention: with scores off by at most d, the weights p change by factors in
[e^-2d, e^2d], so a query's output moves by at most (e^2d - 1) sum_k p_k |v_k - o|;
d = max_k sum_j |dq_j| |k_kj| / sqrt(D)."""
import pytest
import torch

from tests.test_gpu_kv_cache import make_cache

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


def rotate(x, positions, theta=1e4, eps=1e-6):
    """Norm (weights of one) and rotate-half rotation in 64 bits; and each element's
    size before the rotation's cancellation."""
    y = x.double()
    y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt()
    half = y.shape[-1] // 2
    freq = torch.tensor([theta ** (-i / half) for i in range(half)], dtype=torch.float64,
                        device=x.device)
    angle = positions.double()[:, None, None] * freq
    c, s = angle.cos(), angle.sin()
    a, b = y[..., :half], y[..., half:]
    size = (a.abs() * c.abs() + b.abs() * s.abs(), a.abs() * s.abs() + b.abs() * c.abs())
    return torch.cat([a * c - b * s, a * s + b * c], -1), torch.cat(size, -1)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_queries_and_attention_over_the_cache(nr, fmt):
    g = torch.Generator().manual_seed(12)
    space, chan, heads, D, frames = 48, 128, 2, 64, 3
    w_norm, b_norm = torch.ones(chan, device="cuda"), torch.zeros(chan, device="cuda")
    proj = (torch.randn(chan, 3 * heads * D, generator=g) / chan ** 0.5).to(bf).cuda()
    w = torch.ones(D, device="cuda")
    parts = make_cache(fmt, 12, 16, heads, D)
    table = torch.arange(12, dtype=torch.int32, device="cuda")[None]

    def attend(q, k, v):
        p = torch.softmax(torch.einsum("qhd,khd->hqk", q, k) / D ** 0.5, -1)
        return p, torch.einsum("hqk,khd->qhd", p, v)

    for f in range(frames):
        x = torch.randn(1, 6, 8, chan, generator=g).to(bf).cuda()
        h = nr.group_norm(x, 8, w_norm, b_norm, activation="silu")
        qkv = (h.view(space, chan) @ proj).view(space, 3 * heads, D)
        q, k, v = qkv[:, :heads], qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
        at = torch.arange(f * space, (f + 1) * space, device="cuda")
        qr = nr.qk_norm_rope_cache(q, k, v, w, w, at.to(torch.int32), at, *parts).double()
        n = (f + 1) * space
        kc, vc = nr.kv_cache_read(*parts, table,
                                  torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
        kc, vc = kc.double(), vc.double()
        q64, size = rotate(q, at)
        dq = 2.0 ** -18 * size
        dq = dq + 2.0 ** -8 * (q64.abs() + dq)
        assert torch.all((qr - q64).abs() <= dq)
        p, want = attend(q64, kc, vc)
        d = torch.einsum("qhd,khd->hqk", dq, kc.abs()).amax(-1) / D ** 0.5  # [heads, q]
        apart = (vc.transpose(0, 1)[:, None] - want.transpose(0, 1)[:, :, None]).abs()  # h q k d
        bound = torch.expm1(2 * d)[..., None] * (p[..., None] * apart).sum(2)
        err = (attend(qr, kc, vc)[1] - want).abs().transpose(0, 1)
        assert torch.all(err <= bound + 1e-12)
        # the bound is one that a wrong query does not meet
        for other in (torch.zeros_like(qr), -qr):
            off = (attend(other, kc, vc)[1] - want).abs().transpose(0, 1)
            assert (off > bound).float().mean() > 0.5
