"""The rotary angles of the preamble that writes the cache, element by element.

A query head of ones in the first half of each pair and zeros in the second comes
out as A cos a and A sin a, A^2 the inverse of its mean square, with eps = 0 and
weights of one.  Written as A f(r) with r the angle from the nearest quarter turn
and f one of +-cos, +-sin, the result is off by
  A |f'(r)| d   for an angle that is off by d: the reduced angle is cut to 2^-32 turns,
                the constants of a turn are good to 2^-51 of the angle (below 2^-38
                turns here), and r is rounded once to 24 bits: d <= 2^-24 |r| + 1.1 *
                2 pi 2^-32
  2^-21 A |f|   for sincospif (an ulp, 2^-23), rsqrtf (two ulps, 2^-22) and a product
                (2^-24)
and the reference, in 64 bits, by less than 10^-11 of an angle below 2 * 10^4."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,rot,interleaved,mrope", [
    (128, 128, False, False), (256, 256, False, False), (32, 32, False, False),
    (128, 64, False, False), (128, 128, True, False), (64, 16, True, False),
    (128, 128, False, True),
])
def test_far_and_near_angles(nr, D, rot, interleaved, mrope):
    T, half, dev = 26598, rot // 2, "cuda"
    i = torch.arange(half, device=dev)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    q = torch.zeros(T, 1, D, device=dev)
    q[:, :, first] = 1
    w = torch.ones(D, device=dev)
    pos = (torch.arange(T, device=dev) - T // 2).to(torch.int32)
    kw, per_pair = {}, pos.double()[:, None].expand(T, half)
    if mrope:
        pos = torch.stack([pos, pos.flip(0), pos // 3])
        kw["mrope_sections"] = (16, 24, 24)
        axis = torch.repeat_interleave(torch.arange(3, device=dev),
                                       torch.tensor([16, 24, 24], device=dev))
        per_pair = pos.double().t()[:, axis]
    cache = [torch.zeros(T, 1, 1, D, dtype=torch.uint8, device=dev) for _ in range(2)]
    cache += [torch.zeros(T, 1, 1, device=dev) for _ in range(2)]
    out = nr.qk_norm_rope_cache(q, q, q, w, w, pos, torch.arange(T, device=dev), *cache, eps=0.0,
                                rotary_dim=rot, interleaved=interleaved, **kw).double()[:, 0]
    freq = torch.tensor([1e4 ** (-2 * j / rot) for j in range(half)], dtype=torch.float64, device=dev)
    a = per_pair * freq
    A = (2 * D / rot) ** 0.5
    r = a - torch.round(a / (math.pi / 2)) * (math.pi / 2)
    d = 2.0 ** -24 * r.abs() + 1.1 * 2 * math.pi * 2.0 ** -32 + 1e-11
    for got, want, slope in ((out[:, first], a.cos(), a.sin()), (out[:, second], a.sin(), a.cos())):
        tol = A * (slope.abs() * d + d * d + 2.0 ** -21 * want.abs())
        over = (got - A * want).abs() / tol
        assert over.max() <= 1, "%.2f of the tolerance, %d of %d elements over it" % (
            over.max(), int((over > 1).sum()), over.numel())
