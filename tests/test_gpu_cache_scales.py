"""The FP8 cache's scale is the correctly rounded quotient a / 448 for every
significand of a, at the least and the largest binade that a row's clamped magnitude
has and in between: it is computed by a product and a correction, no division."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("exponent", [-100, -96, 0, 8, 127])
def test_every_significand(nr, exponent):
    n, dim = 1 << 23, 16
    bits = torch.arange(n, dtype=torch.int32) + ((exponent + 127) << 23)
    a = bits.view(torch.float32)
    k = torch.zeros(n, 1, dim, device="cuda")
    k[:, 0, 5] = a.cuda()
    v = -k
    page = 64
    codes = [torch.zeros(n // page, page, 1, dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(n // page, page, 1, device="cuda") for _ in range(2)]
    nr.kv_cache_write(k, v, torch.arange(n, device="cuda"), *codes, *scales)
    want = torch.from_numpy(a.numpy() / np.float32(448)).cuda()
    for s in scales:
        assert torch.equal(s.view(-1), want)
    # a * (448 / a), both rounded, is within 2 ulps of 448: the largest code
    assert torch.all(codes[0].view(n, dim)[:, 5] == 0x7E)
    assert torch.all(codes[1].view(n, dim)[:, 5] == 0xFE)
