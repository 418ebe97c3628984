"""The gradient of log probabilities and entropy where a masked logit meets a large incoming gradient:
nothing but finite numbers, next to masked places too.  (A factor common to a row's incoming gradients is
one of its result, so the reference is the result for a small one.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("mask", [-float("inf"), -3e38, -2e9, -1200.0])
@pytest.mark.parametrize("power", [10, 30, 60, 100])
def test_large_gradients_beside_masked_logits(nr, power, mask, dtype):
    g = torch.Generator(device="cuda").manual_seed(power)
    x = torch.randn(5, 3001, generator=g, device="cuda").to(dtype)
    x[:, ::3] = mask
    tokens = torch.tensor([1, 0, -1, 3000, 2], device="cuda")
    r = nr.token_logprobs(x, tokens)
    one = torch.randn(5, generator=g, device="cuda")
    two = torch.randn(5, generator=g, device="cuda")
    small = nr.token_logprobs_backward(one, two, x, tokens, r.lse, r.entropy)
    f = 2.0 ** power
    big = nr.token_logprobs_backward(one * f, two * f, x, tokens, r.lse, r.entropy)
    assert torch.isfinite(small).all()
    # powers of two scale every operation of the formula exactly, but near the end of f32's range below
    near = small.float().abs() < 2.0 ** -100
    assert torch.equal(big.float()[~near], small.float()[~near] * f)
    assert (big.float()[near].abs() <= 2.0 ** (power - 99)).all()
