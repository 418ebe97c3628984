"""The temperatures that log probabilities and their gradient take: where log2(e) / T is infinite, or a
masked logit's distance times 1 / T is not enough for a probability of 0, the call is refused."""
import pytest

from tests.test_abi_host import OK, VALUE
from tests.test_attention_logprobs_host import grad, nrt, score  # noqa: F401


@pytest.mark.parametrize("inv_t,want", [
    (2.0 ** 127, OK), (2.0 ** -90, OK), (1.0, OK), (2.4e38, VALUE), (3.4e38, VALUE), (2.0 ** -91, VALUE),
    (1e-38, VALUE), (float("nan"), VALUE)])
def test_inverse_temperatures(nrt, inv_t, want):  # noqa: F811
    assert score(nrt, rows=0, inv_t=inv_t) == want
    assert grad(nrt, rows=0, inv_t=inv_t) == want


@pytest.mark.parametrize("temperature", [4e-39, 1e28, 1e300])
def test_temperatures_of_the_binding(nrt, monkeypatch, temperature):  # noqa: F811
    import torch

    monkeypatch.setattr(nrt, "_cuda", lambda *ts: None)
    monkeypatch.setattr(nrt, "_launch", lambda device, fn, *args: nrt._check(fn(*args, None)))
    monkeypatch.setattr(nrt, "_checked", {})
    with pytest.raises(nrt.NrError):
        nrt.token_logprobs(torch.zeros(2, 9), torch.zeros(2, dtype=torch.int64), temperature=temperature)
