"""An item's first tile in the many-rows attention kernel: it knows no row's largest score yet, and
its weights' columns are written for what it knows, then for good."""
import pytest
import torch

from tests.test_gpu_cache_attention import compare, problem, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("size", [1.0, 100.0, 1e4])
def test_many_items_of_one_tile(nr, size, dim, fmt):
    """Scores so large that e^score is infinite: nothing of it may stay.  Every item is one tile."""
    p = problem(dim, [45 + i % 80 for i in range(40)], [30 + i % 7 for i in range(40)], 2, 1, dim, 16, fmt,
                torch.bfloat16)
    p["q"] = (p["q"].float() * size).to(torch.bfloat16)
    out, lse = compare(nr, p)
    for _ in range(10):
        again, same = run(nr, p)
        assert torch.equal(again, out) and torch.equal(same, lse)
    nr.device_status()
