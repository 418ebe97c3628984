"""K and Q of any size in attention over the cache: scores are finite wherever scale * q * k is, although
products of the codes with Q, or with K's scale alone, are not."""
import numpy as np
import pytest
import torch

from tests.test_gpu_cache_attention import compare, problem

pytestmark = pytest.mark.gpu

ROWS = {"few": ([3, 2], 2), "many": ([30, 40], 2)}


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("k,q", [(113, -100), (116, -90), (60, 60), (-90, 100), (-60, -60)])
def test_sizes_of_keys_and_queries(nr, k, q, dim, fmt, dtype, rows):
    """K times 2^k, Q times 2^q, the scores' scale times 2^-(k + q)."""
    queries, group = ROWS[rows]
    p = problem(dim, [150, 213], queries, 2, group, dim, 16, fmt, dtype)
    if fmt == "fp8":
        p["parts"][2] *= np.float32(2.0 ** k)
    else:
        p["parts"][2] = (p["parts"][2].astype(int) + k).astype(np.uint8)
    p["q"] = (p["q"].float() * 2.0 ** q).to(dtype)
    compare(nr, p, scale=0.1 * 2.0 ** -(k + q))
