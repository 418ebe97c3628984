"""The workspace that the library asks for is never less than what its launches
write: a mean and a sum of squares for each sample's groups (and its tiles' borders)
where there are two launches, and backwards each channel's two sums for each sample
as well, unless one launch takes a single sample."""
import ctypes
import random

import pytest

F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def query(lib_path):
    import normalisation_rope_transformers_gb300 as nrt

    def f(n, s, c, g, backward, dtype):
        out = ctypes.c_int64(-1)
        assert nrt.lib.nr_group_norm_workspace(n, s, c, g, backward, dtype, ctypes.byref(out)) == 0
        return out.value
    return f


def test_workspace_holds_at_least_one_row_a_sample(query):
    r, two = random.Random(5), 0
    for _ in range(3000):
        dtype = r.choice([F32, BF16])
        vec = 8 if dtype == BF16 else 4
        g = r.choice([1, 2, 3, 8, 32])
        c = g * vec * r.choice([1, 2, 5, 16, 100])
        n, s = r.choice([1, 2, 7, 153, 5000]), int(2 ** r.uniform(0, 24))
        if c > 65536:
            continue
        tiles = -(-c // vec // 512)
        forward, backward = query(n, s, c, g, 0, dtype), query(n, s, c, g, 1, dtype)
        assert forward == 0 or (forward >= 8 * n * (g + tiles) and forward % (8 * n * (g + tiles)) == 0)
        two += forward > 0
        both = 8 * n * (g + tiles + c)
        if backward == 0:
            assert n == 1
        elif backward != 8 * n * c:  # one launch and the sum over samples, or two launches
            assert backward >= both and backward % both == 0
        if n > 1:
            assert backward >= 8 * n * c
    assert two > 500


@pytest.mark.parametrize("n,s,c,g", [(1, 1 << 20, 128, 32), (3, 1 << 18, 320, 32), (1, 1 << 24, 8, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_sizes_take_two_launches(query, n, s, c, g, dtype):
    # a wave of blocks: at least floor(152 / n) chunks a sample, so more than 152 - n in all
    assert query(n, s, c, g, 0, dtype) >= 8 * (152 - n) * (g + 1)
    assert query(n, s, c, g, 1, dtype) >= 8 * (152 - n) * (g + 1 + c)
