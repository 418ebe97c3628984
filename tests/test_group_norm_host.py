"""The geometry of the group-norm launches, on the CPU: the workspace that the
library asks for holds what its blocks write, at every size, and no size is
refused for want of it."""
import ctypes
import random

import pytest

F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def query(lib_path):
    import normalisation_rope_transformers_gb300 as nrt

    def f(n, s, c, g, backward, dtype):
        out = ctypes.c_int64(-1)
        status = nrt.lib.nr_group_norm_workspace(n, s, c, g, backward, dtype, ctypes.byref(out))
        return status, out.value
    return f


def test_workspace_is_never_more_than_a_few_rows_a_block(query):
    """At most (groups + tiles + channels) values of 8 bytes for each of at most 4
    waves of 152 blocks, or one block a sample."""
    r = random.Random(4)
    for _ in range(3000):
        dtype = r.choice([F32, BF16])
        vec = 8 if dtype == BF16 else 4
        g = r.choice([1, 2, 3, 8, 32])
        c = g * vec * r.choice([1, 2, 5, 16, 100])
        if c > 65536:
            continue
        n, s = r.choice([1, 2, 7, 153, 5000]), int(2 ** r.uniform(0, 24))
        for backward in (0, 1):
            status, size = query(n, s, c, g, backward, dtype)
            assert status == 0
            tiles = -(-c // vec // 512)
            blocks = max(4 * 152, n)
            assert 0 <= size <= 8 * blocks * (g + tiles + c), (n, s, c, g)


def test_largest_sizes(query):
    assert query(1, 1 << 36, 64, 8, 0, BF16)[0] == 0
    assert query(1 << 20, 16, 64, 8, 1, BF16)[0] == 0
    assert query(1, 4, 65536, 1, 0, F32)[0] == 0
    assert query((1 << 31) - 1, 1, 65536, 65536, 0, F32)[0] == 2  # too many blocks
