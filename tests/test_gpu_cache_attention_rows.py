"""Attention over the cache with many query rows a sequence (more than 16 for each K/V head on
average, bf16, heads of 64 and 128: a kernel of its own), against 64 bits."""
import numpy as np
import pytest
import torch

import tests.attention_ref as ref
from tests.test_gpu_cache_attention import compare, poison, problem, run, want

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("queries,group", [(17, 1), (5, 4), (16, 8), (33, 4), (43, 3), (70, 2), (9, 40)])
def test_row_counts(nr, queries, group, dim, fmt):
    p = problem(queries, [queries + 60, queries + 131], [queries, queries], 2, group, dim, 16, fmt, bf,
                tree=queries < 40)
    compare(nr, p)


@pytest.mark.parametrize("length", [30, 127, 128, 129, 255, 256, 257, 400, 640])
def test_lengths_around_the_tiles(nr, length):
    p = problem(length, [length, 40], [24, 24], 1, 2, 128, 16, "fp8", bf, tree=True)
    compare(nr, p)


@pytest.mark.parametrize("page", [1, 3, 16, 48, 100, 128, 256])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_page_sizes(nr, page, fmt):
    p = problem(page, [47, 300], [20, 30], 3, 2, 64, page, fmt, bf, tree=True)
    compare(nr, p)


@pytest.mark.parametrize("dim", [64, 128])
def test_one_long_sequence_over_all_blocks(nr, dim):
    p = problem(2, [9000], [20], 2, 2, dim, 64, "fp8", bf, tree=True)
    compare(nr, p)


def test_many_sequences_of_few_tiles(nr):
    """Several items a block, of different numbers of rows."""
    rng = np.random.default_rng(5)
    queries = [int(n) for n in rng.integers(1, 45, 150)]
    lens = [n + int(k) for n, k in zip(queries, rng.integers(0, 300, 150))]
    p = problem(3, lens, queries, 2, 2, 64, 16, "fp8", bf, tree=True)
    compare(nr, p)


def test_prompts(nr):
    """Chains as long as their sequences, beside ones with a context and single tokens."""
    p = problem(4, [300, 150, 260, 90], [300, 40, 1, 90], 2, 1, 64, 16, "fp8", bf)
    compare(nr, p)


@pytest.mark.parametrize("words", [1, 2, 3, 5])
def test_wide_trees_and_their_words(nr, words):
    p = problem(5, [230, 131], [90, 61], 1, 2, 64, 16, "fp8", bf, tree=True, words=3)
    if words < 3:
        p["tree"] = np.ascontiguousarray(p["tree"][:, :words])  # later tokens are seen by nobody
    elif words > 3:
        p["tree"] = np.ascontiguousarray(np.pad(p["tree"], ((0, 0), (0, words - 3)), constant_values=-1))
    compare(nr, p)


@pytest.mark.parametrize("context", [0, 1, 31, 32, 33, 95, 97, 127, 128])
def test_own_tokens_at_any_place_of_a_tile(nr, context):
    p = problem(context, [context + 40, context + 25], [40, 25], 1, 2, 64, 16, "fp8", bf, tree=True)
    compare(nr, p)
    p["tree"] = None
    compare(nr, p)


def test_rows_that_see_nothing(nr):
    p = problem(6, [30, 0, 200, 50], [30, 20, 0, 60], 2, 2, 64, 16, "fp8", bf, tree=True)
    p["tree"][:3] = 0
    p["tree"][55:] = 0
    p["table"][3, 0] = -1
    p["table"][3, 1] = 10 ** 6
    out, lse = compare(nr, p)
    assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()
    assert (out[30:50] == 0).all()


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_scales_far_apart(nr, fmt):
    p = problem(7, [500], [20], 2, 2, 128, 16, fmt, bf)
    rng = np.random.default_rng(3)
    for i in (2, 3):
        if fmt == "fp8":
            p["parts"][i] *= (2.0 ** rng.integers(-14, 3, p["parts"][i].shape)).astype(np.float32)
        else:
            p["parts"][i] = np.clip(p["parts"][i].astype(int) + rng.integers(-12, 3, p["parts"][i].shape),
                                    1, 250).astype(np.uint8)
    compare(nr, p)


def test_scores_that_rise_tile_by_tile(nr):
    """K grows along the sequence, so every tile moves the rows' references."""
    p = problem(8, [1500, 700], [24, 24], 1, 2, 128, 16, "fp8", bf)
    for s in range(2):
        for i, b in enumerate(p["table"][s]):
            if b >= 0:
                p["parts"][2][b] *= np.float32(1.0 + 0.3 * i)
    compare(nr, p)
    p["q"] = -p["q"]
    compare(nr, p, scale=-0.3)


@pytest.mark.parametrize("q_scale", [1e-30, 1e-4, 3000.0, 1e30])
def test_queries_of_any_size(nr, q_scale):
    p = problem(9, [190], [20], 1, 2, 128, 16, "fp8", bf)
    p["q"] = (p["q"].float() * q_scale).to(bf)
    compare(nr, p, scale=0.1 / q_scale)
    compare(nr, p, scale=0.0)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_nan_where_nobody_looks(nr, fmt):
    p = problem(10, [237, 121], [35, 24], 2, 2, 64, 16, fmt, bf, tree=True)
    p["tree"][:, 0] &= ~np.int32(1 << 2)  # token 2 of each draft is seen by nobody
    clean = run(nr, p)
    ref.check(*clean, want(p, 64 ** -0.5), bf)
    slots = []
    for s, n in enumerate(p["lens"]):
        last = p["table"][s, (n - 1) // 16]
        slots += [(last, place) for place in range(n % 16, 16)]
        pos = n - (p["cu"][s + 1] - p["cu"][s]) + 2
        slots.append((p["table"][s, pos // 16], pos % 16))
    used = set(int(b) for s, n in enumerate(p["lens"]) for b in p["table"][s, :-(-n // 16)])
    slots += [(b, 0) for b in range(p["parts"][0].shape[0]) if b not in used]
    poison(p, slots, fmt)
    for a, b in zip(clean, run(nr, p)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("length", [60, 4000])
def test_nan_reaches_those_who_see_it(nr, fmt, length):
    """A NaN in V of a drafted token: its dimensions of the queries that see it, whether a block
    has the whole sequence or a part; in the context: of every query."""
    p = problem(11, [length], [20], 1, 2, 64, 16, fmt, bf, tree=True)
    clean, lse = run(nr, p)
    pos = length - 20 + 3
    b, place = p["table"][0, pos // 16], pos % 16
    if fmt == "fp8":
        p["parts"][1][b, place, 0, 5] = 0x7F
        dims = [5]
    else:
        p["parts"][3][b, place, 0, 1] = 255
        dims = list(range(32, 64))
    dirty, lse2 = run(nr, p)
    assert torch.equal(lse, lse2)
    nan = torch.isnan(dirty)
    expect = torch.zeros_like(nan)
    for t in range(20):
        if p["tree"][t, 0] >> 3 & 1:
            expect[t, :, dims] = True
    assert expect.any() and torch.equal(nan, expect)
    assert torch.equal(dirty[~nan], clean[~nan])
    if fmt == "fp8":
        p["parts"][1][p["table"][0, 0], 1, 0, 7] = 0xFF
        dirty, _ = run(nr, p)
        expect[:, :, 7] = True
        assert torch.equal(torch.isnan(dirty), expect)


def test_nan_query_leaves_its_neighbours_alone(nr):
    p = problem(12, [150], [20], 1, 2, 64, 16, "fp8", bf)
    clean, _ = run(nr, p)
    p["q"][7, 1, 3] = float("nan")
    out, lse = run(nr, p)
    assert torch.isnan(out[7, 1]).all() and torch.isnan(lse[7, 1])
    keep = torch.ones(20, 2, dtype=torch.bool)
    keep[7, 1] = False
    assert torch.equal(out[keep], clean[keep])


def test_bad_offsets_stay_in_bounds(nr):
    p = problem(13, [30, 20, 10], [30, 20, 10], 1, 2, 64, 16, "fp8", bf)
    p["cu"] = np.array([-5, 30, 10, 1000], np.int32)
    p["lens"] = np.array([30, -4, 10], np.int32)
    out, _ = run(nr, p)
    assert torch.isfinite(out[:30]).all()


def test_strided_queries_and_blocks_and_rows_of_no_sequence(nr):
    p = problem(14, [133, 100], [30, 22], 2, 2, 128, 16, "fp8", bf, wide=4096)
    qkv = torch.zeros(55, 8, 128, dtype=bf, device="cuda")
    qkv[1:53, :4] = p["q"].cuda()
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    out = torch.full((55, 4, 128), 7.0, dtype=bf, device="cuda")
    got, lse = nr.cache_attention(qkv[:, :4], *ref.to_gpu(p["parts"], 4096), dev(p["table"]),
                                  dev(p["lens"]), cu_q=dev(p["cu"] + 1), out=out, return_lse=True)
    assert got is out and (out[0] == 7).all() and (out[53:] == 7).all()
    ref.check(out[1:53], lse[1:53], want(p, 128 ** -0.5), bf)


def test_same_bits_each_time_in_graphs_and_on_two_streams(nr):
    ps = [problem(15 + i, [2500 + i, 95, 700], [40, 10, 25], 2, 4, 128, 16, "fp8", bf, tree=True)
          for i in range(2)]
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    args = [[p["q"].cuda(), *ref.to_gpu(p["parts"]), dev(p["table"]), dev(p["lens"]), dev(p["cu"]),
             dev(p["tree"])] for p in ps]
    alone = [nr.cache_attention(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(nr.cache_attention(*args[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for x in got[i]:
            assert torch.equal(x, alone[i])
    held = torch.zeros_like(alone[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nr.cache_attention(*args[0], out=held)
    for _ in range(3):
        held.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, alone[0])
    nr.device_status()


def test_both_kernels_agree(nr):
    """The same queries in one call with many rows and one sequence at a time with few."""
    p = problem(17, [500, 333], [40, 1], 2, 4, 128, 16, "fp8", bf, tree=True)
    out, lse = compare(nr, p)
    one = {**p, "q": p["q"][40:], "table": p["table"][1:], "lens": p["lens"][1:],
           "cu": np.array([0, 1], np.int32), "tree": p["tree"][40:]}
    o, z = compare(nr, one)
    assert torch.allclose(o.float(), out[40:].float(), rtol=2 ** -7, atol=1e-3)
    assert torch.allclose(z, lse[40:], rtol=1e-5)


def test_offsets_past_32_bits(nr):
    blocks, page, heads, dim = 70000, 64, 8, 128
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    p = problem(30, [250], [20], heads, 1, dim, page, "fp8", bf)
    small = ref.to_gpu(p["parts"])
    big = [torch.empty(blocks, *x.shape[1:], dtype=x.dtype, device="cuda") for x in small]
    assert big[0].numel() > 1 << 32
    n = small[0].shape[0]
    for x, y in zip(big, small):
        x[blocks - n:] = y
    table = torch.from_numpy(p["table"] + np.where(p["table"] >= 0, blocks - n, 0).astype(np.int32)).cuda()
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    out, lse = nr.cache_attention(p["q"].cuda(), *big, table, dev(p["lens"]), cu_q=dev(p["cu"]),
                                  return_lse=True)
    ref.check(out, lse, want(p, dim ** -0.5), bf)
