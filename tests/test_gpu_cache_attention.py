"""Attention over the quantised paged cache against a plain reference in 64 bits."""
import numpy as np
import pytest
import torch

import tests.attention_ref as ref
import tests.cache_ref as cache_ref

pytestmark = pytest.mark.gpu


def problem(seed, lens, queries, heads, group, dim, page, fmt, dtype, tree=False, words=None, wide=0):
    """A cache with shuffled pages, queries and tables; (call arguments, reference arguments)."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    blocks = sum(need) + 3
    order = rng.permutation(blocks).astype(np.int32)
    table = np.full((len(lens), max(1, max(need, default=0))), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    parts = ref.make_cache(rng, blocks, page, heads, dim, fmt)
    cu = np.concatenate([[0], np.cumsum(queries)]).astype(np.int32)
    q = torch.from_numpy((1.5 * rng.standard_normal((int(cu[-1]), heads * group, dim)))
                         .astype(np.float32)).to(dtype)
    mask = None
    if tree:
        words = words or -(-max(queries) // 32)
        mask = np.concatenate([ref.tree_masks(rng, n, words) for n in queries])
    return dict(q=q, parts=parts, table=table, lens=np.array(lens, np.int32), cu=cu, tree=mask,
                wide=wide)


def run(nr, p, scale=None, cu=True, **kw):
    dev = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
    return nr.cache_attention(p["q"].cuda(), *ref.to_gpu(p["parts"], p["wide"]), dev(p["table"]),
                              dev(p["lens"]), cu_q=dev(p["cu"]) if cu else None,
                              tree=dev(p["tree"]), scale=scale, return_lse=True, **kw)


def want(p, scale):
    return ref.attention(p["q"].double().numpy(), p["parts"], p["table"], p["lens"], p["cu"],
                         p["tree"], scale, p["q"].dtype == torch.float32)


def compare(nr, p, scale=None, cu=True, **kw):
    out, lse = run(nr, p, scale, cu, **kw)
    ref.check(out, lse, want(p, p["q"].shape[2] ** -0.5 if scale is None else scale), p["q"].dtype)
    return out, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_token_a_sequence(nr, dim, fmt, dtype):
    p = problem(dim, [1, 2, 15, 16, 17, 63, 64, 65, 128, 500], [1] * 10, 2, 4, dim, 16, fmt, dtype)
    compare(nr, p, cu=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_trees(nr, dim, fmt, dtype):
    p = problem(dim + 1, [7, 40, 129, 300], [7, 13, 1, 33], 2, 3, dim, 8, fmt, dtype, tree=True)
    compare(nr, p)


@pytest.mark.parametrize("group", [1, 2, 5, 8, 16, 17, 40])
@pytest.mark.parametrize("queries", [1, 2, 5])
def test_query_heads_of_a_group(nr, group, queries):
    p = problem(group, [70, 33], [queries] * 2, 2, group, 64, 16, "fp8", torch.bfloat16)
    compare(nr, p)


@pytest.mark.parametrize("page", [1, 3, 8, 48, 64, 100, 256])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_page_sizes(nr, page, fmt):
    p = problem(page, [1, 47, 100, 259], [2, 3, 1, 5], 3, 2, 128, page, fmt, torch.bfloat16, tree=True)
    compare(nr, p)


def test_long_sequence_beside_short_ones(nr):
    p = problem(5, [9000, 3, 64, 2500], [1, 1, 1, 1], 1, 4, 128, 64, "fp8", torch.bfloat16)
    compare(nr, p, cu=False)


def test_many_sequences(nr):
    rng = np.random.default_rng(1)
    lens = [int(n) for n in rng.integers(1, 40, 300)]
    p = problem(6, lens, [1] * 300, 1, 2, 64, 16, "fp8", torch.bfloat16)
    compare(nr, p, cu=False)


def test_many_new_tokens_at_once(nr):
    """A prompt attended in one call (a chain of as many queries as positions)."""
    p = problem(7, [150, 90], [150, 40], 1, 2, 64, 16, "fp8", torch.bfloat16)
    compare(nr, p)


def test_wide_tree(nr):
    p = problem(8, [200, 131], [100, 97], 2, 2, 128, 16, "fp8", torch.bfloat16, tree=True)
    compare(nr, p)


def test_more_words_than_needed_and_fewer(nr):
    p = problem(9, [60, 50], [5, 3], 1, 2, 64, 16, "fp8", torch.bfloat16, tree=True, words=4)
    compare(nr, p)
    p = problem(10, [90, 50], [40, 3], 1, 2, 64, 16, "fp8", torch.bfloat16, tree=True, words=2)
    p["tree"] = np.ascontiguousarray(p["tree"][:, :1])  # tokens from 32 on are seen by nobody
    compare(nr, p)


def test_rows_that_see_nothing(nr):
    """Empty masks without a context, sequences without tokens or queries, positions without a
    page, more queries than tokens."""
    p = problem(11, [4, 0, 30, 40, 2], [4, 1, 0, 3, 5], 2, 3, 64, 16, "fp8", torch.bfloat16, tree=True)
    p["tree"][:2] = 0
    p["tree"][5:8] = 0
    p["table"][3] = [-1, 10 ** 6, 5]  # only the last 8 positions are there
    out, lse = compare(nr, p)
    assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()
    p = problem(12, [2, 0], [5, 2], 2, 3, 64, 16, "fp8", torch.bfloat16)  # chains
    out, lse = compare(nr, p)
    assert (out[:3] == 0).all() and torch.isinf(lse[:3]).all()


def test_length_past_the_table(nr):
    p = problem(13, [64, 20], [2, 2], 1, 2, 64, 16, "fp8", torch.bfloat16)
    p["table"] = np.ascontiguousarray(p["table"][:, :2])
    p["lens"][0] = 66  # its new tokens are past the table: 32 positions remain
    compare(nr, p)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_strided_queries_and_blocks(nr, dtype):
    p = problem(14, [33, 100], [3, 2], 2, 2, 128, 16, "fp8", dtype, wide=4096)
    parts = ref.to_gpu(p["parts"], 4096)
    assert parts[0].stride(0) > parts[0][0].numel()
    qkv = torch.zeros(5, 4 + 2 + 2, 128, dtype=dtype, device="cuda")
    qkv[:, :4] = p["q"].cuda()
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    out, lse = nr.cache_attention(qkv[:, :4], *parts, dev(p["table"]), dev(p["lens"]),
                                  cu_q=dev(p["cu"]), return_lse=True)
    ref.check(out, lse, want(p, 128 ** -0.5), dtype)


def test_mxfp4_scales_at_odd_addresses(nr):
    p = problem(15, [33, 100], [3, 2], 3, 2, 128, 16, "mxfp4", torch.bfloat16)
    parts = ref.to_gpu(p["parts"])
    for i in (2, 3):
        buf = torch.zeros(parts[i].numel() + 3, dtype=torch.uint8, device="cuda")
        buf[3:] = parts[i].flatten()
        parts[i] = buf[3:].view(parts[i].shape)
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    out, lse = nr.cache_attention(p["q"].cuda(), *parts, dev(p["table"]), dev(p["lens"]),
                                  cu_q=dev(p["cu"]), return_lse=True)
    ref.check(out, lse, want(p, 128 ** -0.5), torch.bfloat16)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_scales_far_apart(nr, fmt, dtype):
    """Tokens whose K or V is many powers of two larger than the others'."""
    p = problem(16, [200], [3], 2, 2, 128, 16, fmt, dtype)
    rng = np.random.default_rng(3)
    for i in (2, 3):
        if fmt == "fp8":
            p["parts"][i] *= (2.0 ** rng.integers(-14, 3, p["parts"][i].shape)).astype(np.float32)
        else:
            p["parts"][i] = np.clip(p["parts"][i].astype(int) + rng.integers(-12, 3, p["parts"][i].shape),
                                    1, 250).astype(np.uint8)
    compare(nr, p)


def test_zero_scales(nr):
    """A cache of zeros (its scales among them): every weight is the same, the output zero."""
    p = problem(17, [70], [2], 1, 2, 64, 16, "fp8", torch.bfloat16)
    for x in p["parts"]:
        x[:] = 0
    out, lse = run(nr, p)
    assert (out == 0).all()
    assert torch.allclose(lse, torch.tensor([69.0, 70.0], device="cuda").log()[:, None].expand(2, 2),
                          rtol=1e-6)


def poison(p, slots, fmt):
    """NaN codes and scales at (block, place) slots."""
    for b, place in slots:
        for i in range(2):
            p["parts"][i][b, place] = 0x7F if fmt == "fp8" else 0x77
            p["parts"][2 + i][b, place] = np.float32(np.inf if i else np.nan) if fmt == "fp8" else 255


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_nan_where_nobody_looks(nr, fmt, dtype):
    """Behind the sequence's end, in pages of nobody, and in a drafted token that no query
    sees: the result is that of a clean cache, bit for bit."""
    p = problem(18, [37, 21], [5, 4], 2, 2, 64, 16, fmt, dtype, tree=True)
    p["tree"] &= ~np.int32(1 << 2)  # token 2 of each draft is seen by nobody
    clean = run(nr, p)
    ref.check(*clean, want(p, 64 ** -0.5), dtype)
    slots = []
    for s, n in enumerate(p["lens"]):
        last = p["table"][s, (n - 1) // 16]
        slots += [(last, place) for place in range(n % 16, 16)]
        pos = n - (p["cu"][s + 1] - p["cu"][s]) + 2
        slots.append((p["table"][s, pos // 16], pos % 16))
    used = set(int(b) for s, n in enumerate(p["lens"]) for b in p["table"][s, :-(-n // 16)])
    slots += [(b, 0) for b in range(p["parts"][0].shape[0]) if b not in used]
    poison(p, slots, fmt)
    dirty = run(nr, p)
    for a, b in zip(clean, dirty):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_nan_reaches_those_who_see_it(nr, fmt):
    """A NaN in V of a drafted token: its dimensions of the queries that see it, nothing else."""
    p = problem(19, [37], [6], 1, 2, 64, 16, fmt, torch.bfloat16, tree=True)
    p["tree"][:, 0] = [1, 3, 5, 9, 19, 33]  # tokens 1 and 4 see token 1
    clean, lse = run(nr, p)
    pos = 37 - 6 + 1
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
    for t in (1, 4):
        expect[t, :, dims] = True
    assert torch.equal(nan, expect)
    assert torch.equal(dirty[~nan], clean[~nan])


def test_infinite_scores_of_a_query(nr):
    """A NaN query gives NaN and leaves its neighbours alone."""
    p = problem(20, [50], [3], 1, 4, 64, 16, "fp8", torch.bfloat16)
    clean, _ = run(nr, p)
    p["q"][1, 2, 7] = float("nan")
    out, lse = run(nr, p)
    assert torch.isnan(out[1, 2]).all() and torch.isnan(lse[1, 2])
    keep = torch.ones(3, 4, dtype=torch.bool)
    keep[1, 2] = False
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("q_scale", [1e-30, 1e-4, 3000.0, 1e30])
def test_queries_of_any_size(nr, q_scale):
    p = problem(21, [90], [3], 1, 4, 128, 16, "fp8", torch.bfloat16)
    p["q"] = (p["q"].float() * q_scale).to(torch.bfloat16)
    compare(nr, p, scale=0.1 / q_scale)


def test_negative_and_zero_scale(nr):
    p = problem(22, [90], [3], 1, 4, 64, 16, "fp8", torch.bfloat16)
    compare(nr, p, scale=-0.2)
    compare(nr, p, scale=0.0)


def test_rows_of_no_sequence_keep_what_they_held(nr):
    p = problem(23, [30, 20], [2, 3], 1, 2, 64, 16, "fp8", torch.bfloat16)
    p["q"] = torch.cat([p["q"][:1], p["q"], p["q"][:2]])
    p["cu"] = p["cu"] + 1  # one row in front, two behind
    out = torch.full(p["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    got, _ = run(nr, p, out=out)
    assert got is out
    assert (out[0] == 7).all() and (out[-2:] == 7).all()
    w = want(p, 64 ** -0.5)
    ref.check(out, None, w, torch.bfloat16)


def test_bad_offsets_stay_in_bounds(nr):
    """cu_q that leaves q, lengths below zero: clamped, no row outside is written."""
    p = problem(24, [30, 20, 10], [2, 3, 1], 1, 2, 64, 16, "fp8", torch.bfloat16)
    p["cu"] = np.array([-5, 2, 1, 1000], np.int32)
    p["lens"] = np.array([30, -4, 10], np.int32)
    out, _ = run(nr, p)
    assert torch.isfinite(out).all()


def test_same_bits_each_time_and_in_a_graph(nr):
    p = problem(25, [3000, 45, 700], [5, 1, 9], 2, 4, 128, 16, "fp8", torch.bfloat16)
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    args = [p["q"].cuda(), *ref.to_gpu(p["parts"]), dev(p["table"]), dev(p["lens"])]
    cu = dev(p["cu"])
    out, lse = nr.cache_attention(*args, cu_q=cu, return_lse=True)
    again, _ = nr.cache_attention(*args, cu_q=cu, return_lse=True)
    assert torch.equal(out, again)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        nr.cache_attention(*args, cu_q=cu)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    held = torch.zeros_like(out)
    with torch.cuda.graph(graph):
        nr.cache_attention(*args, cu_q=cu, out=held)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, out)
    # lengths are read on the device: a replay follows them
    lens2 = np.array([1200, 45, 90], np.int32)
    args[6].copy_(dev(lens2))
    graph.replay()
    torch.cuda.synchronize()
    ref.check(held, None, want({**p, "lens": lens2}, 128 ** -0.5), torch.bfloat16)


def test_two_streams_at_once(nr):
    ps = [problem(26 + i, [700 + i, 45], [3, 1], 2, 4, 64, 16, "fp8", torch.bfloat16) for i in range(2)]
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    args = [[p["q"].cuda(), *ref.to_gpu(p["parts"]), dev(p["table"]), dev(p["lens"]), dev(p["cu"])]
            for p in ps]
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


def test_offsets_past_32_bits(nr):
    """A cache of more than 4 GiB: the last blocks' codes and the table's far end."""
    blocks, page, heads, dim = 70000, 64, 8, 128
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    p = problem(30, [150], [2], heads, 1, dim, page, "fp8", torch.bfloat16)
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
    ref.check(out, lse, want(p, dim ** -0.5), torch.bfloat16)


def test_nothing_to_do(nr):
    p = problem(31, [5], [1], 1, 1, 64, 16, "fp8", torch.bfloat16)
    parts = ref.to_gpu(p["parts"])
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    out = nr.cache_attention(p["q"][:0].cuda(), *parts, i32(0, 3), i32(0))
    assert out.shape == (0, 1, 64)
    out = nr.cache_attention(p["q"][:0].cuda(), *parts, i32(2, 3), i32(2), cu_q=i32(3),
                             tree=i32(0, 1))
    assert out.shape == (0, 1, 64)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("group,queries", [(1, [7, 9]), (3, [3, 2]), (4, [1, 1]), (4, [4, 4]), (5, [1, 5]),
                                           (8, [3, 3]), (23, [1, 1]), (6, [13, 1, 1])])
def test_rows_on_both_sides_of_each_variant(nr, dim, fmt, group, queries):
    """8, 16 and 24 query rows an item, the average and single sequences on either side."""
    p = problem(group + dim, [50 + 90 * i for i in range(len(queries))], queries, 2, group, dim, 16, fmt,
                torch.bfloat16, tree=True)
    compare(nr, p)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_rising_scores(nr, dim, dtype):
    """Scores that rise slowly along the sequence (each step's maximum above the one before it, by less
    and by more than the references lag), and fall."""
    for sign in (1, -1):
        for width in (0.02, 0.3, 4.0):
            p = problem(dim, [900, 37], [1, 1], 1, 4, dim, 16, "fp8", dtype)
            codes, scales = p["parts"][0], p["parts"][2]
            one = cache_ref.quant(np.ones((1, 1, 1, dim), np.float32), "fp8")[0][0, 0, 0]
            for s, n in enumerate((900, 37)):
                for pos in range(n):
                    at = p["table"][s, pos // 16], pos % 16
                    codes[at] = one
                    scales[at] = width * (pos if sign > 0 else n - pos) / dim ** 0.5 / 448
            p["q"] = torch.ones_like(p["q"])
            compare(nr, p, cu=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 2, 4])
def test_nan_reaches_those_who_see_it_whatever_the_rows(nr, group, dim, fmt, dtype):
    """6, 12 and 24 query rows an item; two sequences, two heads, the NaN in one of each; one more in
    front of the drafts, which everyone of its sequence sees."""
    p = problem(20 + group, [70, 37], [6, 6], 2, group, dim, 16, fmt, dtype, tree=True)
    p["tree"][6:, 0] = [1, 3, 5, 9, 19, 33]  # tokens 1 and 4 see token 1
    clean, lse = run(nr, p)
    block = 32 if fmt == "mxfp4" else 1
    expect = torch.zeros(clean.shape, dtype=torch.bool, device="cuda")

    def spoil(s, pos, head, d):
        b, place = p["table"][s, pos // 16], pos % 16
        if fmt == "fp8":
            p["parts"][1][b, place, head, d] = 0xFF
        else:
            p["parts"][3][b, place, head, d // 32] = 255
        return slice(d // block * block, d // block * block + block)

    dims = spoil(1, 37 - 6 + 1, 1, 37)
    for t in (7, 10):
        expect[t, group:, dims] = True
    dims = spoil(0, 40, 0, dim - 1)
    expect[:6, :group, dims] = True
    dirty, lse2 = run(nr, p)
    assert torch.equal(lse, lse2)
    nan = torch.isnan(dirty)
    assert torch.equal(nan, expect)
    assert torch.equal(dirty[~nan], clean[~nan])
