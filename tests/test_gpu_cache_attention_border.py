"""Where attention over the cache goes from the kernel for few query rows to the one for many: sizes on
both sides of the border that the source names, which kernel each of them takes, and the many-rows
kernel's addresses in a cache of more than 4 GiB."""
import os
import re

import numpy as np
import pytest
import torch

import tests.attention_ref as ref
from tests.test_gpu_cache_attention import compare, problem, run, want
from tests.test_kernel_loads_host import CSRC, code

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:DEBUG")]  # of the graph's dump
bf = torch.bfloat16

FEW = int(re.search(r"\bkFewRows = (\d+);", code(os.path.join(CSRC, "cache_attention.cu"))).group(1))


def kernels(nr, p, path):
    """The names of the kernels that a call launches, from a captured graph."""
    dev = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
    args = [p["q"].cuda(), *ref.to_gpu(p["parts"]), *(dev(p[k]) for k in ("table", "lens", "cu", "tree"))]
    nr.cache_attention(*args)
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    graph.enable_debug_mode()
    with torch.cuda.graph(graph):
        nr.cache_attention(*args)
    graph.debug_dump(str(path))
    with open(path) as f:
        return set(re.findall(r"cache_attention_(?:rows_)?kernel", f.read()))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("queries,group", [
    ([FEW - 1] * 2, 1), ([FEW] * 2, 1), ([FEW + 1] * 2, 1), ([FEW + 2] * 2, 1),  # rows of each sequence
    ([FEW // 8] * 2, 8), ([FEW // 8 + 1] * 2, 8), ([FEW // 4 + 1] * 2, 4),
    ([1, 2 * FEW - 1], 1), ([1, 2 * FEW], 1), ([2, 2 * FEW], 1)])  # averages of FEW, FEW + 1/2, FEW + 1
def test_both_sides_of_the_border(nr, tmp_path, queries, group, fmt, dim):
    p = problem(sum(queries) + dim, [max(queries) + 60, max(queries) + 131], queries, 2, group, dim, 16, fmt,
                bf, tree=True)
    compare(nr, p)
    many = dim <= 128 and sum(queries) * group > FEW * len(queries)
    assert kernels(nr, p, tmp_path / "graph.dot") == {
        "cache_attention_rows_kernel" if many else "cache_attention_kernel"}


def test_f32_tensors_take_the_kernel_for_few_rows(nr, tmp_path):
    p = problem(1, [150, 160], [40, 50], 2, 2, 128, 16, "fp8", torch.float32, tree=True)
    compare(nr, p)
    assert kernels(nr, p, tmp_path / "graph.dot") == {"cache_attention_kernel"}


@pytest.mark.parametrize("fmt,blocks", [("fp8", 70000), ("mxfp4", 140000)])
def test_many_rows_past_32_bits(nr, tmp_path, fmt, blocks):
    """The last blocks of the cache: loads of both sides, and the second look at V's NaN."""
    page, heads, dim = 64, 8, 128
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    p = problem(30, [250], [20], heads, 2, dim, page, fmt, bf)
    assert 20 * 2 > FEW
    small = ref.to_gpu(p["parts"])
    big = [torch.empty(blocks, *x.shape[1:], dtype=x.dtype, device="cuda") for x in small]
    assert big[0].numel() > 1 << 32
    n = small[0].shape[0]
    at = np.where(p["table"] >= 0, p["table"] + blocks - n, -1).astype(np.int32)
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731

    def call():
        return nr.cache_attention(p["q"].cuda(), *big, dev(at), dev(p["lens"]), cu_q=dev(p["cu"]),
                                  return_lse=True)

    for x, y in zip(big, small):
        x[blocks - n:] = y
    out, lse = call()
    ref.check(out, lse, want(p, dim ** -0.5), bf)
    # a NaN in V of the sixth new token, head 3, dimension 70: the tokens from it on see it
    pos = 250 - 20 + 5
    b, place = at[0, pos // page], pos % page
    if fmt == "fp8":
        big[1][b, place, 3, 70] = 0x7F
        dims = slice(70, 71)
    else:
        big[3][b, place, 3, 2] = 255
        dims = slice(64, 96)
    dirty, same = call()
    expect = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    expect[5:, 6:8, dims] = True
    nan = torch.isnan(dirty)
    assert torch.equal(nan, expect) and torch.equal(same, lse)
    assert torch.equal(dirty[~nan], out[~nan])
