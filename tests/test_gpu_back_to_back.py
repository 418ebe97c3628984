"""Calls back to back on the same memory, with no other kernel between them and new
data every call: each kernel is scheduled while the one before it still runs, and
must see what that one wrote.  Wanted is, bit for bit, what the same calls give one
at a time, with the device waited for after each and the shared memory filled with
NaN before it.  Run eagerly and as one captured graph."""
import ctypes

import pytest
import torch

from tests.test_gpu_kv_cache import make_cache

pytestmark = pytest.mark.gpu
bf = torch.bfloat16
F32, BF16 = 0, 1
CALLS = 8


def both_ways(run, spoil, outs):
    """run(i) for each call: alone, then together, eagerly and from a graph."""
    want = []
    for i in range(CALLS):
        spoil()
        torch.cuda.synchronize()
        run(i)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs[i]])
    assert not torch.equal(want[0][0], want[1][0])  # the data does change
    clear = [t for o in outs for t in o]

    def check(how):
        torch.cuda.synchronize()
        for i in range(CALLS):
            for j, (a, b) in enumerate(zip(outs[i], want[i])):
                assert torch.equal(a, b), "%s: call %d, output %d" % (how, i, j)
        for t in clear:
            t.zero_()
        spoil()
        torch.cuda.synchronize()

    check("alone")
    for _ in range(3):
        for i in range(CALLS):
            run(i)
        check("eager")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(CALLS):
            run(i)
    for _ in range(5):
        graph.replay()
        check("graph")


class Norms:
    """CALLS inputs of one size; one workspace, mean and rstd for all of them."""

    def __init__(self, nr, n, s, c, g, dtype):
        self.nr, self.size, self.dtype = nr, (n, s, c, g), dtype
        gen = torch.Generator(device="cuda").manual_seed(c)
        self.x, self.dy = [], []
        for i in range(CALLS):  # each of a level and width of its own
            t = torch.randn(n, s, c, generator=gen, device="cuda") * (1 + i) + 3 * i - 9
            self.x.append(t.to(dtype))
            self.dy.append((torch.randn(n, s, c, generator=gen, device="cuda") + i).to(dtype))
        self.w = torch.randn(c, generator=gen, device="cuda")
        self.b = torch.randn(c, generator=gen, device="cuda")
        self.mean, self.rstd = (torch.empty(n, g, device="cuda") for _ in range(2))
        self.out = [torch.zeros_like(t) for t in self.x]
        self.dx = [torch.zeros_like(t) for t in self.x]
        self.dw, self.db = ([torch.zeros(c, device="cuda") for _ in range(CALLS)] for _ in range(2))
        self.code = BF16 if dtype == bf else F32
        self.ws = [self.workspace(back) for back in (0, 1)]

    def workspace(self, back):
        need = ctypes.c_int64()
        assert self.nr.lib.nr_group_norm_workspace(*self.size, back, self.code,
                                                   ctypes.byref(need)) == 0
        return torch.empty(need.value, dtype=torch.uint8, device="cuda")

    def spoil(self):
        for t in (self.mean, self.rstd):
            t.fill_(float("nan"))
        for w in self.ws:
            w.fill_(0xFF)  # NaN in every float

    def stream(self):
        return torch.cuda.current_stream().cuda_stream

    def forward(self, i):
        assert self.nr.lib.nr_group_norm(
            self.out[i].data_ptr(), self.mean.data_ptr(), self.rstd.data_ptr(),
            self.x[i].data_ptr(), self.w.data_ptr(), self.b.data_ptr(), F32, *self.size, 1e-5, 1,
            self.code, self.ws[0].data_ptr() if self.ws[0].numel() else None, self.ws[0].numel(),
            self.stream()) == 0

    def backward(self, i):
        assert self.nr.lib.nr_group_norm_backward(
            self.dx[i].data_ptr(), self.dw[i].data_ptr(), self.db[i].data_ptr(),
            self.dy[i].data_ptr(), self.x[i].data_ptr(), self.mean.data_ptr(), self.rstd.data_ptr(),
            self.w.data_ptr(), self.b.data_ptr(), F32, *self.size, 1, self.code,
            self.ws[1].data_ptr() if self.ws[1].numel() else None, self.ws[1].numel(),
            self.stream()) == 0


# two launches of a few blocks, of a wave of them, with groups across tiles; and one launch
NORMS = [(1, 26229, 48, 3), (3, 7161, 320, 32), (2, 300, 4104, 3), (160, 600, 128, 4),
         (4, 1024, 640, 32), (2, 256, 1280, 32)]


@pytest.mark.parametrize("n,s,c,g", NORMS)
@pytest.mark.parametrize("dtype", [bf, torch.float32])
def test_group_norms(nr, n, s, c, g, dtype):
    t = Norms(nr, n, s, c, g, dtype)
    both_ways(t.forward, t.spoil, [[o] for o in t.out])


@pytest.mark.parametrize("n,s,c,g", NORMS)
@pytest.mark.parametrize("dtype", [bf, torch.float32])
def test_group_norms_with_their_gradients(nr, n, s, c, g, dtype):
    """The gradient reads the mean and rstd that the call before it wrote, in the
    place where the next call writes its own."""
    t = Norms(nr, n, s, c, g, dtype)

    def run(i):
        t.forward(i)
        t.backward(i)

    both_ways(run, t.spoil, list(map(list, zip(t.out, t.dx, t.dw, t.db))))


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("tokens,heads,page", [(3, 2, 4), (700, 8, 16), (6000, 8, 64)])
@pytest.mark.parametrize("fused", [False, True])
def test_cache_turns(nr, fmt, tokens, heads, page, fused):
    """Written and read back in turn, in the same slots."""
    dim, blocks = 128, -(-tokens // page) + 1
    parts = make_cache(fmt, blocks, page, heads, dim)
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    shape = (CALLS, tokens, heads, dim)
    scale = torch.exp2(torch.arange(CALLS, device="cuda") * 3.0 - 9)[:, None, None, None]
    k = (torch.randn(shape, generator=gen, device="cuda") * scale).to(bf)
    v = (torch.randn(shape, generator=gen, device="cuda") / scale).to(bf)
    slots = torch.randperm(blocks * page, generator=gen, device="cuda")[:tokens].sort().values
    table = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
    cu = torch.tensor([0, blocks * page], dtype=torch.int32, device="cuda")
    w, pos = torch.ones(dim, device="cuda"), torch.arange(tokens, dtype=torch.int32, device="cuda")
    outs = [[torch.zeros(blocks * page, heads, dim, dtype=bf, device="cuda") for _ in range(2)] +
            [torch.zeros(tokens, heads, dim, dtype=bf, device="cuda")] for _ in range(CALLS)]

    def run(i):
        if fused:
            nr.qk_norm_rope_cache(v[i], k[i], v[i], w, w, pos, slots, *parts, q_out=outs[i][2])
        else:
            nr.kv_cache_write(k[i], v[i], slots, *parts)
        nr.kv_cache_read(*parts, table, cu, k_out=outs[i][0], v_out=outs[i][1])

    def spoil():
        at = slots // page, slots % page
        for p in parts:
            p[at] = 0x7E if p.dtype == torch.uint8 else float("nan")

    both_ways(run, spoil, outs)
