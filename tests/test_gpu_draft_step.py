"""The operators of a verification step one after the other, as they would be used: a norm to
8 bits, the projections, the preamble that writes K and V into the cache, attention of chains
and trees of drafted tokens, a norm with the residual, logits, the drafts' log probabilities
and their gradient.  Each operator's outputs are compared with 64 bits from what it read; a
captured step must give the same bits with new data."""
import numpy as np
import pytest
import torch

import tests.attention_ref as attention
import tests.test_gpu_rmsnorm_quant as norms
import tests.test_gpu_token_logprobs as logprobs
from tests.test_gpu_back_to_back import both_ways

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


class Step:
    """Weights, a cache with `context` tokens of each sequence, and buffers for a step."""

    def __init__(self, nr, fmt, dtype, dim, heads, group, context, drafts, page=16, vocab=2003, seed=0):
        self.nr, self.dtype, self.dim, self.heads, self.hq = nr, dtype, dim, heads, heads * group
        rng = np.random.default_rng(seed)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        n, hidden = sum(drafts), 128 * heads * group
        self.lens = np.array([c + d for c, d in zip(context, drafts)], np.int32)
        need = [-(-int(v) // page) for v in self.lens]
        order = rng.permutation(sum(need) + 2).astype(np.int32)
        self.table = np.full((len(need), max(need)), -1, np.int32)
        starts = np.concatenate([[0], np.cumsum(need)])
        for s, k in enumerate(need):
            self.table[s, :k] = order[starts[s]:starts[s] + k]
        self.cu = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
        self.tree = np.concatenate([attention.tree_masks(rng, d, 2) for d in drafts])
        at = lambda s, p: int(self.table[s, p // page]) * page + p % page  # noqa: E731
        slots = [at(s, c + j) for s, (c, d) in enumerate(zip(context, drafts)) for j in range(d)]
        dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
        self.slots = torch.tensor(slots, device="cuda")
        # a drafted token's position is its depth behind the context
        depth = [sum(bin(int(w) & 0xFFFFFFFF).count("1") for w in row) - 1 for row in self.tree]
        self.positions = torch.tensor([c + depth[self.cu[s] + j] for s, (c, d) in
                                       enumerate(zip(context, drafts)) for j in range(d)],
                                      dtype=torch.int32, device="cuda")
        self.d_table, self.d_lens, self.d_cu, self.d_tree = map(dev, (self.table, self.lens, self.cu,
                                                                      self.tree))
        self.parts = attention.to_gpu(attention.make_cache(rng, sum(need) + 2, page, heads, dim, fmt))
        make = lambda *s: torch.randn(*s, generator=self.gen, device="cuda")  # noqa: E731
        self.w1, self.w2 = ((1 + 0.1 * make(hidden)).to(dtype) for _ in range(2))
        self.wq, self.wk = ((1 + 0.1 * make(dim)) for _ in range(2))
        self.w_qkv = (make(hidden, (self.hq + 2 * heads) * dim) / hidden ** 0.5).to(dtype)
        self.w_o = (make(self.hq * dim, hidden) / (self.hq * dim) ** 0.5).to(dtype)
        self.w_v = (3 * make(hidden, vocab) / hidden ** 0.5).to(dtype)
        self.x = make(n, hidden).to(dtype)
        self.tokens = torch.randint(-1, vocab, (n,), generator=self.gen, device="cuda")
        self.g, self.h = make(n), make(n)

    def held(self, codes, scales):
        return (codes.view(torch.float8_e4m3fn).to(f32) * scales[:, None]).to(self.dtype)

    def run(self, x):
        nr, r = self.nr, {"residual": x.clone()}
        r["c1"], r["s1"] = nr.rmsnorm_quant(x, self.w1, scales="row")
        qkv = (self.held(r["c1"], r["s1"]) @ self.w_qkv).view(x.shape[0], -1, self.dim)
        q, k, v = qkv.split([self.hq, self.heads, self.heads], 1)
        r["q"] = nr.qk_norm_rope_cache(q, k, v, self.wq, self.wk, self.positions, self.slots,
                                       *self.parts)
        r["out"], r["lse"] = nr.cache_attention(r["q"], *self.parts, self.d_table, self.d_lens,
                                                cu_q=self.d_cu, tree=self.d_tree, return_lse=True)
        r["y"] = r["out"].flatten(1) @ self.w_o
        r["before"] = r["residual"].clone()
        r["c2"], r["s2"] = nr.rmsnorm_quant(r["y"], self.w2, residual=r["residual"], scales="row")
        r["logits"] = self.held(r["c2"], r["s2"]) @ self.w_v
        r["p"] = nr.token_logprobs(r["logits"], self.tokens, top=4)
        r["dlogits"] = nr.token_logprobs_backward(self.g, self.h, r["logits"], self.tokens,
                                                  r["p"].lse, r["p"].entropy)
        return r

    def check(self, x, r):
        n, _ = norms.normed(x.cpu(), self.w1.cpu(), None, 1e-6, False)
        norms.check(r["c1"], r["s1"], n, "row")
        want = attention.attention(r["q"].double().cpu().numpy(), [p.cpu().numpy() for p in self.parts],
                                   self.table, self.lens, self.cu, self.tree, self.dim ** -0.5,
                                   self.dtype == f32)
        attention.check(r["out"], r["lse"], want, self.dtype)
        n, new = norms.normed(r["y"].cpu(), self.w2.cpu(), r["before"].cpu(), 1e-6, False)
        norms.check(r["c2"], r["s2"], n, "row")
        assert torch.equal(r["residual"].cpu(), new)
        logprobs.check(r["p"], r["logits"], self.tokens, 4, 1.0)
        logprobs.check_grad(r["dlogits"], self.g, self.h, r["logits"], self.tokens, r["p"], 1.0)


SIZES = [  # head dimension, cache heads, query heads of each, contexts, drafts
    (128, 2, 4, [130, 0, 37], [13, 1, 5]),
    (64, 3, 1, [300], [1]),
    (128, 1, 2, [5, 1000, 64, 0, 77], [1, 1, 1, 1, 1]),
    (256, 1, 2, [40, 9], [7, 33]),
    (64, 2, 8, [700, 20], [61, 40]),
]


@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("dim,heads,group,context,drafts", SIZES)
def test_step(nr, dim, heads, group, context, drafts, fmt, dtype):
    s = Step(nr, fmt, dtype, dim, heads, group, context, drafts)
    s.check(s.x, s.run(s.x))


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("size", [0, 4])
def test_captured_step(nr, fmt, size):
    """Replayed with other data; beside it the same step run eagerly on another stream."""
    s = Step(nr, fmt, bf, *SIZES[size])
    kept = [p.clone() for p in s.parts]
    x = s.x.clone()
    s.run(x)  # first calls outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = s.run(x)
    for turn in range(3):
        x.copy_(torch.randn(x.shape, generator=s.gen, device="cuda") * (1 + turn))
        for p, k in zip(s.parts, kept):
            p.copy_(k)
        graph.replay()
        torch.cuda.synchronize()
        s.check(x, r)
        got = [r[k].clone() for k in ("c1", "out", "lse", "c2", "dlogits")] + [r["p"].logprob.clone()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            e = s.run(x)
        side.synchronize()
        again = [e[k] for k in ("c1", "out", "lse", "c2", "dlogits")] + [e["p"].logprob]
        assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("fmt,dtype,size", [("fp8", bf, 0), ("mxfp4", bf, 2), ("fp8", f32, 3),
                                            ("fp8", bf, 4)])
def test_steps_back_to_back(nr, fmt, dtype, size):
    """The framework's kernels alone, with no other between them and new data every call: written
    into the same slots, attended, scored and differentiated in the same buffers."""
    s = Step(nr, fmt, dtype, *SIZES[size])
    n = s.x.shape[0]
    make = lambda *d: torch.randn(8, n, *d, generator=s.gen, device="cuda").to(dtype)  # noqa: E731
    q, k, v, x = make(s.hq, s.dim), make(s.heads, s.dim), make(s.heads, s.dim), make(s.hq * s.dim)
    w = torch.ones(s.hq * s.dim, dtype=dtype, device="cuda")
    outs = [[torch.zeros_like(q[0]), torch.zeros_like(x[0]),
             torch.zeros(n, s.hq * s.dim, dtype=torch.uint8, device="cuda"),
             torch.zeros(n, device="cuda")] for _ in range(8)]
    normed = torch.zeros_like(q[0])

    def run(i):
        nr.qk_norm_rope_cache(q[i], k[i], v[i], s.wq, s.wk, s.positions, s.slots, *s.parts,
                              q_out=normed)
        nr.cache_attention(normed, *s.parts, s.d_table, s.d_lens, cu_q=s.d_cu, tree=s.d_tree,
                           out=outs[i][0])
        rows = outs[i][0].flatten(1)
        nr.rmsnorm_quant(rows, w, codes=outs[i][2], scales_out=outs[i][3])
        p = nr.token_logprobs(rows, s.tokens)
        nr.token_logprobs_backward(s.g, s.h, rows, s.tokens, p.lse, p.entropy, dlogits=outs[i][1])

    def spoil():
        page = s.parts[0].shape[1]
        at = s.slots // page, s.slots % page
        for p in s.parts:
            p[at] = 0x7E if p.dtype == torch.uint8 else float("nan")
        normed.fill_(float("nan"))

    both_ways(run, spoil, outs)
