"""Workloads of attention over the quantised cache, of the norm with an 8-bit output, and of token log probabilities, with
their plain forms.

A case is one call on inputs made from a seed.  With `own` false, run() computes the plain form from elementary
torch operations; with `own` true it calls the package.  exact() computes the same outputs in 64 bits from the
definitions.

    kind     what it is
    attend   attention of one token, a chain or a tree of drafted tokens over sequences of the paged cache
    quant    residual addition + RMSNorm with an e4m3 output and scales made from the data
    score    log probabilities of given tokens, entropy and the top alternatives of rows of logits
    grad     the gradient of the log probabilities and the entropy with respect to the logits
"""
import math

import torch

own = False

F32_MAX = 3.4028234663852886e38
TINY = 2.0 ** -100  # smallest magnitude that a group is scaled by
F8 = torch.float8_e4m3fn
F8_SCALE = torch.float8_e8m0fnu


def listed():
    return [
        # one chat, one new token, grouped-query: latency
        {"name": "attend_one", "kind": "attend", "seqs": 1, "tokens": 1501, "draft": 1, "tree": False, "qheads": 32,
         "heads": 8, "dim": 128, "page": 16, "fmt": "fp8", "dtype": "bf16"},
        # one decode step of a batch of chats of very different lengths
        {"name": "attend_decode", "kind": "attend", "seqs": 48, "tokens": 400009, "draft": 1, "tree": False,
         "qheads": 32, "heads": 8, "dim": 128, "page": 64, "fmt": "fp8", "dtype": "bf16"},
        # trees of drafted tokens verified over longer contexts
        {"name": "attend_tree", "kind": "attend", "seqs": 6, "tokens": 60013, "draft": 61, "tree": True, "qheads": 32,
         "heads": 8, "dim": 128, "page": 64, "fmt": "fp8", "dtype": "bf16"},
        # short chains of drafted tokens over a 4-bit cache
        {"name": "attend_chain_4bit", "kind": "attend", "seqs": 29, "tokens": 150001, "draft": 5, "tree": False,
         "qheads": 24, "heads": 6, "dim": 128, "page": 16, "fmt": "mxfp4", "dtype": "bf16"},
        # a small tree in 32 bits, wide heads
        {"name": "attend_tree_f32", "kind": "attend", "seqs": 3, "tokens": 9001, "draft": 11, "tree": True, "qheads": 8,
         "heads": 4, "dim": 256, "page": 8, "fmt": "fp8", "dtype": "f32"},
        # one decode step: the norm in front of an 8-bit product, a scale a token
        {"name": "quant_decode", "kind": "quant", "rows": 8, "hidden": 5120, "scales": "row", "residual": True,
         "dtype": "bf16"},
        # a prefill batch, a scale for each 128 values
        {"name": "quant_prefill", "kind": "quant", "rows": 8192, "hidden": 5120, "scales": "group", "residual": True,
         "dtype": "bf16"},
        # an odd number of rows in 32 bits, microscaled, no residual
        {"name": "quant_mx_f32", "kind": "quant", "rows": 2049, "hidden": 4096, "scales": "mx", "residual": False,
         "dtype": "f32"},
        # verifying a few drafted tokens, with alternatives to show
        {"name": "score_decode", "kind": "score", "rows": 5, "vocab": 131072, "top": 20, "temperature": 1.0,
         "dtype": "bf16"},
        # scoring a long prompt over an odd vocabulary
        {"name": "score_prompt", "kind": "score", "rows": 4093, "vocab": 151551, "top": 5, "temperature": 0.7,
         "dtype": "bf16"},
        # training: a small batch in 32 bits, and a large one
        {"name": "grad_small_f32", "kind": "grad", "rows": 96, "vocab": 32003, "entropy": True, "temperature": 1.0,
         "dtype": "f32"},
        {"name": "grad_large", "kind": "grad", "rows": 4096, "vocab": 131072, "entropy": True, "temperature": 1.0,
         "dtype": "bf16"},
    ]


def draw(rng):
    def between(lo, hi):  # even over the logarithm
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["attend", "attend", "attend", "quant", "score", "grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "attend":
        heads, dim = rng.choice([1, 2, 4, 6, 8, 12]), rng.choice([64, 128, 128, 256])
        group = rng.choice([1, 2, 3, 4, 5, 8])
        draft = rng.choice([1, 1, between(2, 100)])
        # sequences of a batch share no tokens; the pairs of query and key stay below the listed tree's
        seqs = between(1, 150)
        most = min(160 * 1024 * 1024 // (heads * dim), 100 * 1000 * 1000 // (draft * heads * group))
        tokens = seqs * draft + between(1, max(2, most - seqs * draft))
        return {"kind": kind, "seqs": seqs, "tokens": tokens, "draft": draft,
                "tree": draft > 1 and rng.random() < 0.6, "qheads": heads * group, "heads": heads, "dim": dim,
                "page": rng.choice([1, 8, 16, 32, 48, 64, 128]), "fmt": rng.choice(["fp8", "fp8", "mxfp4"]),
                "dtype": dtype}
    if kind == "quant":
        scales = rng.choice(["row", "group", "mx"])
        hidden = {"row": 8, "group": 128, "mx": 32}[scales]
        hidden *= max(1, between(128, 16384) // hidden)
        return {"kind": kind, "rows": between(1, 40 * 1024 * 1024 // hidden), "hidden": hidden, "scales": scales,
                "residual": rng.random() < 0.7, "dtype": dtype}
    vocab = between(1000, 262144)
    rows = between(1, 500 * 1000 * 1000 // vocab // (2 if dtype == "f32" else 1))
    case = {"kind": kind, "rows": rows, "vocab": vocab, "temperature": rng.choice([1.0, 1.0, 0.6, 1.3]),
            "dtype": dtype}
    if kind == "score":
        case["top"] = rng.choice([0, 1, 5, 20, 32])
    else:
        case["entropy"] = rng.random() < 0.6
    return case


def type_of(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _drafts(case):
    """Drafted tokens of each sequence: not all drafts have the same number."""
    return [max(1, case["draft"] - 2 * (i % 4)) for i in range(case["seqs"])]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = {"case": case}
    kind, dt = case["kind"], type_of(case["dtype"])
    if kind == "quant":
        rows, hidden = case["rows"], case["hidden"]
        width = torch.exp(0.7 * normal(hidden))  # some channels are wide
        s["x"] = (normal(rows, hidden) * width).to(dt)
        s["w"] = (1 + 0.1 * normal(hidden)).to(dt)
        s["residual"] = (normal(rows, hidden) * width).to(dt) if case["residual"] else None
        return s
    if kind in ("score", "grad"):
        rows, vocab = case["rows"], case["vocab"]
        # rows that are sure of a few tokens, and rows that are not
        sure = 1 + 3 * torch.rand(rows, 1, generator=g, device=dev)
        z = normal(rows, vocab)
        s["logits"] = z.mul_(sure).to(dt)
        tokens = torch.randint(0, vocab, (rows,), generator=g, device=dev)
        best = s["logits"].argmax(1)
        s["tokens"] = torch.where(torch.rand(rows, generator=g, device=dev) < 0.6, best, tokens)
        s["tokens"][::7] = -1 if rows > 7 else s["tokens"][::7]  # padding
        if kind == "grad":
            s["dlogprob"] = normal(rows) / rows
            s["dentropy"] = 0.01 * normal(rows) / rows if case["entropy"] else None
            s["lse"], s["entropy"] = _stats(s["logits"], case["temperature"])
        return s
    heads, dim, page = case["heads"], case["dim"], case["page"]
    drafts = torch.tensor(_drafts(case), device=dev)
    # random cuts: some sequences are short, some long
    spare = case["tokens"] - int(drafts.sum())
    cuts = torch.randint(0, spare + 1, (case["seqs"] - 1,), generator=g, device=dev).sort().values
    cuts = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), spare)])
    lens = cuts[1:] - cuts[:-1] + drafts
    need = [-(-v // page) for v in lens.tolist()]
    blocks = sum(need) + max(4, sum(need) // 8)  # the cache is not full
    order = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(len(need), max(need), dtype=torch.int32, device=dev)
    at = 0
    for i, v in enumerate(need):
        table[i, :v] = order[at:at + v]
        at += v
    s["table"], s["lens"] = table, lens.to(torch.int32)
    s["cu"] = torch.cat([drafts.new_zeros(1), drafts.cumsum(0)]).to(torch.int32)
    for name in ("k", "v"):
        if case["fmt"] == "fp8":
            x = normal(blocks, page, heads, dim)
            if name == "k":
                x *= torch.exp(0.5 * normal(heads, dim))  # K has a few wide channels
            scale = x.abs().amax(-1) / 448
            s[name + "_cache"] = (x / scale[..., None]).clamp_(-448, 448).to(F8).view(torch.uint8)
            s[name + "_scale"] = scale
        else:
            s[name + "_cache"] = torch.randint(0, 256, (blocks, page, heads, dim // 2), generator=g, device=dev,
                                               dtype=torch.uint8)
            s[name + "_scale"] = torch.randint(124, 127, (blocks, page, heads, dim // 32), generator=g, device=dev,
                                               dtype=torch.uint8)
    rows = sum(_drafts(case))
    s["q"] = (1.5 * normal(rows, case["qheads"], dim)).to(dt)
    s["tree"] = None
    if case["tree"]:
        words = -(-case["draft"] // 32)
        r = torch.Generator().manual_seed(seed)
        flat = []
        for n in _drafts(case):
            seen = []  # a drafted token sees its ancestors and itself
            for j in range(n):
                parent = int(torch.randint(-1, j, (1,), generator=r)) if j else -1
                seen.append((seen[parent] if parent >= 0 else 0) | 1 << j)
            flat += seen
        flat = [[(v >> 32 * k & 0xFFFFFFFF) - (v >> 32 * k + 31 & 1 and 1 << 32) for k in range(words)] for v in flat]
        s["tree"] = torch.tensor(flat, dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------------------
# plain forms, in 32 bits
# ---------------------------------------------------------------------------
def _load(s, name):
    """The pages of every sequence, widened: [seqs, width * page, heads, dim]."""
    cache, scale = s[name + "_cache"], s[name + "_scale"]
    at = s["table"].long()
    codes, sc = cache[at].flatten(1, 2), scale[at].flatten(1, 2)
    if sc.dtype == torch.float32:
        return codes.view(F8).float() * sc[..., None]
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = grid[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(sc.float() - 127)[..., None]).flatten(-2)


def _visible(s, draft):
    """[seqs, draft, positions]: what each query sees."""
    cu, lens = s["cu"].long(), s["lens"].long()
    t, p = torch.arange(draft, device=cu.device), torch.arange(s["table"].shape[1] * s["case"]["page"],
                                                                device=cu.device)
    own_tokens = (cu[1:] - cu[:-1])[:, None, None]
    j = p - (lens[:, None, None] - own_tokens)  # [seqs, 1, positions]
    if s["tree"] is None:
        drafted = j <= t[:, None]
    else:
        row = (cu[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)
        bits = (s["tree"][row][..., None] >> torch.arange(32, device=cu.device, dtype=torch.int32) & 1).flatten(-2)
        inside = ((j >= 0) & (j < bits.shape[-1])).expand(-1, draft, -1)
        drafted = bits.gather(-1, j.clamp(0, bits.shape[-1] - 1).expand(-1, draft, -1)).bool() & inside
    return (j < 0) | (drafted & (j < own_tokens))


def _attend(s):
    case = s["case"]
    heads, dim, draft, cu = case["heads"], case["dim"], case["draft"], s["cu"].long()
    group = case["qheads"] // heads
    k, v = _load(s, "k").transpose(1, 2), _load(s, "v").transpose(1, 2)  # [seqs, heads, positions, dim]
    row = (cu[:-1, None] + torch.arange(draft, device=cu.device)).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[row].unflatten(2, (heads, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = q @ k.transpose(-1, -2) * dim ** -0.5  # [seqs, heads, group * draft, positions]
    score = score.unflatten(2, (group, draft)).masked_fill_(~_visible(s, draft)[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(top == -math.inf, 0., top))
    total = weight.sum(-1, keepdim=True)
    out = (weight / total).flatten(2, 3) @ v
    out = torch.where(total.flatten(2, 3) > 0, out, 0.).unflatten(2, (group, draft))
    lse = (top + torch.log(total)).squeeze(-1)
    rows = torch.arange(s["q"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu[1:], rows, right=True)
    t = rows - cu[seq]
    return {"out": out.permute(0, 3, 1, 2, 4).flatten(2, 3)[seq, t].to(s["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2).flatten(2, 3)[seq, t]}


def _quant(s):
    case, x = s["case"], s["x"].float()
    if case["residual"]:
        x = (x + s["residual"].float()).to(s["x"].dtype)
        s["residual"].copy_(x)
        x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * s["w"].float()
    y = y.unflatten(1, (-1, {"row": case["hidden"], "group": 128, "mx": 32}[case["scales"]]))
    a = y.abs().amax(-1, keepdim=True).clamp(TINY, F32_MAX)
    if case["scales"] == "mx":
        m, e = torch.frexp(a)  # a = m 2^e, m in [1/2, 1)
        e = e - 9 + (m > 0.875)  # the least power of two with a / 2^e <= 448
        codes, scale = torch.ldexp(y, -e), (e + 127).to(torch.uint8).view(F8_SCALE)
    else:
        top = torch.full_like(a, 448)  # a tensor: divided by, each quotient is rounded once
        codes, scale = y * (top / a), a / top
    codes = codes.clamp(-448, 448).to(F8).flatten(1)
    scale = scale.squeeze(-1)
    return {"codes": codes, "scales": scale.squeeze(-1) if case["scales"] == "row" else scale,
            "residual": s["residual"]}


def _stats(logits, temperature):
    z = logits.float() / temperature
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(-1)
    log = torch.log(total)
    return top.squeeze(-1) + log, log - (e.mul_(z.sub_(top))).sum(-1) / total


def _score(s):
    case, logits = s["case"], s["logits"]
    rows, vocab = logits.shape
    lse, entropy = _stats(logits, case["temperature"])
    inside = (s["tokens"] >= 0) & (s["tokens"] < vocab)
    z = logits.gather(1, s["tokens"].clamp(0, vocab - 1)[:, None]).squeeze(1).float() / case["temperature"]
    out = {"logprob": torch.where(inside, z - lse, 0.), "entropy": entropy, "lse": lse}
    if case["top"]:
        # the order of the values as whole numbers, equal values by their index
        bits = (logits.float() + 0.).view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) << 32
        key -= torch.arange(vocab, device=key.device)
        ids = key.topk(case["top"], dim=1).values.neg_() & 0xFFFFFFFF
        out["top_ids"] = ids
        out["top_logprob"] = logits.gather(1, ids).float() / case["temperature"] - lse[:, None]
    return out


def _grad(s):
    case, logits = s["case"], s["logits"]
    logp = logits.float() / case["temperature"] - s["lse"][:, None]
    p = torch.exp(logp)
    inside = (s["tokens"] >= 0) & (s["tokens"] < logits.shape[1])
    d = torch.where(inside, s["dlogprob"], 0.)
    dz = p * -d[:, None]
    if case["entropy"]:
        dz -= s["dentropy"][:, None] * p * (logp + s["entropy"][:, None])
    dz.scatter_add_(1, s["tokens"].clamp(0, logits.shape[1] - 1)[:, None], d[:, None])
    return {"dlogits": (dz / case["temperature"]).to(logits.dtype)}


def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        import normalisation_rope_transformers_gb300 as nr

        if kind == "attend":
            out, lse = nr.cache_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                          s["lens"], cu_q=s["cu"] if case["draft"] > 1 else None, tree=s["tree"],
                                          scale=case["dim"] ** -0.5, return_lse=True)
            return {"out": out, "lse": lse}
        if kind == "quant":
            codes, scales = nr.rmsnorm_quant(s["x"], s["w"], residual=s["residual"], eps=1e-6, scales=case["scales"])
            return {"codes": codes.view(F8), "scales": scales.view(F8_SCALE) if case["scales"] == "mx" else scales,
                    "residual": s["residual"]}
        if kind == "score":
            r = nr.token_logprobs(s["logits"], s["tokens"], top=case["top"], temperature=case["temperature"])
            out = {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse}
            return {**out, "top_logprob": r.top_logprob, "top_ids": r.top_ids} if case["top"] else out
        return {"dlogits": nr.token_logprobs_backward(s["dlogprob"], s["dentropy"], s["logits"], s["tokens"],
                                                      s["lse"], s["entropy"], temperature=case["temperature"])}
    return {"attend": _attend, "quant": _quant, "score": _score, "grad": _grad}[kind](s)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    kind = case["kind"]
    if kind == "attend":
        held = case["heads"] * (2 * case["dim"] + 8 if case["fmt"] == "fp8" else case["dim"] + case["dim"] // 16)
        rows, q = sum(_drafts(case)), case["qheads"] * case["dim"]
        return {"bytes": case["tokens"] * held + rows * (2 * q * es + 4 * case["qheads"]),
                "flops": 4 * q * rows * case["tokens"] / case["seqs"]}
    if kind == "quant":
        n = case["rows"] * case["hidden"]
        scales = {"row": 4 * case["rows"], "group": n // 32, "mx": n // 32}[case["scales"]]
        return {"bytes": n * (es * (3 if case["residual"] else 1) + 1) + scales, "flops": 8 * n}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * es * (1 if kind == "score" else 2) + 32 * case["rows"], "flops": 6 * n}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _nearest(v, grid):
    """The values of the sorted `grid` nearest to |v| (ties to the even place), with v's sign; past the end, the
    end."""
    mag = v.abs()
    hi = torch.searchsorted(grid, mag).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    to_lo, to_hi = mag - grid[lo], grid[hi] - mag
    at = torch.where((to_lo < to_hi) | ((to_lo == to_hi) & (lo % 2 == 0)), lo, hi)
    return torch.copysign(grid[at], v)


def exact(case, seed):
    s = prepare(case, seed)
    kind, d, dev = case["kind"], torch.float64, torch.device("cuda")
    if kind == "quant":
        v, parts = s["x"].double(), {"row": 1, "group": case["hidden"] // 128, "mx": case["hidden"] // 32}
        if case["residual"]:
            v = (v + s["residual"].double()).to(s["x"].dtype)
            s["residual"] = v
            v = v.double()
        v = v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * s["w"].double()
        top = v.view(case["rows"], parts[case["scales"]], -1).abs().amax(2).clamp(TINY, F32_MAX)
        unit = 2.0 ** torch.ceil(torch.log2(top / 448)) if case["scales"] == "mx" else top / 448
        steps = [m * 2.0 ** -9 for m in range(8)]
        steps += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
        grid = torch.tensor(steps[:-1], dtype=d, device=dev)  # up to 448: the last place is the NaN's
        v = v.view(case["rows"], parts[case["scales"]], -1)
        codes = torch.cat([_nearest(x / u[..., None], grid) for x, u in zip(v.split(1024), unit.split(1024))])
        return {"codes": codes.flatten(1), "scales": unit[:, 0] if case["scales"] == "row" else unit,
                "residual": s["residual"]}
    if kind in ("score", "grad"):
        parts = {}
        for i in range(0, case["rows"], 256):  # some rows at a time, to hold less
            z = s["logits"][i:i + 256].double() / case["temperature"]
            tokens = s["tokens"][i:i + 256]
            pad = (tokens < 0) | (tokens >= case["vocab"])
            place = torch.where(pad, 0, tokens)[:, None]
            if kind == "score":
                logp = torch.log_softmax(z, 1)
                p = logp.exp()
                got = {"logprob": logp.gather(1, place)[:, 0].masked_fill(pad, 0),
                       "entropy": -torch.where(p > 0, p * logp, 0).sum(1), "lse": torch.logsumexp(z, 1)}
                if case["top"]:
                    got["top_logprob"] = logp.topk(case["top"], dim=1).values
            else:
                logp = z - s["lse"][i:i + 256, None].double()
                p = logp.exp()
                up = s["dlogprob"][i:i + 256].double().masked_fill(pad, 0)[:, None]
                got = -up * p
                if case["entropy"]:
                    h = s["entropy"][i:i + 256, None].double()
                    got -= s["dentropy"][i:i + 256, None].double() * p * (logp + h)
                got[torch.arange(len(tokens), device=dev), place[:, 0]] += up[:, 0]
                got = {"dlogits": got / case["temperature"]}
            for k, v in got.items():
                parts.setdefault(k, []).append(v)
        res = {k: torch.cat(v) for k, v in parts.items()}
        return {**res, "top_ids": None} if case.get("top") else res
    page, dim, group = case["page"], case["dim"], case["qheads"] // case["heads"]
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=d, device=dev)
    outs, lses, first = [], [], 0
    for i, length in enumerate(s["lens"].tolist()):
        pages = s["table"][i, :-(-length // page)].long()
        wide = []
        for name in ("k", "v"):
            codes = s[name + "_cache"][pages].flatten(0, 1)[:length]
            sc = s[name + "_scale"][pages].flatten(0, 1)[:length]
            if case["fmt"] == "fp8":
                wide.append(codes.view(F8).double() * sc.double()[..., None])
            else:
                pair = torch.stack([codes % 16, codes // 16], -1).flatten(-2).long()
                v = torch.where(pair > 7, -grid[pair % 8], grid[pair % 8])
                wide.append((v.unflatten(-1, (-1, 32)) * 2.0 ** (sc.double()[..., None] - 127)).flatten(-2))
        n = _drafts(case)[i]
        seen = torch.ones(n, length, dtype=torch.bool, device=dev)
        for t in range(n):
            bits = ((1 << t + 1) - 1) if s["tree"] is None else sum(
                (w & 0xFFFFFFFF) << 32 * k for k, w in enumerate(s["tree"][first + t].tolist()))
            seen[t, length - n:] = torch.tensor([bool(bits >> j & 1) for j in range(n)], device=dev)
        q = s["q"][first:first + n].double()
        o, z = torch.empty_like(q), torch.empty(n, case["qheads"], dtype=d, device=dev)
        for h in range(case["qheads"]):
            k, v = (x[:, h // group] for x in wide)
            score = (q[:, h] @ k.T / math.sqrt(dim)).masked_fill(~seen, -math.inf)
            z[:, h] = torch.logsumexp(score, 1)
            o[:, h] = torch.softmax(score, 1) @ v
        outs.append(o)
        lses.append(z)
        first += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
