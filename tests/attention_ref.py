"""Plain attention over a quantised paged cache, in 64 bits, and how far f32 arithmetic with
rounded weights may be from it."""
from __future__ import annotations

import numpy as np
import torch

import tests.cache_ref as ref


def make_cache(rng, blocks, page, heads, dim, fmt):
    """(k codes, v codes, k scales, v scales) as numpy arrays, of normal values."""
    parts = [ref.quant(rng.standard_normal((blocks, page, heads, dim)).astype(np.float32), fmt)
             for _ in range(2)]
    return [parts[0][0], parts[1][0], parts[0][1], parts[1][1]]


def tree_masks(rng, n, words):
    """Words [n, words] int32 of a random tree: each token sees itself and its ancestors."""
    seen = []
    for j in range(n):
        parent = int(rng.integers(-1, j)) if j else -1
        seen.append((seen[parent] if parent >= 0 else 0) | 1 << j)
    return np.array([[v >> 32 * k & 0xFFFFFFFF for k in range(words)] for v in seen],
                    np.uint32).reshape(n, words).view(np.int32)


def sees(length, queries, t, words):
    """Which positions of a sequence query t sees (words: its mask, or None)."""
    out = np.zeros(length, bool)
    for p in range(length):
        j = p - (length - queries)
        if j < 0:
            out[p] = True
        elif words is None:
            out[p] = j <= t
        elif j // 32 < len(words):
            out[p] = bool(int(words[j // 32]) >> (j % 32) & 1)
    return out


def attention(q, parts, table, lens, cu, tree, scale, f32):
    """(out, lse, tolerance of out, tolerance of lse) in 64 bits for q [tokens, heads, dim] (its
    stored values); rows of no sequence are NaN.

    The tolerances count roundings.  u = 2^-24 is f32's half step.  A score is a sum of dim
    exact products (f32 tensors: Q kept to 2^-22) in dim / 16 steps of f32, two units each, and
    is multiplied by two factors: e_s = (dim / 8 + 16) u mag, mag = scale sum |q k| (f32: + 4 * 2^-24 mag).  A
    weight is exp of it (2^-22 of the approximation, and the exponent's own roundings, a few
    units of its size, within e_s) and rounded for the product: 2^-11, or 2^-22 in two parts.
    The sums over n positions: n / 16 steps, two units each, and what joins them.  out is a
    quotient of two such sums, hence everything twice but the weights' last rounding, and is
    rounded itself."""
    codes_k, codes_v, scale_k, scale_v = parts
    with np.errstate(invalid="ignore"):
        k, v = ref.held(codes_k, scale_k), ref.held(codes_v, scale_v)
    blocks, page, heads, dim = k.shape
    tokens, hq, _ = q.shape
    group = hq // heads
    u = 2.0 ** -24
    out = np.full((tokens, hq, dim), np.nan)
    lse, tol, ltol = (np.full(s, np.nan) for s in ((tokens, hq), (tokens, hq, dim), (tokens, hq)))
    for s in range(len(lens)):
        n, first = int(lens[s]), int(cu[s])
        queries = int(cu[s + 1]) - first
        at, ok = [], []
        for p in range(n):
            b = int(table[s, p // page]) if p // page < table.shape[1] else -1
            ok.append(0 <= b < blocks)
            at.append((b if ok[-1] else 0, p % page))
        at = np.array(at, np.int64).reshape(n, 2)
        ks, vs = k[at[:, 0], at[:, 1]], v[at[:, 0], at[:, 1]]  # [n, heads, dim]
        for t in range(queries):
            see = np.array(ok, bool) & sees(n, queries, t, None if tree is None else tree[first + t])
            for h in range(hq):
                r = (first + t, h)
                if not see.any():
                    out[r], lse[r], tol[r], ltol[r] = 0, -np.inf, 0, 0
                    continue
                kk, vv = ks[see, h // group], vs[see, h // group]
                qq = q[r].astype(np.float64)
                score = scale * (kk @ qq)
                mag = float(np.max(np.abs(scale) * (np.abs(kk) @ np.abs(qq))))
                top = score.max()
                w = np.exp(score - top)
                lse[r] = top + np.log(w.sum())
                w /= w.sum()
                out[r] = w @ vv
                e_s = (dim / 8 + 16 + (4 if f32 else 0)) * u * mag
                steps = (2 * n / 16 + 64) * u
                spread = w @ np.abs(vv)
                # What a weight below f16's range loses: its smallest step is 2^-24, so half of it,
                # 2^-25, of weights that are held times 2^7 (many rows) or 2^11 relative to a
                # reference that the largest weight is not below: 2^-32 of the largest.
                floor = len(w) * 2.0 ** -32 * np.abs(vv).max() * w.max()
                mx = 0.0 if scale_k.dtype == np.float32 else 2.0 ** -36
                tol[r] = (spread * ((2.0 ** -22 if f32 else 2.0 ** -11)
                                    + 2 * (e_s + 2.0 ** -21 + steps + mx))
                          + floor + (u if f32 else 2.0 ** -8) * np.abs(out[r]))
                ltol[r] = e_s + 2.0 ** -21 + steps + 4 * u * abs(lse[r])
    return out, lse, tol, ltol


def check(got, lse, want, dtype, what=""):
    w_out, w_lse, tol, ltol = want
    rows = ~np.isnan(w_lse[:, 0]) if w_lse.size else np.zeros(0, bool)
    g = got.double().cpu().numpy()
    off = np.abs(g - w_out)[rows]
    bad = ~(off <= tol[rows] * (1 + 1e-9) + 1e-300)
    assert not bad.any(), "%s: out off by %g, allowed %g" % (what, off[bad].max(), tol[rows][bad].max())
    if lse is not None:
        lg = lse.double().cpu().numpy()[rows]
        same = lg == w_lse[rows]
        with np.errstate(invalid="ignore"):
            assert (same | (np.abs(lg - w_lse[rows]) <= ltol[rows])).all(), what + ": lse"


def to_gpu(parts, wide_blocks=0):
    """The cache's parts on the GPU; wide_blocks: that many bytes between neighbouring blocks."""
    out = []
    for x in parts:
        t = torch.from_numpy(x)
        if wide_blocks:
            size = int(np.prod(x.shape[1:]))
            pad = wide_blocks // x.dtype.itemsize
            buf = torch.zeros(x.shape[0], size + pad, dtype=t.dtype)
            buf[:, :size] = t.reshape(x.shape[0], size)
            big = buf.cuda()
            stride = list(t.stride())
            stride[0] = size + pad
            out.append(torch.as_strided(big, x.shape, stride))
        else:
            out.append(t.cuda())
    return out
