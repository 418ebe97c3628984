"""V scales of any size and sign in attention over the cache: what a row holds for its second product
is relative to the largest weight times V scale, so that a token to which nobody attends costs the
others nothing, however large its V."""
import numpy as np
import pytest
import torch

import tests.attention_ref as ref
import tests.cache_ref as cache_ref
from tests.test_gpu_cache_attention import problem, run

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


def close(got, p, scale, heads_at=slice(None)):
    """Compare with 64 bits (some query heads of each token).  Roundings, u = 2^-24 f32's half step: a score is a sum of dim products in
    dim / 16 steps, two units each, and is multiplied by two factors, so e_p = (dim / 8 + 16) u mag_p with
    mag_p = scale sum |q k_p| (f32 tensors: Q in 22 bits, four units more); its weight has that relative
    error and 2^-21 of the exponential, and is rounded for the product (2^-11, or 2^-22 in two
    parts); sums over n positions take n / 16 steps.  out = N / D with N = sum w v, D = sum w: the errors
    of N, and those of D times out.  What is held for f16, w |s| with s a position's largest scale, is
    2^7.5 or more for its largest, and f16's smallest step 2^-24: half of it is 2^-32.5 of that, times the
    codes.  Weights below 2^-118 of the largest (2^8 behind a reference, 2^-126) may count as nothing."""
    out, lse = (x.double().cpu().numpy() for x in got)
    q, parts, table, lens, cu, tree = (p[k] for k in ("q", "parts", "table", "lens", "cu", "tree"))
    f32 = q.dtype == torch.float32
    q = q.double().numpy()
    k, v = (cache_ref.held(parts[i], parts[2 + i]) for i in range(2))
    s = parts[3].astype(np.float64) if parts[3].dtype == np.float32 else 2.0 ** (parts[3].max(-1) - 127.0)
    _, page, heads, dim = k.shape
    group, u = q.shape[1] // heads, 2.0 ** -24
    for i, n in enumerate(lens):
        at = np.arange(n)
        at = table[i, at // page], at % page
        for t in range(cu[i + 1] - cu[i]):
            see = ref.sees(n, cu[i + 1] - cu[i], t, None if tree is None else tree[cu[i] + t])
            for h in range(q.shape[1])[heads_at]:
                kk, vv, ss = (x[at][see, h // group] for x in (k, v, np.abs(s)))
                qq = q[cu[i] + t, h]
                score = scale * (kk @ qq)
                w = np.exp(score - score.max())
                total = w.sum()
                o = w @ vv / total
                e = (dim / 8 + 16 + (4 if f32 else 0)) * u * abs(scale) * (np.abs(kk) @ np.abs(qq))
                e = e + 2.0 ** -21 + (2 * n / 16 + 64) * u + 2.0 ** -36
                held = e + (2.0 ** -22 if f32 else 2.0 ** -11)
                codes = np.abs(vv) / np.maximum(ss, 1e-300)[:, None]
                tol = ((w * held) @ np.abs(vv) + np.abs(o) * (w * e).sum()) / total
                tol += 2.0 ** -32 * (w * ss).max() * codes.sum(0) / total + 2.0 ** -118 * np.abs(vv).sum(0)
                tol += (u if f32 else 2.0 ** -8) * np.abs(o)
                off = np.abs(out[cu[i] + t, h] - o)
                assert (off <= tol).all(), (i, t, h, (off / tol).max(), off.max(), np.abs(o).max())
                z = score.max() + np.log(total)
                assert abs(lse[cu[i] + t, h] - z) <= (w * e).sum() / total + 4 * u * abs(z), (i, t, h, "lse")


# queries of three sequences and the query heads of a K/V head: few rows, and many
ROWS = {"few": ([3, 2, 1], 2), "many": ([30, 17, 40], 2)}


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("dtype", [bf, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ratio", [20, 26, 32, 40, 60])
def test_large_values_that_nobody_attends_to(nr, ratio, dim, fmt, dtype, rows):
    """One token of each sequence has a score e^-29 (heads of 64) to e^-57 (256) below the others' and V
    2^ratio above theirs: the first of the sequence, one in the middle, the last in front of the new ones."""
    queries, group = ROWS[rows]
    lens = [150, 213, 97]
    p = problem(ratio + dim, lens, queries, 2, group, dim, 16, fmt, dtype)
    p["q"] = p["q"].abs()
    for i, pos in enumerate((0, 100, lens[2] - queries[2] - 1)):
        at = p["table"][i, pos // 16], pos % 16
        p["parts"][0][at] = 0xFE if fmt == "fp8" else 0xFF  # K: -3 everywhere
        p["parts"][2][at] = 3 / 448 if fmt == "fp8" else 126
        if fmt == "fp8":
            p["parts"][3][at] *= 2.0 ** ratio
        else:
            p["parts"][3][at] += ratio
    close(run(nr, p), p, dim ** -0.5)


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("dtype", [bf, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_values_that_grow_and_shrink_along_the_sequence(nr, fmt, dtype, rows):
    """V's scales move by 2^80 along 700 positions, scores by 2^90 the other way and the same way."""
    queries, group = ROWS[rows]
    lens, dim = [700, 650, 500], 64
    for grow in (1, -1):
        for up in (1, -1):
            p = problem(5, lens, queries, 2, group, dim, 16, fmt, dtype)
            p["q"] = torch.ones_like(p["q"])
            for i, n in enumerate(lens):
                pos = np.arange(n)
                at = p["table"][i, pos // 16], pos % 16
                e = (grow * (pos - n / 2) / n * 80).round().astype(int)[:, None]
                size = 0.25 + (pos if up > 0 else n - pos) / n * 8  # K: that in each dimension
                if fmt == "fp8":
                    p["parts"][3][at] *= (2.0 ** e).astype(np.float32)
                    p["parts"][0][at] = 0x7E
                    p["parts"][2][at] = (size / 448)[:, None].astype(np.float32)
                else:
                    p["parts"][3][at] = (p["parts"][3][at] + e[..., None]).astype(np.uint8)
                    p["parts"][0][at] = 0x22  # 1
                    p["parts"][2][at] = (127 + np.floor(np.log2(size)))[:, None, None].astype(np.uint8)
            close(run(nr, p), p, dim ** -0.5)


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("dtype", [bf, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_negative_scales(nr, dim, dtype, rows):
    """FP8 scales are any f32: negative ones turn the sign of what a token holds, as kv_cache_read says."""
    queries, group = ROWS[rows]
    p = problem(dim, [150, 213, 97], queries, 2, group, dim, 16, "fp8", dtype)
    rng = np.random.default_rng(1)
    for i in (2, 3):
        p["parts"][i] *= rng.choice([-1, 1], p["parts"][i].shape).astype(np.float32)
    close(run(nr, p), p, dim ** -0.5)
    p["parts"][3] = -np.abs(p["parts"][3])
    close(run(nr, p), p, dim ** -0.5)


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("dtype", [bf, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("exponent", [-108, -100, 100, 119, 125, 126, 127])
def test_scales_near_the_ends_of_the_range(nr, exponent, dtype, rows):
    """V's scales of 2^exponent to 2^(exponent + 1), codes so small that sums stay inside f32's range."""
    queries, group = ROWS[rows]
    p = problem(exponent + 200, [90, 57, 64], queries, 2, group, 128, 16, "fp8", dtype)
    rng = np.random.default_rng(exponent + 200)
    codes = [0x01, 0x81, 0x02, 0x82] if exponent > 100 else [0x70, 0xF0, 0x68, 0xEB]
    p["parts"][1] = rng.choice(np.array(codes, np.uint8), p["parts"][1].shape)
    p["parts"][3] = (2.0 ** exponent * rng.uniform(1, 2, p["parts"][3].shape)).astype(np.float32)
    close(run(nr, p), p, 128 ** -0.5)


@pytest.mark.parametrize("scores,values,dim", [
    (300, 0, 64), (-300, 0, 128), (300, 60, 128), (300, -60, 64), (-40, 100, 64), (0, 100, 128),
    (0, -100, 64), (40, -100, 128)])
def test_references_that_move_from_tile_to_tile(nr, scores, values, dim):
    """Sequences so long that a block walks many tiles of each: scores that move by `scores` along them
    and V's scales by 2^values, with normal values on top of both."""
    lens, queries, group = [5000, 4100, 3000], [14, 20, 13], 2
    p = problem(dim, lens, queries, 8, group, dim, 64, "fp8", bf)
    rng = np.random.default_rng(7)
    for i, n in enumerate(lens):
        pos = np.arange(n)
        at = p["table"][i, pos // 64], pos % 64
        k = rng.standard_normal((n, 8, dim)) + (pos / n * scores / dim ** 0.5)[:, None, None]
        p["parts"][0][at], p["parts"][2][at] = cache_ref.quant(k.astype(np.float32), "fp8")
        p["parts"][3][at] *= (2.0 ** np.round((pos / n - 0.5) * values)).astype(np.float32)[:, None]
    p["q"] = torch.ones_like(p["q"]) + 0.1 * p["q"]  # the scores' drift is that of their sum
    close(run(nr, p), p, dim ** -0.5, slice(None, None, 5))
