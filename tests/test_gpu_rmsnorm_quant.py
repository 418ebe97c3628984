"""RMSNorm with e4m3 codes and scales made from the data, against 64 bits.

u = 2^-24.  The sum of squares is one of positive terms: at most 16 vectors of 8 a thread, 5 steps
of a butterfly and 32 warps, so its relative error is below (128 + 37) u and its root's half of
that; the mean, the reciprocal root (refined) and the products add less than 10 u.  n is within
DELTA = 100 u of itself.  A code is the nearest of n * 448 / a, or its neighbour where a
relative error of DELTA carries that over a rounding border."""
import numpy as np
import pytest
import torch

from tests.cache_ref import CEIL, E4M3, FLOOR, nearest

pytestmark = pytest.mark.gpu
DELTA = 100 * 2.0 ** -24
bf, f32 = torch.bfloat16, torch.float32
EXTENT = {"row": None, "group": 128, "mx": 32}


def normed(x, w, residual, eps, gemma):
    """(n in 64 bits, the new residual) of stored values."""
    if residual is not None:
        residual = (x.float() + residual.float()).to(x.dtype)
        x = residual
    v = x.double().numpy()
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        inv = 1 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
        return v * inv * (w.double().numpy() + (1 if gemma else 0)), residual


def check(codes, scales, n, layout):
    rows, hidden = n.shape
    ext = EXTENT[layout] or hidden
    g = n.reshape(rows, -1, ext)
    a = np.abs(np.where(np.isnan(g), 0, g)).max(-1)
    a = np.minimum(np.maximum(a, float(FLOOR)), float(CEIL))
    got = scales.cpu().numpy().reshape(rows, -1)
    assert got.shape == a.shape
    if layout == "mx":
        s = got.astype(np.int64) - 127
        lo, hi = a * (1 - DELTA), a * (1 + DELTA)
        assert (lo / 2.0 ** s <= 448).all() and (hi / 2.0 ** (s - 1) > 448).all()
        p = g / (2.0 ** s)[..., None]
    else:
        assert (np.abs(got - a / 448) <= DELTA * a / 448).all()
        p = g * (448 / a)[..., None]
    c = codes.cpu().numpy().reshape(g.shape)
    nan = np.isnan(p)
    assert ((c[nan] & 0x7F) == 0x7F).all()
    p, c = p[~nan], c[~nan]
    mag = np.abs(p)
    low, high = nearest(mag * (1 - DELTA), E4M3), nearest(mag * (1 + DELTA), E4M3)
    m = c & 0x7F
    assert ((m >= low) & (m <= high)).all()
    assert (((c & 0x80) != 0) == np.signbit(p))[m > 0].all()


def case(seed, rows, hidden, dtype, residual):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, hidden, generator=g) * torch.exp(torch.randn(hidden, generator=g))).to(dtype)
    w = (1 + 0.2 * torch.randn(hidden, generator=g)).to(dtype)
    r = torch.randn(rows, hidden, generator=g).to(dtype) if residual else None
    return x, w, r


def run(nr, x, w, r, layout, **kw):
    rd = None if r is None else r.cuda()
    codes, scales = nr.rmsnorm_quant(x.cuda(), w.cuda(), residual=rd, scales=layout, **kw)
    return codes, scales, rd


SHAPES = [(1, 128), (3, 256), (7, 1024), (32, 4096), (40, 4096), (300, 640), (257, 2176), (260, 5120),
          (2, 16384), (258, 8192), (259, 16384)]


@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("layout", ["row", "group", "mx"])
@pytest.mark.parametrize("dtype", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True], ids=["", "res"])
def test_shapes(nr, rows, hidden, layout, dtype, residual):
    x, w, r = case(rows + hidden, rows, hidden, dtype, residual)
    gemma = rows % 2 == 1
    codes, scales, rd = run(nr, x, w, r, layout, eps=1e-5, gemma=gemma)
    n, new = normed(x, w, r, 1e-5, gemma)
    check(codes, scales, n, layout)
    if residual:
        assert torch.equal(rd.cpu(), new)


@pytest.mark.parametrize("hidden,dtype", [(8, bf), (24, bf), (4, f32), (1000, bf), (32768, bf), (30000, bf)])
def test_row_scales_of_any_width(nr, hidden, dtype):
    for rows in (5, 300):
        x, w, r = case(hidden, rows, hidden, dtype, True)
        codes, scales, rd = run(nr, x, w, r, "row")
        n, new = normed(x, w, r, 1e-6, False)
        check(codes, scales, n, "row")
        assert torch.equal(rd.cpu(), new)


@pytest.mark.parametrize("layout", ["row", "group", "mx"])
@pytest.mark.parametrize("rows", [4, 300])
def test_rows_at_the_ends_of_the_range(nr, layout, rows):
    """Zero rows, rows of subnormal and of huge values, zero weights, one NaN."""
    x, w, _ = case(1, rows, 512, f32, False)
    x[0] = 0
    x[1] *= 1e-41
    x[2] *= 1e15
    w[128:256] = 0
    w[300] = 1e-30
    codes, scales, _ = run(nr, x, w, None, layout, eps=1e-6)
    n, _ = normed(x, w, None, 1e-6, False)
    check(codes, scales, n, layout)
    x[3, 7] = float("nan")
    codes, scales, _ = run(nr, x, w, None, layout)
    n, _ = normed(x, w, None, 1e-6, False)
    check(codes, scales, n, layout)  # the whole row is NaN


@pytest.mark.parametrize("layout", ["row", "group", "mx"])
def test_weights_beyond_plain_products(nr, layout):
    """v w leaves f32's range while n does not."""
    x, w, _ = case(2, 5, 256, f32, False)
    x *= 1e18
    w *= 1e25
    codes, scales, _ = run(nr, x, w, None, layout)
    n, _ = normed(x, w, None, 1e-6, False)
    check(codes, scales, n, layout)


def test_given_outputs_are_filled_and_nothing_else(nr):
    x, w, r = case(3, 9, 384, bf, True)
    buf = torch.full((9 * 384 + 512,), 0x55, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((9 * 3 + 64,), 7.0, device="cuda")
    codes, scales = buf[256:-256].view(9, 384), sbuf[32:-32].view(9, 3)
    c, s = nr.rmsnorm_quant(x.cuda(), w.cuda(), residual=r.cuda(), scales="group", codes=codes,
                            scales_out=scales)
    assert c is codes and s is scales
    n, _ = normed(x, w, r, 1e-6, False)
    check(codes, scales, n, "group")
    assert (buf[:256] == 0x55).all() and (buf[-256:] == 0x55).all()
    assert (sbuf[:32] == 7).all() and (sbuf[-32:] == 7).all()


def test_against_the_static_scale(nr):
    """With the row's own scale the static entry point gives the codes of the bf16-rounded
    value: at most one step away."""
    x, w, _ = case(4, 6, 1024, bf, False)
    codes, scales, _ = run(nr, x, w, None, "row")
    for i in range(6):
        static = nr.rmsnorm_quant_fp8(x[i:i + 1].cuda(), w.cuda(), float(scales[i]))
        step = (static[0].int() & 0x7F) - (codes[i].int() & 0x7F)
        assert (step.abs() <= 1).all()


def test_offsets_past_32_bits(nr):
    rows, hidden = 131073, 32768
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    x = torch.zeros(rows, hidden, dtype=bf, device="cuda")
    small, w, _ = case(5, 2, hidden, bf, False)
    x[0], x[-1] = small[0].cuda(), small[1].cuda()
    for layout in ("row", "mx"):
        codes, scales = nr.rmsnorm_quant(x, w.cuda(), scales=layout)
        n, _ = normed(small, w, None, 1e-6, False)
        check(codes[[0, -1]], scales[[0, -1]], n, layout)
        del codes


def test_same_bits_in_a_graph_and_with_no_rows(nr):
    x, w, r = case(6, 33, 2048, bf, True)
    xd, wd = x.cuda(), w.cuda()
    codes, scales, _ = run(nr, x, w, r, "mx")
    held = torch.zeros_like(codes), torch.zeros_like(scales)
    rd = r.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nr.rmsnorm_quant(xd, wd, residual=rd, scales="mx", codes=held[0], scales_out=held[1])
    for _ in range(2):
        rd.copy_(r)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held[0], codes) and torch.equal(held[1], scales)
    c, s = nr.rmsnorm_quant(xd[:0], wd)
    assert c.shape == (0, 2048) and s.shape == (0,)
