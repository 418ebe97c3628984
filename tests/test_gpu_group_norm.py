"""Group norm (channels last, optional SiLU) and its gradient on the GPU against
the formulas in 64 bits.

Tolerances, with U = 2^-24 and first-order terms (n is the longest chain of f32
additions that a sum takes: the rows of a thread, then lanes, channels and
blocks; CHAIN = 512 covers every size here):
  mean   a thread adds differences d to its first value f: |error| <= CHAIN U
         (mean |x| + mean |x - mean|) * 2
  rstd   M2 is a sum of squares taken by the same chains, and its square root
         halves the relative error: <= CHAIN U + (mean's error / deviation)^2
  z      = (x - mean) rstd w + b: the mean's error times rstd |w|, the relative
         errors of rstd and of three f32 operations on |xhat w|, one on |b|
  y      silu' is below 1.1; the activation's own error is below 2^-20 |y| (bf16,
         hardware exponential) or 8 U (|y| + |z| U) (f32), and below 2^-126 |z|
         where the sigmoid underflows; the store rounds by 2^-8 |y| (bf16) or U |y|
Gradients: dz moves by at most |dy| (silu'' is below 0.5 in size) dz' = |dy| 0.5 tol_z
+ 16 U |dy|; sums over n values move by the sum of their terms' errors plus CHAIN U
times the sum of their sizes.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
bf = torch.bfloat16
U, CHAIN = 2.0 ** -24, 512


def plain(x, groups, w, b, eps, act):
    """Everything in 64 bits; x [n, s, c]."""
    n, s, c = x.shape
    v = x.view(n, s, groups, c // groups)
    mean = v.mean((1, 3))
    var = ((v - mean[:, None, :, None]) ** 2).mean((1, 3))
    rstd = (var + eps) ** -0.5

    def wide(t):
        return t.repeat_interleave(c // groups, 1)[:, None]

    xhat = (x - wide(mean)) * wide(rstd)
    z = xhat * w + b
    y = z * torch.sigmoid(z) if act == "silu" else z
    return mean, rstd, xhat, z, y, wide


def bounds(x, groups, w, b, eps, act):
    mean, rstd, xhat, z, y, wide = plain(x, groups, w, b, eps, act)
    n, s, c = x.shape
    v = x.view(n, s, groups, -1)
    size = v.abs().mean((1, 3)) + (v - mean[:, None, :, None]).abs().mean((1, 3))
    t_mean = 2 * CHAIN * U * size
    t_rstd = rstd * (CHAIN * U + (t_mean * rstd) ** 2)
    t_z = (wide(t_mean) + U * (x - wide(mean)).abs()) * wide(rstd) * w.abs()
    t_z = t_z + (wide(t_rstd / rstd) + 4 * U) * (xhat * w).abs() + 2 * U * b.abs()
    return mean, rstd, xhat, z, y, wide, t_mean, t_rstd, t_z


def check_forward(x, groups, w, b, eps, act, y, mean, rstd, what=""):
    dt = x.dtype
    x64 = x.double().reshape(x.shape[0], -1, x.shape[-1])
    w64 = torch.ones(x.shape[-1], device=x.device).double() if w is None else w.double()
    b64 = torch.zeros_like(w64) if b is None else b.double()
    m, r, xhat, z, y64, wide, t_mean, t_rstd, t_z = bounds(x64, groups, w64, b64, eps, act)
    assert torch.all((mean.double() - m).abs() <= t_mean + 1e-44), what + " mean"
    assert torch.all((rstd.double() - r).abs() <= t_rstd), what + " rstd"
    tol = 1.1 * t_z + z.abs() * 2.0 ** -126
    if dt == bf:
        tol = tol + (2.0 ** -8 + 2.0 ** -20) * (y64.abs() + tol) + 2.0 ** -133
    else:
        tol = tol + 12 * U * (y64.abs() + z.abs() * U) + 2.0 ** -149
    err = (y.double().view_as(y64) - y64).abs()
    worst = (err - tol).max()
    assert worst <= 0, "%s y: %g over the tolerance" % (what, worst)


def inputs(n, space, chan, dtype, wdtype, seed=0, level=0.5, width=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (n, *space) if isinstance(space, tuple) else (n, space)
    x = torch.randn(*shape, chan, generator=g, device="cuda") * width
    x = (x + level * torch.randn(chan, generator=g, device="cuda") + level).to(dtype)
    if wdtype is None:
        return x, None, None
    w = (1 + 0.3 * torch.randn(chan, generator=g, device="cuda")).to(wdtype)
    b = (0.3 * torch.randn(chan, generator=g, device="cuda")).to(wdtype)
    return x, w, b


SIZES = [
    (1, 1, 8, 1), (1, 1, 64, 8), (2, 3, 8, 8), (3, 1, 320, 32), (1, 7, 24, 3), (2, 256, 1280, 32),
    (2, (16, 16), 640, 32), (1, (5, 9, 11), 128, 32), (4, 33, 512, 1), (1, 2560, 128, 32),
    (1, 2561, 128, 32), (5, 700, 40, 5), (1, 5000, 8, 1), (1, 5000, 8, 8), (3, (77, 93), 320, 32),
    (200, 65, 64, 4), (1, 300, 4104, 3), (2, 90, 8208, 3), (1, 40, 12288, 6), (1, 30, 65536, 1),
    (1, 100000, 16, 2), (160, 4000, 16, 1), (1, 436, 1824, 1), (3, 19, 1112, 8), (2, 9000, 96, 6),
    (1, 500, 120, 15), (1, 20000, 4096, 16), (2, 50, 680, 17),
    # one launch, clusters of 2, 4 and 8 blocks, the last of them short or without rows
    (1, 9, 2048, 1), (1, 33, 1024, 2), (3, 2600, 128, 32), (1, 20480, 64, 32), (1, 20481, 64, 32),
    (2, 10239, 64, 8), (7, 41, 1280, 4), (1, 40960, 16, 1), (1, 40961, 16, 1),
    (9, 1000, 256, 8),
]


@pytest.mark.parametrize("n,space,chan,groups", SIZES)
@pytest.mark.parametrize("dtype,wdtype,act", [(bf, bf, "silu"), (bf, torch.float32, None),
                                              (torch.float32, torch.float32, "silu"),
                                              (torch.float32, bf, "silu"),
                                              (torch.float32, None, None)])
def test_forward(nr, n, space, chan, groups, dtype, wdtype, act):
    x, w, b = inputs(n, space, chan, dtype, wdtype, seed=chan + groups)
    y, mean, rstd = nr.group_norm(x, groups, w, b, activation=act, stats=True)
    assert y.shape == x.shape and y.dtype == dtype and mean.shape == (n, groups)
    check_forward(x, groups, w, b, 1e-5, act, y, mean, rstd)
    assert torch.equal(nr.group_norm(x, groups, w, b, activation=act), y)  # and the same bits again


@pytest.mark.parametrize("n,space,chan,groups", [(2, 100, 64, 8), (1, 60000, 64, 8)])
def test_in_place_and_given_output(nr, n, space, chan, groups):
    x, w, b = inputs(n, space, chan, bf, bf)
    want = nr.group_norm(x, groups, w, b, activation="silu")
    out = torch.empty_like(x)
    assert nr.group_norm(x, groups, w, b, activation="silu", out=out) is out
    assert torch.equal(out, want)
    assert nr.group_norm(x, groups, w, b, activation="silu", out=x) is x
    assert torch.equal(x, want)


@pytest.mark.parametrize("space", [100, 60000])
def test_channels_far_from_zero_and_an_outlier(nr, space):
    """Means of 10^4 deviations, and one value of 10^5 deviations in the first place."""
    x, w, b = inputs(2, space, 64, torch.float32, torch.float32, level=1e4)
    y, mean, rstd = nr.group_norm(x, 8, w, b, stats=True)
    check_forward(x, 8, w, b, 1e-5, None, y, mean, rstd, "offset")
    x, w, b = inputs(2, space, 64, torch.float32, torch.float32)
    x[0, 0, 0] = 1e5
    x[1, 0, 63] = -1e5
    y, mean, rstd = nr.group_norm(x, 8, w, b, stats=True)
    check_forward(x, 8, w, b, 1e-5, None, y, mean, rstd, "outlier")


@pytest.mark.parametrize("space", [9, 60000])
@pytest.mark.parametrize("value", [0.0, 1.0, -3.0, 0.3])
def test_constant_groups(nr, space, value):
    x = torch.full((1, space, 32), value, device="cuda")
    w, b = torch.ones(32, device="cuda"), torch.linspace(-2, 2, 32, device="cuda")
    y, mean, rstd = nr.group_norm(x, 4, w, b, eps=1e-3, stats=True)
    check_forward(x, 4, w, b, 1e-3, None, y, mean, rstd)


@pytest.mark.parametrize("dtype", [bf, torch.float32])
def test_activations_far_out(nr, dtype):
    """z from -200 to 200: no NaN, zero or -0 far below, z far above."""
    x = torch.randn(1, 64, 16, device="cuda").to(dtype)
    w = torch.full((16,), 1e-3, device="cuda")
    b = torch.linspace(-200, 200, 16, device="cuda")
    y, mean, rstd = nr.group_norm(x, 2, w, b, activation="silu", stats=True)
    check_forward(x, 2, w, b, 1e-5, "silu", y, mean, rstd)


def test_a_nan_stays_in_its_group(nr):
    for space in (50, 60000):
        x, w, b = inputs(2, space, 64, bf, torch.float32)
        clean = nr.group_norm(x, 8, w, b, activation="silu")
        x[1, space // 2, 19] = float("nan")  # group 2
        y = nr.group_norm(x, 8, w, b, activation="silu")
        assert torch.isnan(y[1, :, 16:24]).all()
        y[1, :, 16:24] = clean[1, :, 16:24]
        assert torch.equal(y, clean)


@pytest.mark.parametrize("shape", [(0, 5, 64), (2, 0, 64)])
def test_no_elements(nr, shape):
    x = torch.empty(shape, dtype=bf, device="cuda")
    w = torch.ones(64, device="cuda")
    y, mean, rstd = nr.group_norm(x, 8, w, w, stats=True)
    assert y.shape == shape and mean.shape == (shape[0], 8)
    dx, dw, db = nr.group_norm_backward(x, x, mean, rstd, w, w)
    assert dx.shape == shape and not dw.any() and not db.any()


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------
def check_backward(nr, n, space, chan, groups, dtype, wdtype, act, seed=0):
    x, w, b = inputs(n, space, chan, dtype, wdtype, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    dy = (torch.randn(x.shape, generator=g, device="cuda") + 0.2).to(dtype)
    _, mean, rstd = nr.group_norm(x, groups, w, b, activation=act, stats=True)
    dx, dw, db = nr.group_norm_backward(dy, x, mean, rstd, w, b, activation=act)
    assert dx.shape == x.shape and dx.dtype == dtype
    again = nr.group_norm_backward(dy, x, mean, rstd, w, b, activation=act)
    assert torch.equal(again[0], dx) and (w is None or torch.equal(again[1], dw))
    # the formula in 64 bits, from the same mean and rstd
    x64 = x.double().reshape(n, -1, chan)
    d64 = dy.double().view_as(x64)
    w64 = torch.ones(chan, device="cuda").double() if w is None else w.double()
    b64 = torch.zeros_like(w64) if b is None else b.double()
    m, r = mean.double(), rstd.double()

    def wide(t):
        return t.repeat_interleave(chan // groups, 1)[:, None]

    xhat = (x64 - wide(m)) * wide(r)
    z = xhat * w64 + b64
    t_z = U * (6 * (xhat * w64).abs() + 2 * b64.abs())
    dz, t_dz = d64, U * d64.abs()
    if act == "silu":
        s = torch.sigmoid(z)
        dz = d64 * (s * (1 + z * (1 - s)))
        # the f32 form loses up to 4 U of 1 + |z| terms, the bf16 one 2^-20 of them
        t_dz = d64.abs() * (0.5 * t_z + (2.0 ** -20 if dtype == bf else 16 * U) *
                            (s * (1 + (z * (1 - s)).abs()) + s) + 2.0 ** -120)
    t_xhat = 4 * U * xhat.abs()
    S1, S2 = dz.sum((0, 1)), (dz * xhat).sum((0, 1))
    t1 = t_dz.sum((0, 1)) + CHAIN * U * dz.abs().sum((0, 1))
    t2 = (t_dz * xhat.abs() + dz.abs() * t_xhat).sum((0, 1)) + CHAIN * U * (dz * xhat).abs().sum((0, 1))
    if w is not None:
        assert dw.dtype == w.dtype and db.dtype == w.dtype
        store = 2.0 ** -8 if w.dtype == bf else U
        assert torch.all((db.double() - S1).abs() <= t1 + store * (S1.abs() + t1) + 1e-40), "db"
        assert torch.all((dw.double() - S2).abs() <= t2 + store * (S2.abs() + t2) + 1e-40), "dw"
    else:
        assert dw is None and db is None

    def group_mean(t):
        return t.reshape(n, t.shape[1], groups, -1).mean((1, 3))

    h = dz * w64
    c1, c2 = group_mean(h), group_mean(h * xhat)
    dx64 = wide(r) * (h - wide(c1) - xhat * wide(c2))
    t_h = t_dz * w64.abs() + 2 * U * h.abs()
    t_c1 = group_mean(t_h) + CHAIN * U * group_mean(h.abs())
    t_c2 = group_mean(t_h * xhat.abs() + h.abs() * t_xhat) + CHAIN * U * group_mean((h * xhat).abs())
    t_dx = wide(r) * (t_h + wide(t_c1) + xhat.abs() * wide(t_c2) + t_xhat * wide(c2.abs()) +
                      8 * U * (h.abs() + wide(c1.abs()) + (xhat * wide(c2)).abs()))
    t_dx = t_dx + (2.0 ** -8 if dtype == bf else U) * (dx64.abs() + t_dx) + 1e-40
    err = (dx.double().view_as(dx64) - dx64).abs()
    assert torch.all(err <= t_dx), "dx: %g over" % (err - t_dx).max()


@pytest.mark.parametrize("n,space,chan,groups", SIZES)
@pytest.mark.parametrize("dtype,wdtype,act", [(bf, bf, "silu"), (bf, torch.float32, None),
                                              (torch.float32, torch.float32, "silu"),
                                              (torch.float32, None, None)])
def test_backward(nr, n, space, chan, groups, dtype, wdtype, act):
    check_backward(nr, n, space, chan, groups, dtype, wdtype, act, seed=chan)


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("n,space,chan,groups", [(2, 30, 32, 4), (1, 9000, 24, 3)])
def test_gradient_against_differences(nr, act, n, space, chan, groups):
    """<grad, v> against central differences of sum(dy * f(p + h v)) in 64 bits, h =
    10^-4: the differences' own error is h^2 times a third derivative (below 10
    times the sum of |dy| |v|^3 here) and 2^-53 / h of the sum; the kernel's is an
    f32 one, CHAIN U times the sums of its terms."""
    x, w, b = inputs(n, space, chan, torch.float32, torch.float32, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    dy = torch.randn(x.shape, generator=g, device="cuda")
    _, mean, rstd = nr.group_norm(x, groups, w, b, activation=act, stats=True)
    grads = nr.group_norm_backward(dy, x, mean, rstd, w, b, activation=act)
    base = [t.double() for t in (x, w, b)]
    h = 1e-4
    for i, grad in enumerate(grads):
        v = torch.randn(base[i].shape, generator=g, device="cuda").double()

        def loss(step):
            p = [t + step * v if i == j else t for j, t in enumerate(base)]
            return (dy.double() * plain(*(p[0], groups, p[1], p[2], 1e-5, act))[4]).sum()

        want = (loss(h) - loss(-h)) / (2 * h)
        got = (grad.double() * v).sum()
        spread = dy.double().abs().sum()
        tol = 10 * h * h * spread * 30 + CHAIN * U * (grad.double().abs() * v.abs()).sum() * 4
        tol = tol + 2.0 ** -50 / h * spread
        assert (got - want).abs() <= tol, (i, float(got), float(want), float(tol))


@pytest.mark.parametrize("which", ["dy", "x"])
def test_gradient_in_place(nr, which):
    for space in (40, 60000):
        x, w, b = inputs(2, space, 64, bf, torch.float32)
        dy = torch.randn_like(x)
        _, mean, rstd = nr.group_norm(x, 8, w, b, activation="silu", stats=True)
        want = nr.group_norm_backward(dy, x, mean, rstd, w, b, activation="silu")
        place = dy if which == "dy" else x
        got = nr.group_norm_backward(dy, x, mean, rstd, w, b, activation="silu", dx=place)
        assert got[0] is place and torch.equal(place, want[0])
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


def test_outputs_stay_inside_their_buffers(nr):
    from tests.gpu_util import Guarded
    for n, space, chan, groups in ((3, 41, 40, 5), (1, 30011, 24, 3)):
        for dtype in (bf, torch.float32):
            x, w, b = inputs(n, space, chan, dtype, torch.float32)
            out = Guarded(x.shape, dtype)
            _, mean, rstd = nr.group_norm(x, groups, w, b, out=out.t, stats=True)
            dx = Guarded(x.shape, dtype)
            nr.group_norm_backward(x, x, mean, rstd, w, b, dx=dx.t)
            torch.cuda.synchronize()
            out.check()
            dx.check()


def test_two_streams_and_replayed_graphs(nr):
    """Calls on two streams at once, and two graphs (forward + backward) replayed
    in turn: each call's workspace is its own."""
    cases = [inputs(1, 20000, 64, bf, torch.float32, seed=i) for i in range(2)]

    def both(x, w, b):
        y, mean, rstd = nr.group_norm(x, 8, w, b, activation="silu", stats=True)
        return (y, *nr.group_norm_backward(y, x, mean, rstd, w, b, activation="silu"))

    want = [both(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = both(*cases[i])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    graphs, outs = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both(*c))
        graphs.append(g)
    for _ in range(2):
        cases[0][0].normal_()
        cases[1][0].mul_(0.5)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for c, o in zip(cases, outs):
            assert all(torch.equal(x, y) for x, y in zip(both(*c), o))


def test_past_2_to_31_elements(nr):
    """Rows around element 2^31, forward and backward, against 64-bit sums."""
    chan, groups = 64, 4
    space = (1 << 31) // chan + 5000
    x = torch.empty(1, space, chan, dtype=bf, device="cuda").normal_()
    w, b = torch.ones(chan, device="cuda"), torch.zeros(chan, device="cuda")
    y, mean, rstd = nr.group_norm(x, groups, w, b, stats=True)
    total = torch.zeros(groups, dtype=torch.float64, device="cuda")
    square = torch.zeros_like(total)
    for part in x[0].split(1 << 22):
        v = part.double().view(-1, groups, chan // groups)
        total += v.sum((0, 2))
        square += (v * v).sum((0, 2))
    m = total / (space * chan // groups)
    var = square / (space * chan // groups) - m * m
    # chains of up to 2^14 additions in a thread, random in sign: 10^-5 is generous
    assert torch.allclose(mean[0].double(), m, atol=1e-5)
    assert torch.allclose(rstd[0].double(), (var + 1e-5) ** -0.5, rtol=1e-5)
    dx, dw, db = nr.group_norm_backward(x, x, mean, rstd, w, b)
    at = (1 << 31) // chan
    for r0 in (0, at - 2, space - 3):
        v = x[0, r0:r0 + 3].double().view(3, groups, -1)
        xhat = (v - mean[0].double()[:, None]) * rstd[0].double()[:, None]
        got = y[0, r0:r0 + 3].double().view_as(xhat)
        assert torch.all((got - xhat).abs() <= 2.0 ** -8 * xhat.abs() + 1e-4)
        # dy = x: the gradient along x vanishes up to eps and rounding
        assert dx[0, r0:r0 + 3].abs().max() <= 1e-3
