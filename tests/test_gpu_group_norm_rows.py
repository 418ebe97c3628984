"""Every row of a group norm is taken exactly once, forward and backward.

Rounding cannot hide a lost or doubled row here.  Gradient: integers, with mean 0
and rstd 1 given, so that every f32 sum is exact in any order (all partial sums stay
below 2^24) and db and dw have to be equal to the integer sums.  Forward: one row of
value B, the others zero; a thread that does not have the row adds exact zeros, so
with k rows in the thread that has it
  mean   B / space within 2 U for the thread's own mean and one rounding for each
         product, addition and quotient of the joins that meet it (fewer than 500
         in all): 2^-15 relative
  rstd   M2 = s2 - s1^2 / k loses at most 3 k U where the row is the thread's first
         (s1^2 / k is then k times M2), k <= 700 at the sizes here, and what the means'
         roundings add in the joins is below that: 2^-12 relative, half of it in
         rstd
A row that is lost gives mean 0, one taken twice 2 B / space."""
import pytest
import torch

from tests.test_gpu_group_norm import SIZES

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def space_of(space):
    return space[0] * space[1] * (space[2] if len(space) > 2 else 1) if isinstance(space, tuple) else space


FLAT = sorted({(n, space_of(s), c, g) for n, s, c, g in SIZES})


@pytest.mark.parametrize("n,space,chan,groups", FLAT)
@pytest.mark.parametrize("dtype", [bf, f32])
def test_each_row_in_the_statistics(nr, n, space, chan, groups, dtype):
    B, eps = 1024.0, 1.0
    gen = torch.Generator().manual_seed(space + chan)
    vec = 8 if dtype == bf else 4
    lanes = max(1, 512 // -(-chan // vec))  # rows that a block may take side by side
    rows = {0, 1, space - 1, space - 2, space // 2, space - lanes, space - lanes - 1, lanes, lanes - 1,
            8 * lanes, 8 * lanes - 1, space - space % lanes, space - space % lanes - 1}
    rows |= set(torch.randint(0, space, (6,), generator=gen).tolist())
    rows = sorted(r for r in rows if 0 <= r < space)
    x = torch.zeros(n, space, chan, dtype=dtype, device="cuda")
    want_mean = B / space
    want_rstd = (B * B * (space - 1) / space ** 2 + eps) ** -0.5
    means, rstds = [], []
    for r in rows:
        s = r % n
        x[s, r] = B
        _, mean, rstd = nr.group_norm(x, groups, eps=eps, stats=True)
        x[s, r] = 0
        means.append(mean)
        rstds.append(rstd)
    for r, mean, rstd in zip(rows, means, rstds):
        s = r % n
        assert torch.all((mean[s].double() / want_mean - 1).abs() <= 2.0 ** -15), (r, "mean")
        assert torch.all((rstd[s].double() / want_rstd - 1).abs() <= 2.0 ** -12), (r, "rstd")
        other = torch.arange(n, device="cuda") != s
        assert not mean[other].any() and torch.all(rstd[other] == 1)


def whole(shape, lo, hi, gen, dtype):
    return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("n,space,chan,groups", FLAT)
@pytest.mark.parametrize("dtype", [bf, f32])
def test_gradient_sums_of_integers_are_exact(nr, n, space, chan, groups, dtype):
    gen = torch.Generator(device="cuda").manual_seed(space)
    x = whole((n, space, chan), -2, 2, gen, dtype)
    dy = whole((n, space, chan), 1, 3, gen, dtype)
    w, b = whole((chan,), 1, 2, gen, f32), torch.zeros(chan, device="cuda")
    assert 3 * 2 * n * space < 1 << 24  # every sum over a channel
    mean, rstd = torch.zeros(n, groups, device="cuda"), torch.ones(n, groups, device="cuda")
    dx, dw, db = nr.group_norm_backward(dy, x, mean, rstd, w, b)
    x64, d64 = x.double(), dy.double()
    assert torch.equal(db.double(), d64.sum((0, 1)))
    assert torch.equal(dw.double(), (d64 * x64).sum((0, 1)))
    # dx = w dy - m1 - x m2, m1 and m2 means of integers below 6 and 12 in size.  A
    # group's f32 sums are exact up to 2^24; beyond, its channels' exact sums are
    # joined with a rounding each (at most channels + 608 blocks of them), and the
    # product with 1 / n, the two f32 operations and the store round once each.
    h = d64 * w.double()
    m1 = h.view(n, space, groups, -1).mean((1, 3), keepdim=True)
    m2 = (h * x64).view(n, space, groups, -1).mean((1, 3), keepdim=True)
    want = (h.view(n, space, groups, -1) - m1 - x64.view(n, space, groups, -1) * m2).view_as(h)
    U = 2.0 ** -24
    exact = 12 * space * (chan // groups) < 1 << 24
    chain = 8 if exact else 8 + chan // groups + 608
    tol = chain * U * 6 + x64.abs() * (chain * U * 12) + 8 * U * want.abs()
    tol = tol + (2.0 ** -8 if dtype == bf else U) * (want.abs() + tol)
    assert torch.all((dx.double() - want).abs() <= tol)


def test_gradient_past_2_to_31_elements(nr):
    """x and dy of their own, rows past element 2^31 of a level of their own, dx filled
    beforehand; everything against 64-bit sums over chunks of rows.  A thread has at
    most 3500 rows ((2^25 + 5000) / 64 lanes / 152 blocks) and a join fewer than 600
    parts: a sum's error is at most 4100 U of the sum of its terms' sizes."""
    chan, groups, U, chain = 64, 4, 2.0 ** -24, 4100
    per = chan // groups
    cut = (1 << 31) // chan
    space = cut + 5000
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(1, space, chan, dtype=bf, device="cuda").normal_(generator=gen)
    dy = torch.empty_like(x).normal_(generator=gen)
    x[0, cut:] += 100
    dy[0, cut:] += 50
    w = 1 + 0.25 * torch.randn(chan, generator=gen, device="cuda")
    b = torch.randn(chan, generator=gen, device="cuda")
    y, mean, rstd = nr.group_norm(x, groups, w, b, stats=True)

    def chunks():
        for r0 in range(0, space, 1 << 20):
            yield r0, min(r0 + (1 << 20), space)

    d = torch.float64
    zero = lambda n: torch.zeros(n, dtype=d, device="cuda")  # noqa: E731
    total, size = zero(groups), zero(groups)
    for r0, r1 in chunks():
        v = x[0, r0:r1].double().view(-1, groups, per)
        total += v.sum((0, 2))
        size += v.abs().sum((0, 2))
    count = space * per
    m64 = total / count
    square = zero(groups)
    for r0, r1 in chunks():
        square += (x[0, r0:r1].double().view(-1, groups, per) - m64[:, None]).square().sum((0, 2))
    r64 = (square / count + 1e-5) ** -0.5
    # the 5000 rows move the mean by 0.0149 and the variance by 1.49
    t_mean = 2 * chain * U * size / count
    assert t_mean.max() < 1e-3
    assert torch.all((mean[0].double() - m64).abs() <= t_mean)
    assert torch.all((rstd[0].double() / r64 - 1).abs() <= chain * U + (t_mean * r64) ** 2)

    dx = torch.full_like(x, -77.0)
    got, dw, db = nr.group_norm_backward(dy, x, mean, rstd, w, b, dx=dx)
    assert got is dx
    m, r = mean[0].double(), rstd[0].double()
    S1, S2, A1, A2 = zero(chan), zero(chan), zero(chan), zero(chan)

    def parts(r0, r1):
        xhat = ((x[0, r0:r1].double().view(-1, groups, per) - m[:, None]) * r[:, None]).view(-1, chan)
        return xhat, dy[0, r0:r1].double()

    for r0, r1 in chunks():
        xhat, dz = parts(r0, r1)
        S1 += dz.sum(0)
        S2 += (dz * xhat).sum(0)
        A1 += dz.abs().sum(0)
        A2 += (dz * xhat).abs().sum(0)
    # the 5000 rows are 250000 of each db; what is lost or doubled shows
    t1, t2 = (chain + 8) * U * A1, (chain + 8) * U * A2
    assert t1.max() < 20000
    assert torch.all((db.double() - S1).abs() <= t1) and torch.all((dw.double() - S2).abs() <= t2)
    w64 = w.double()
    c1 = (w64 * S1).view(groups, per).sum(1) / count
    c2 = (w64 * S2).view(groups, per).sum(1) / count
    e1 = (w64.abs() * (t1 + 8 * U * A1)).view(groups, per).sum(1) / count
    e2 = (w64.abs() * (t2 + 8 * U * A2)).view(groups, per).sum(1) / count
    wide = lambda t: t.repeat_interleave(per)  # noqa: E731
    for r0, r1 in chunks():
        xhat, dz = parts(r0, r1)
        h = dz * w64
        want = wide(r) * (h - wide(c1) - xhat * wide(c2))
        tol = wide(r) * (wide(e1) + xhat.abs() * wide(e2) +
                         8 * U * (h.abs() + wide(c1.abs()) + (xhat * wide(c2)).abs()))
        tol = tol + 2.0 ** -8 * (want.abs() + tol) + 1e-40
        assert torch.all((dx[0, r0:r1].double() - want).abs() <= tol), r0
        z = xhat * w64 + b.double()
        tol = 2.0 ** -8 * z.abs() + 16 * U * ((xhat * w64).abs() + b.double().abs()) + 1e-40
        assert torch.all((y[0, r0:r1].double() - z).abs() <= tol), r0
