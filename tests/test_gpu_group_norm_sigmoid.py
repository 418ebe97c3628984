"""The sigmoid of the group-norm gradient, seen in the f32 db of one row.

With x = 0, mean 0, rstd 1 and w = 1, z is b and db is dz = dy s (1 + z (1 - s)) of one
row, in f32 whatever x is.  U = 2^-24.  For bf16 x the sigmoid s comes from the hardware:
-z log2(e) is rounded once and its constant is off by 2^-26 (together 1.3 |z| U of e^-z),
ex2.approx is off by 2^-22, the sum rounds once and rcp.approx is off by an ulp: at
most (1.3 |z| + 7) U of s for z < 0, and of that e^-z / (1 + e^-z) <= 1 - s for z >= 0
with 3 U more.  For f32 x it is expf (2 ulps) and a division: 8 U.  dz then moves by
|1 + z - 2 z s| times s's error, and three more roundings of at most U s (1 + |z| (1 -
s)) each follow.  Below 2^-126 the hardware's results are zero."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_derivative_of_one_row(nr, dtype):
    chan, U = 65536, 2.0 ** -24
    b = torch.linspace(-100, 100, chan, device="cuda")
    b = torch.where(torch.arange(chan, device="cuda") % 2 == 0, b, b / 16)
    x = torch.zeros(1, 1, chan, dtype=dtype, device="cuda")
    dy = torch.ones_like(x)
    w, mean, rstd = torch.ones(chan, device="cuda"), torch.zeros(1, 1, device="cuda"), \
        torch.ones(1, 1, device="cuda")
    _, _, db = nr.group_norm_backward(dy, x, mean, rstd, w, b, activation="silu")
    z = b.double()
    s = 1 / (1 + (-z).exp())
    rest = 1 / (1 + z.exp())  # 1 - s
    want = s * (1 + z * rest)
    if dtype == torch.bfloat16:
        ds = torch.where(z < 0, s * (1.3 * z.abs() + 7) * U, s * ((1.3 * z + 7) * rest + 3) * U)
    else:
        ds = 8 * U * s
    tol = (1 + z - 2 * z * s).abs() * ds + z.abs() * ds * ds + 3 * U * s * (1 + z.abs() * rest)
    # 1 - s is taken from the rounded s: U of s more in it, times z
    tol = tol + U * z.abs() * s * s + 2.0 ** -126 * (1 + z.abs())
    over = ((db.double() - want).abs() / tol).max()
    assert over <= 1, over
