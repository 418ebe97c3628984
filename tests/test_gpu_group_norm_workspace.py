"""Group norm through the C ABI with a workspace of exactly the bytes that the query
names, between guard bands and filled with NaN: nothing outside it is written, and
nothing in it is read before it is written."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32
F32, BF16 = 0, 1
BAND = 4096

SIZES = [
    (1, 40, 64, 8), (2, 256, 1280, 32), (7, 41, 1280, 4), (200, 65, 64, 4),  # one launch
    (1, 20481, 64, 32), (2, 10239, 64, 8), (4, 1024, 640, 32), (9, 1000, 256, 8),  # clusters
    (1, 26229, 48, 3), (3, 7161, 320, 32), (160, 4000, 16, 1), (1, 100001, 8, 1),  # two launches
    (1, 300, 4104, 3), (2, 90, 8208, 3), (1, 30, 65536, 1), (3, 700, 12288, 6),  # groups across tiles
]


@pytest.mark.parametrize("n,s,c,g", SIZES)
@pytest.mark.parametrize("dtype", [bf, f32])
def test_a_workspace_of_the_queried_size(nr, n, s, c, g, dtype):
    code = BF16 if dtype == bf else F32
    gen = torch.Generator(device="cuda").manual_seed(c)
    x = torch.randn(n, s, c, generator=gen, device="cuda").to(dtype)
    dy = torch.randn(n, s, c, generator=gen, device="cuda").to(dtype)
    w, b = (torch.randn(c, generator=gen, device="cuda") for _ in range(2))
    out, dx, dw, db = (torch.empty_like(t) for t in (x, x, w, b))
    mean, rstd = (torch.empty(n, g, device="cuda") for _ in range(2))

    def guarded(backward):
        need = ctypes.c_int64(-1)
        assert nr.lib.nr_group_norm_workspace(n, s, c, g, backward, code, ctypes.byref(need)) == 0
        buf = torch.full((need.value + 2 * BAND,), 0x5A, dtype=torch.uint8, device="cuda")
        buf[BAND:BAND + need.value] = 0xFF  # NaN in every float
        return buf, need.value

    def check(buf, need):
        assert torch.all(buf[:BAND] == 0x5A), "written in front of the workspace"
        assert torch.all(buf[BAND + need:] == 0x5A), "written behind the workspace"

    stream = torch.cuda.current_stream().cuda_stream
    buf, need = guarded(0)
    assert nr.lib.nr_group_norm(out.data_ptr(), mean.data_ptr(), rstd.data_ptr(), x.data_ptr(),
                                w.data_ptr(), b.data_ptr(), F32, n, s, c, g, 1e-5, 1, code,
                                buf.data_ptr() + BAND, need, stream) == 0
    check(buf, need)
    want = nr.group_norm(x, g, w, b, activation="silu", stats=True)
    assert all(torch.equal(a, t) for a, t in zip((out, mean, rstd), want))
    assert torch.isfinite(out).all()
    buf, need = guarded(1)
    assert nr.lib.nr_group_norm_backward(dx.data_ptr(), dw.data_ptr(), db.data_ptr(), dy.data_ptr(),
                                         x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), w.data_ptr(),
                                         b.data_ptr(), F32, n, s, c, g, 1, code,
                                         buf.data_ptr() + BAND, need, stream) == 0
    check(buf, need)
    want = nr.group_norm_backward(dy, x, mean, rstd, w, b, activation="silu")
    assert all(torch.equal(a, t) for a, t in zip((dx, dw, db), want))
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
