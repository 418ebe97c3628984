"""The quantised K/V cache on the GPU against the plain reference (numpy, 64
bits; tests/cache_ref.py).

Writing has fixed f32 roundings, so codes and scales are compared bit for bit.
Reading back multiplies a code by its scale in f32 and rounds once, so it is
compared with that too.  Every test checks that what a call may not touch kept
its bits."""
import numpy as np
import pytest
import torch

from tests import cache_ref as ref

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


def make_cache(fmt, blocks, page, heads, dim, seed=0, interleaved=False):
    """Four parts filled with random old contents (no e4m3 NaN among them)."""
    g = torch.Generator().manual_seed(seed)
    width = dim if fmt == "fp8" else dim // 2
    shape = (blocks, 2, page, heads) if interleaved else (2, blocks, page, heads)
    codes = torch.randint(0, 256, (*shape, width), generator=g, dtype=torch.uint8) & 0xF7
    if fmt == "fp8":
        scales = torch.rand(shape, generator=g) + 0.1
    else:
        scales = torch.randint(120, 130, (*shape, dim // 32), generator=g, dtype=torch.uint8)
    codes, scales = codes.cuda(), scales.cuda()
    if interleaved:
        return codes[:, 0], codes[:, 1], scales[:, 0], scales[:, 1]
    return codes[0], codes[1], scales[0], scales[1]


def flat(t):
    """[slots, ...] on the host."""
    t = t.cpu().numpy()
    return t.reshape(-1, *t.shape[2:])


def f32(t):
    return t.detach().float().cpu().numpy()


def check_written(parts, before, k, v, slots, fmt):
    """The slots hold the reference's codes and scales, the others what they had."""
    n = parts[0].shape[0] * parts[0].shape[1]
    keep = [i for i, s in enumerate(slots) if 0 <= s < n]
    at = [int(slots[i]) for i in keep]
    for part, old, src, which in ((parts[0], before[0], k, 0), (parts[2], before[2], k, 1),
                                  (parts[1], before[1], v, 0), (parts[3], before[3], v, 1)):
        want = old.copy()
        want[at] = ref.quant(f32(src)[keep], fmt)[which]
        got = flat(part)
        assert np.array_equal(got.view(np.uint8), want.view(np.uint8)), (
            "part of %s: %d bytes differ" % ("codes" if which == 0 else "scales",
                                             int((got.view(np.uint8) != want.view(np.uint8)).sum())))


def run_write(nr, fmt, tokens, heads, dim, page, dtype, seed=1, interleaved=False, edit=None,
              strided=False):
    g = torch.Generator().manual_seed(seed)
    blocks = -(-tokens // page) + 3
    parts = make_cache(fmt, blocks, page, heads, dim, seed, interleaved)
    before = [flat(p) for p in parts]
    k = torch.randn(tokens, heads, dim, generator=g) * torch.exp(
        torch.randn(tokens, heads, 1, generator=g) * 3)
    v = torch.randn(tokens, heads, dim, generator=g)
    if edit is not None:
        edit(k, v)
    k, v = k.to(dtype).cuda(), v.to(dtype).cuda()
    if strided:  # views of one fused row [K | pad | V]
        row = torch.zeros(tokens, 2 * heads + 1, dim, dtype=dtype, device="cuda")
        row[:, :heads], row[:, heads + 1:] = k, v
        k, v = row[:, :heads], row[:, heads + 1:]
    slots = torch.randperm(blocks * page, generator=g)[:tokens]
    if tokens > 3:
        slots[1], slots[3] = -1, blocks * page  # padding, and past the end
    nr.kv_cache_write(k, v, slots.cuda(), *parts)
    torch.cuda.synchronize()
    check_written(parts, before, k, v, slots.tolist(), fmt)
    return parts, slots


@pytest.mark.parametrize("dtype", [bf, torch.float32])
@pytest.mark.parametrize("fmt,dim", [("fp8", d) for d in (16, 32, 48, 64, 80, 96, 112, 128, 160, 192,
                                                         240, 256, 272, 512)] +
                         [("mxfp4", d) for d in (32, 64, 96, 128, 160, 224, 256, 288, 512)])
def test_write_head_dims(nr, fmt, dim, dtype):
    run_write(nr, fmt, 37, 3, dim, 16, dtype, seed=dim)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("tokens,heads,page", [(1, 1, 1), (1, 8, 16), (2, 7, 3), (5, 1, 128),
                                               (333, 5, 24), (4096, 8, 64)])
def test_write_sizes_and_pages(nr, fmt, tokens, heads, page):
    run_write(nr, fmt, tokens, heads, 128, page, bf, seed=tokens)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("dtype", [bf, torch.float32])
def test_write_strided_rows_into_interleaved_blocks(nr, fmt, dtype):
    run_write(nr, fmt, 70, 4, 64, 8, dtype, interleaved=True, strided=True)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("dtype", [bf, torch.float32])
def test_write_edge_values(nr, fmt, dtype):
    def edit(k, v):
        k[0] = 0                      # a row of zeros
        k[2, 0, :] = 1e-42            # below the scales' floor (bf16: subnormal)
        k[2, 1, 5] = float("inf")
        k[4, 0, 7] = float("-inf")
        k[4, 1] = 3.3e38
        v[0, 0] = 2.0 ** -100
        v[0, 1] = torch.arange(64) * 7.0 - 200  # ties and exact grid points among them
        v[5, 0] = torch.where(torch.arange(64) % 2 == 0, 6.0, -0.0)
        v[5, 1] = torch.linspace(-448, 448, 64)
        k[1] = float("nan")           # a padded token: not looked at
        if fmt == "fp8":
            v[6, 1, 3] = float("nan")  # stays NaN, spoils nothing else
    run_write(nr, fmt, 9, 2, 64, 4, dtype, edit=edit)


def test_write_rounding_of_every_e4m3_and_e2m1_boundary(nr):
    """Rows whose largest value pins the scale to 1 hold every grid point, every
    midpoint between two and the f32 neighbours of each."""
    pts = np.concatenate([ref.E4M3, (ref.E4M3[1:] + ref.E4M3[:-1]) / 2]).astype(np.float32)
    pts = np.concatenate([pts, np.nextafter(pts, np.float32(0)), np.nextafter(pts, np.float32(999))])
    pts = pts[pts <= 448]
    rows = -(-len(pts) // 127)
    x = np.full((rows, 1, 128), 448, np.float32)
    body = np.zeros(rows * 127, np.float32)
    body[:len(pts)] = pts
    x[:, 0, :127] = body.reshape(rows, 127)
    x[1::2] *= -1
    k = torch.from_numpy(x).cuda()
    parts = make_cache("fp8", rows, 1, 1, 128)
    nr.kv_cache_write(k, k, torch.arange(rows, device="cuda"), *parts)
    assert np.array_equal(flat(parts[0]), ref.quant_fp8(x)[0])
    assert np.all(flat(parts[2]) == 1)
    m = np.concatenate([ref.E2M1, (ref.E2M1[1:] + ref.E2M1[:-1]) / 2]).astype(np.float32)
    m = np.concatenate([m, np.nextafter(m, np.float32(0)), np.nextafter(m, np.float32(9))])
    m = np.concatenate([m[m <= 6], -m[m <= 6]])
    x = np.full((-(-len(m) // 31), 1, 32), 6, np.float32)
    body = np.zeros(x.shape[0] * 31, np.float32)
    body[:len(m)] = m
    x[:, 0, :31] = body.reshape(-1, 31)
    k = torch.from_numpy(x).cuda()
    parts = make_cache("mxfp4", x.shape[0], 1, 1, 32)
    nr.kv_cache_write(k, k, torch.arange(x.shape[0], device="cuda"), *parts)
    assert np.array_equal(flat(parts[0]), ref.quant_mxfp4(x)[0])
    assert np.all(flat(parts[2]) == 127)


def test_scales_are_the_correctly_rounded_quotients(nr):
    """2^16 significands over many exponents: scale = a / 448 bit for bit."""
    rng = np.random.default_rng(5)
    a = rng.integers(0, 1 << 23, 1 << 16).astype(np.uint32)
    a |= (rng.integers(28, 254, 1 << 16).astype(np.uint32)) << 23
    a = a.view(np.float32)
    x = np.zeros((1 << 12, 16, 16), np.float32)
    x[:, :, 3] = a.reshape(1 << 12, 16)
    k = torch.from_numpy(x).cuda()
    parts = make_cache("fp8", 1 << 8, 16, 16, 16)
    nr.kv_cache_write(k, k, torch.arange(1 << 12, device="cuda"), *parts)
    want = ref.quant_fp8(x)
    assert np.array_equal(flat(parts[2]), want[1])
    assert np.array_equal(flat(parts[0]), want[0])


@pytest.mark.parametrize("dtype", [bf, torch.float32])
def test_rows_of_nan_and_infinity(nr, dtype):
    """All NaN: the scale's floor.  fp8 codes stay NaN; 4-bit codes have no NaN and
    become 6 of either sign.  Infinities take the largest code, others zero."""
    x = torch.randn(3, 1, 64)
    x[0] = float("nan")
    x[1, 0, ::2] = float("inf")
    x[2, 0, 33] = float("-inf")
    k = x.to(dtype).cuda()
    parts = make_cache("fp8", 3, 1, 1, 64)
    nr.kv_cache_write(k, k, torch.arange(3, device="cuda"), *parts)
    want = ref.quant_fp8(f32(k))
    got = flat(parts[0])
    assert np.array_equal(got[1:], want[0][1:]) and np.all((got[0] & 0x7F) == 0x7F)
    assert np.array_equal(flat(parts[2]), want[1])
    parts = make_cache("mxfp4", 3, 1, 1, 64)
    nr.kv_cache_write(k, k, torch.arange(3, device="cuda"), *parts)
    want = ref.quant_mxfp4(f32(k))
    got = flat(parts[0])
    assert np.array_equal(got[1:], want[0][1:]) and np.all((got[0] & 0x77) == 0x77)
    assert np.array_equal(flat(parts[2]), want[1])


def test_one_token_of_any_stride_and_side_streams(nr):
    """A single token's stride says nothing; inputs made on another stream are
    used after a wait."""
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        k = torch.randn(1, 5, 64, device="cuda").to(bf).as_strided((1, 5, 64), (3, 64, 1))
        parts = make_cache("fp8", 1, 2, 5, 64)
        before = [flat(p) for p in parts]
        slots = torch.tensor([1], device="cuda")
    torch.cuda.current_stream().wait_stream(s)
    nr.kv_cache_write(k, k, slots, *parts)
    check_written(parts, before, k, k, [1], "fp8")


def test_read_takes_its_type_from_given_outputs(nr):
    parts = make_cache("fp8", 2, 4, 1, 16)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    out = torch.empty(8, 1, 16, device="cuda")
    for kw in (dict(k_out=out), dict(rows=8, k_out=out), dict(rows=8, v_out=out)):
        k, v = nr.kv_cache_read(*parts, table, cu, **kw)
        assert k.dtype == v.dtype == torch.float32
    k, v = nr.kv_cache_read(*parts, table, cu, 8)
    assert k.dtype == v.dtype == bf


def test_no_tokens(nr):
    parts = make_cache("fp8", 2, 4, 2, 64)
    before = [flat(p) for p in parts]
    e = torch.empty(0, 2, 64, dtype=bf, device="cuda")
    nr.kv_cache_write(e, e, torch.empty(0, dtype=torch.int64, device="cuda"), *parts)
    assert all(np.array_equal(flat(p), b) for p, b in zip(parts, before))


# ---------------------------------------------------------------------------
# reading back
# ---------------------------------------------------------------------------
def run_read(nr, fmt, lens, heads, dim, page, dtype, extra=0, first=0, drop=(), interleaved=False,
             shift=0, seed=2):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    blocks = sum(need) + 2
    parts = make_cache(fmt, blocks, page, heads, dim, seed, interleaved)
    order = torch.randperm(blocks, generator=g).tolist()
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    for i, n in enumerate(need):
        for j in range(n):
            table[i, j] = order.pop()
    for s, j, value in drop:
        table[s, j] = value
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    rows = cu[-1] + extra
    canary = -77.0
    size = rows * heads * dim

    def out():  # `shift` elements past an aligned start
        t = torch.full((size + shift,), canary, dtype=dtype, device="cuda")
        return t[shift:].view(rows, heads, dim)

    ko, vo = out(), out()
    nr.kv_cache_read(*parts, table.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), k_out=ko,
                     v_out=vo)
    torch.cuda.synchronize()
    for o, c, s in ((ko, parts[0], parts[2]), (vo, parts[1], parts[3])):
        want = ref.read(c.cpu().numpy(), s.cpu().numpy(), table.numpy(), cu, rows)
        left = np.isnan(want)
        w = torch.from_numpy(want.astype(np.float32)).to(dtype)  # the f32 product, rounded once
        w[torch.from_numpy(left)] = canary
        assert torch.equal(o.cpu(), w)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("dtype", [bf, torch.float32])
@pytest.mark.parametrize("lens,page", [([1], 1), ([1], 16), ([0], 4), ([16], 16), ([17], 16),
                                       ([5, 0, 0, 33, 1, 64], 16), ([0, 0, 7], 3),
                                       ([300, 2], 128), ([3] * 40, 2)])
def test_read_lengths(nr, fmt, dtype, lens, page):
    run_read(nr, fmt, lens, 3, 64, page, dtype, extra=5)


@pytest.mark.parametrize("dim", [16, 48, 80, 112, 128, 256, 512])
def test_read_head_dims_fp8(nr, dim):
    run_read(nr, "fp8", [9, 30], 5, dim, 8, bf, interleaved=True)


@pytest.mark.parametrize("dim", [32, 96, 160, 256, 512])
def test_read_head_dims_mxfp4(nr, dim):
    run_read(nr, "mxfp4", [9, 30], 5, dim, 8, torch.float32, interleaved=True)


def test_read_leaves_rows_outside_the_sequences(nr):
    run_read(nr, "fp8", [10, 3], 2, 64, 4, bf, extra=70, first=9)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_read_missing_pages_are_zeros(nr, fmt):
    run_read(nr, fmt, [40, 9], 2, 64, 8, bf, drop=[(0, 1, -5), (0, 3, 1 << 30), (1, 0, 7)])


@pytest.mark.parametrize("dtype,shift", [(bf, 8), (torch.float32, 4)])
def test_read_into_outputs_that_start_16_bytes_past_32(nr, dtype, shift):
    run_read(nr, "fp8", [21], 3, 48, 8, dtype, shift=shift)


def test_read_more_sequences_than_are_searched_in_shared_memory(nr):
    run_read(nr, "fp8", [1, 0, 2] * 700, 1, 16, 2, bf, extra=3)


def test_read_table_too_narrow_for_a_length_reads_zeros(nr):
    """cu_seqlens beyond the table: the rows past its blocks are zeros."""
    parts = make_cache("fp8", 4, 4, 1, 16)
    table = torch.tensor([[2]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    k, v = nr.kv_cache_read(*parts, table, cu, 9)
    assert torch.count_nonzero(k[4:]) == 0 and torch.count_nonzero(v[4:]) == 0
    want = ref.held(parts[0].cpu().numpy(), parts[2].cpu().numpy())[2]
    assert np.array_equal(k[:4].float().cpu().numpy(),
                          torch.from_numpy(want).float().to(bf).float().numpy())


def test_read_nothing(nr):
    parts = make_cache("fp8", 2, 4, 2, 64)
    k, v = nr.kv_cache_read(*parts, torch.zeros(0, 1, dtype=torch.int32, device="cuda"),
                            torch.zeros(1, dtype=torch.int32, device="cuda"), 0)
    assert k.shape == (0, 2, 64) and v.shape == (0, 2, 64)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_a_cache_beyond_32_bits(nr, fmt):
    """Slots whose byte offsets pass 2^32 (and 2^31) are written and read."""
    heads, dim, page = 16, 256, 64
    width = dim if fmt == "fp8" else dim // 2
    blocks = (1 << 32) // (page * heads * width) + 40
    codes = [torch.zeros(blocks, page, heads, width, dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    if fmt == "fp8":
        scales = [torch.zeros(blocks, page, heads, device="cuda") for _ in range(2)]
    else:
        scales = [torch.full((blocks, page, heads, dim // 32), 127, dtype=torch.uint8, device="cuda")
                  for _ in range(2)]
    n = blocks * page
    slots = torch.tensor([n - 1, n // 2, n // 2 + 1, 5, n - page, 0])
    g = torch.Generator().manual_seed(3)
    k = torch.randn(6, heads, dim, generator=g).to(bf).cuda()
    v = torch.randn(6, heads, dim, generator=g).to(bf).cuda()
    nr.kv_cache_write(k, v, slots.cuda(), *codes, *scales)
    for src, c, s in ((k, codes[0], scales[0]), (v, codes[1], scales[1])):
        want = ref.quant(f32(src), fmt)
        at = slots.cuda()
        assert np.array_equal(c.view(n, heads, width)[at].cpu().numpy(), want[0])
        assert np.array_equal(s.view(n, heads, -1)[at].cpu().numpy().reshape(want[1].shape), want[1])
        assert int(torch.count_nonzero(c.view(n, -1).any(1))) == 6  # nothing else written
    table = torch.tensor([[blocks - 1], [n // 2 // page]], dtype=torch.int32).cuda()
    cu = torch.tensor([0, page, 2 * page], dtype=torch.int32).cuda()
    ko, _ = nr.kv_cache_read(*codes, *scales, table, cu, 2 * page)
    want = ref.held(*ref.quant(f32(k), fmt)).astype(np.float32)
    assert torch.equal(ko[page - 1].cpu(), torch.from_numpy(want[0]).to(bf))
    assert torch.equal(ko[0].cpu(), torch.from_numpy(want[4]).to(bf))
    assert torch.equal(ko[page + n // 2 % page].cpu(), torch.from_numpy(want[1]).to(bf))


def test_outputs_past_2_to_31_elements(nr):
    """read: row offsets beyond 2^31 elements of the output."""
    heads, dim, page = 8, 512, 64
    rows = (1 << 31) // (heads * dim) + 100
    blocks = 64
    parts = make_cache("fp8", blocks, page, heads, dim)
    seqs = -(-rows // (blocks * page))
    table = torch.arange(blocks, dtype=torch.int32).repeat(seqs, 1).cuda()
    cu = (torch.arange(seqs + 1) * blocks * page).clamp(max=rows).to(torch.int32).cuda()
    k, v = nr.kv_cache_read(*parts, table, cu, rows)
    for r in (0, rows - 1, (1 << 31) // (heads * dim), (1 << 31) // (heads * dim) - 1):
        b, p = divmod(r % (blocks * page), page)
        for o, c, s in ((k, parts[0], parts[2]), (v, parts[1], parts[3])):
            want = ref.held_fp8(c[b, p].cpu().numpy(), s[b, p].cpu().numpy()).astype(np.float32)
            assert torch.equal(o[r].cpu(), torch.from_numpy(want).to(bf))


def test_two_streams_and_a_replayed_graph(nr):
    """Writes on two streams into caches of their own, and a write + read
    captured and replayed with new inputs in the same places."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = []
    for i in range(2):
        parts = make_cache("fp8", 8, 16, 4, 128, seed=i)
        k = torch.randn(100, 4, 128, device="cuda", dtype=bf)
        sets.append((parts, k, torch.randperm(128, device="cuda")[:100], [flat(p) for p in parts]))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (parts, k, slots, _) in zip(streams, sets):
            with torch.cuda.stream(s):
                nr.kv_cache_write(k, k, slots, *parts)
    torch.cuda.synchronize()
    for parts, k, slots, before in sets:
        check_written(parts, before, k, k, slots.tolist(), "fp8")

    parts, k, slots, _ = sets[0]
    slots.copy_(torch.arange(100))
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    cu = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nr.kv_cache_write(k, k, slots, *parts)
        ko, vo = nr.kv_cache_read(*parts, table, cu, 100)
    for seed in range(3):
        k.copy_(torch.randn(100, 4, 128, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        want = ref.held(*ref.quant(f32(k), "fp8")).astype(np.float32)
        assert torch.equal(ko.cpu(), torch.from_numpy(want).to(bf))
        assert torch.equal(vo, ko)
