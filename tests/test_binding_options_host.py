"""Options of the cache and group-norm calls that are not plain numbers, on the
CPU with the launch replaced by a recorder: a call passes the values that its
options have at that call, whatever an earlier call of the same layout was given,
and nothing that a caller passed is kept."""
import pytest
import torch

bf, I32 = torch.bfloat16, torch.int32


@pytest.fixture
def nrt(lib_path, monkeypatch):
    """The binding with its device check off; launched(): the arguments of the last launch."""
    import normalisation_rope_transformers_gb300 as nrt
    calls = []
    monkeypatch.setattr(nrt, "_cuda", lambda *ts: None)
    monkeypatch.setattr(nrt, "_launch", lambda device, fn, *args: calls.append(args))
    monkeypatch.setattr(nrt, "_checked", {})
    nrt.launched = lambda: calls[-1]
    yield nrt
    del nrt.launched


def parts(blocks=4, page=4, heads=2, dim=64):
    codes = [torch.zeros(blocks, page, heads, dim, dtype=torch.uint8) for _ in range(2)]
    return codes + [torch.zeros(blocks, page, heads) for _ in range(2)]


def kept(entry):
    """Everything in the keys, nested tuples opened."""
    for v in entry:
        if isinstance(v, tuple):
            yield from kept(v)
        else:
            yield v


def no_tensor_kept(nrt):
    return not any(isinstance(v, torch.Tensor) for key in nrt._checked for v in kept(key))


def floats(args):
    return [a for a in args if isinstance(a, float)]


def test_rows_changed_in_place(nrt):
    cu = torch.tensor([0, 5], dtype=I32)
    rows = cu[-1]
    for n in (5, 12, 5):
        cu[1] = n
        k, v = nrt.kv_cache_read(*parts(), torch.zeros(1, 4, dtype=I32), cu, rows)
        assert k.shape == v.shape == (n, 2, 64) and nrt.launched()[-2] == n
    assert no_tensor_kept(nrt)


def test_group_norm_options_changed_in_place(nrt):
    x = torch.zeros(2, 5, 64, dtype=bf)
    eps, groups = torch.tensor(0.5), torch.tensor(8)
    for e, n in ((0.5, 8), (0.25, 8), (0.25, 4), (0.5, 8)):
        eps.fill_(e)
        groups.fill_(n)
        _, mean, _ = nrt.group_norm(x, groups, eps=eps, stats=True)
        assert mean.shape == (2, n) and floats(nrt.launched()) == [e]
    assert no_tensor_kept(nrt)


def preamble(nrt, positions=None, **kw):
    t, w = torch.zeros(3, 2, 64, dtype=bf), torch.ones(64)
    p = torch.zeros(3, dtype=I32) if positions is None else positions
    nrt.qk_norm_rope_cache(t, t, t, w, w, p, torch.arange(3), *parts(), **kw)
    args = nrt.launched()
    (cfg,) = [a for a in args if isinstance(a, nrt.RopeConfig)]
    return floats(args)[0], args[-3], cfg  # eps, gemma


def test_preamble_options_changed_in_place(nrt):
    eps, theta, gemma = torch.tensor(0.5), torch.tensor(1e4), torch.tensor(0)
    rot, inter = torch.tensor(64), torch.tensor(0)
    l3 = torch.tensor([8.0, 1.0, 4.0, 8192.0])
    kw = dict(eps=eps, theta=theta, gemma=gemma, rotary_dim=rot, interleaved=inter,
              llama3=tuple(l3))
    preamble(nrt, **kw)
    for t, value, field in ((theta, 5e5, "theta"), (rot, 32, "rotary_dim"), (inter, 1, "interleaved")):
        t.fill_(value)
        assert getattr(preamble(nrt, **kw)[2], field) == value
    eps.fill_(0.25)
    gemma.fill_(1)
    assert preamble(nrt, **kw)[:2] == (0.25, 1)
    l3[0] = 32.0
    assert preamble(nrt, **kw)[2].llama3_factor == 32.0
    assert no_tensor_kept(nrt)


def test_preamble_sections_changed_in_place(nrt):
    sections = torch.tensor([16, 8, 8])
    pos = torch.zeros(3, 3, dtype=I32)
    for s in ((16, 8, 8), (8, 8, 16), (16, 8, 8)):
        sections.copy_(torch.tensor(s))
        cfg = preamble(nrt, pos, mrope_sections=sections)[2]
        assert tuple(cfg.mrope_section) == s
    assert no_tensor_kept(nrt)


def test_plain_options_of_one_layout_are_one_entry(nrt):
    x = torch.zeros(2, 5, 64, dtype=bf)
    for eps in (1e-5, 1e-5, torch.tensor(0.5), 0.5):
        nrt.group_norm(x, 8, eps=eps)
    assert len(nrt._checked) == 2
    for rows in (5, torch.tensor(5)):
        nrt.kv_cache_read(*parts(), torch.zeros(1, 4, dtype=I32), torch.tensor([0, 5], dtype=I32), rows)
    assert len(nrt._checked) == 3
