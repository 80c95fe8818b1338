"""The norms around a block against 64 bits: types, gates, strides, rows in place."""

import math

import pytest
import torch

import prompt64 as p64

pytestmark = pytest.mark.gpu
F, B, H16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def fgm():
    import fine_grained_moe_gb300 as m
    m.lib()
    return m


def rows(N, D, dtype, g, size=1.0):
    t = torch.randn(N, D, generator=g, device="cuda") * size
    t[:, ::97] *= 9
    return t.to(dtype)


def gate_of(kind, N, D, dtype, g):
    shape = {None: None, "channel": (D,), "token": (N, 1), "full": (N, D)}[kind]
    return None if shape is None else torch.randn(shape, generator=g, device="cuda").to(dtype)


def check(fgm, h, y=None, post=None, gate=None, pre=None, post_norm=True, pre_norm=True, a=1.0, b=1.0, offset=0.0, eps=1e-6, **kw):
    want, dw, wn, dn = p64.block(h, y, post, gate, pre, post_norm, a, b, offset, eps)
    o, n = fgm.block_norm(h, y, post_gain=post, gate=gate, pre_gain=pre, post_norm=post_norm, pre_norm=pre_norm, residual_scale=a, block_scale=b,
                          gain_offset=offset, eps=eps, **kw)
    p64.within(o, want, p64.rounded(want, dw, o.dtype))
    if pre_norm:
        p64.within(n, wn, p64.rounded(wn, dn, n.dtype))
    else:
        assert n is None
    return o, n


@pytest.mark.parametrize("D", [1, 7, 8, 33, 256, 1000, 1409, 2816, 4096, 4104, 5003, 8192, 8200, 16384, 16383])
@pytest.mark.parametrize("N", [1, 5, 700])
def test_widths(fgm, N, D):
    g = torch.Generator(device="cuda").manual_seed(D)
    post, pre = (torch.rand(D, generator=g, device="cuda") + 0.5 for _ in range(2))
    check(fgm, rows(N, D, B, g, 2.0), rows(N, D, B, g), post=post, pre=pre)


@pytest.mark.parametrize("h", [F, B, H16])
@pytest.mark.parametrize("y", [F, B, H16])
@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("D", [256, 259])
def test_types_and_gates(fgm, h, y, gate, D):
    g = torch.Generator(device="cuda").manual_seed(7)
    N = 1300
    for gains, xn in ((F, B), (B, F), (H16, H16)):
        post, pre = ((torch.rand(D, generator=g, device="cuda") + 0.5).to(gains) for _ in range(2))
        out = torch.empty(N, D, dtype=xn, device="cuda")
        check(fgm, rows(N, D, h, g), rows(N, D, y, g), post=post, pre=pre, gate=gate_of(gate, N, D, y, g), a=0.7, b=-1.3, offset=1.0, xn=out)


@pytest.mark.parametrize("D", [512, 515, 9000])
def test_parts_left_out(fgm, D):
    g = torch.Generator(device="cuda").manual_seed(8)
    h, y = rows(901, D, F, g), rows(901, D, B, g)
    gain = torch.rand(D, generator=g, device="cuda")
    for kind in (None, "channel", "token", "full"):
        gate = gate_of(kind, 901, D, B, g)
        check(fgm, h, y, gate=gate)
        check(fgm, h, y, gate=gate, post_norm=False)
        check(fgm, h, y, gate=gate, post_norm=False, pre_norm=False)
        check(fgm, h, y, gate=gate, post=gain, pre_norm=False)
        check(fgm, h, y, gate=gate, pre=gain, offset=1.0)
    check(fgm, h)
    check(fgm, h, pre=gain, a=0.5)
    check(fgm, h, pre_norm=False, a=0.5)


@pytest.mark.parametrize("D", [640, 641])
def test_in_place(fgm, D):
    g = torch.Generator(device="cuda").manual_seed(9)
    for h_type in (F, B):
        h, y = rows(777, D, h_type, g), rows(777, D, B, g)
        o, n = check(fgm, h, y)
        h1, y1 = h.clone(), y.clone()
        o1, n1 = fgm.block_norm(h1, y1, h_out=h1, xn=y1)
        assert o1 is h1 and n1 is y1 and torch.equal(o1, o) and torch.equal(n1, n)


@pytest.mark.parametrize("D", [128, 130])
def test_slices(fgm, D):
    g = torch.Generator(device="cuda").manual_seed(10)
    wide = rows(500, 4 * D, B, g)
    h, y, gate, o = (wide[:, i * D:(i + 1) * D] for i in range(4))
    want = check(fgm, h.clone(), y.clone(), gate=gate.clone())
    got = fgm.block_norm(h, y, gate=gate, h_out=o)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # the last column of wide rows as a gate a token, one row's gate for all
    check(fgm, h, y, gate=wide[:, 1:2])
    check(fgm, h, y, gate=wide[0, :D])
    check(fgm, h, y, gate=wide[:1, :D].expand(500, D))


def test_values(fgm):
    g = torch.Generator(device="cuda").manual_seed(11)
    h, y = rows(12, 384, F, g), rows(12, 384, F, g)
    y[1], h[2], y[3] = 0, 0, y[3] * 1e-12
    h[4] *= 1e15
    check(fgm, h, y)
    check(fgm, h, y, eps=0.1)
    y[5, 7], h[6, 1] = math.nan, math.nan
    o, n = fgm.block_norm(h, y)
    assert o[5].isnan().all() and n[[5, 6]].isnan().all() and o[6].isnan().sum() == 1
    rest = [i for i in range(12) if i not in (5, 6)]
    assert o[rest].isfinite().all() and n[rest].isfinite().all()


def test_rows_that_span_32_bits(fgm):
    N, D = 262_150, 8200
    h = torch.zeros(N, D, dtype=B, device="cuda")
    h[-3:] = rows(3, D, B, torch.Generator(device="cuda").manual_seed(1))
    o, n = fgm.block_norm(h, h_out=h)
    want, dw, wn, dn = p64.block(o[-3:], None, None, None, None, True, 1.0, 1.0, 0.0, 1e-6)
    p64.within(n[-3:], wn, p64.rounded(wn, dn, B))
    assert (n[:5] == 0).all()


def test_binding_refusals(fgm):
    h, y = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 64, device="cuda")
    for call in (lambda: fgm.block_norm(h[0]), lambda: fgm.block_norm(h, y[:3]), lambda: fgm.block_norm(h.double()), lambda: fgm.block_norm(h.t(), y.t()),
                 lambda: fgm.block_norm(h, y, post_gain=torch.ones(63, device="cuda")), lambda: fgm.block_norm(h, y, gate=torch.ones(4, device="cuda")),
                 lambda: fgm.block_norm(h, y, post_gain=torch.ones(64, device="cuda"), pre_gain=torch.ones(64, device="cuda").bfloat16()),
                 lambda: fgm.block_norm(h, y, h_out=h.bfloat16()), lambda: fgm.block_norm(h, y, pre_norm=False, xn=y), lambda: fgm.block_norm(h, y, h_out=h, xn=h),
                 lambda: fgm.block_norm(h, gate=h), lambda: fgm.block_norm(h, y, post_norm=False, post_gain=torch.ones(64, device="cuda")),
                 lambda: fgm.block_norm(h, y, eps=-1.0), lambda: fgm.block_norm(h, y, h_out=y), lambda: fgm.block_norm(h.expand(4, 64)[:0], y[:0])):
        with pytest.raises(fgm.FgmError):
            call()
